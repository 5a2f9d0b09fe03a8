"""C ABI of the token-side operators, no GPU: sizes of the descriptions, every
refusal with its status (pointers are fake addresses, never dereferenced) and
the workspace sizes."""

import ctypes

import pytest

from kan_testutil import ensure_built


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from kolmogorov_arnold_network_amd import _lib
    return _lib


# fake, 256-aligned device addresses 1 TiB apart
A = [(k + 1) << 40 for k in range(16)]
SIZE_MAX = ctypes.c_size_t(-1).value


def embed(L, **kw):
    d = dict(N=10, V=20, D=8, dtype=0, row_dtype=0, id_dtype=0, scale=1.0)
    d.update(kw)
    return L.kan_embed_desc_t(*d.values())


def recur(L, **kw):
    d = dict(B=2, T=6, D=8, x_row=8, x_seq=48, g_row=8, g_seq=48, dx_row=8, dx_seq=48, dg_row=8, dg_seq=48,
             dtype=0, grad_dtype=0)
    d.update(kw)
    return L.kan_recur_desc_t(*d.values())


def distill(L, **kw):
    d = dict(N=4, V=100, K=5, z_row=100, dz_row=100, dtype=0, teacher_dtype=0, id_dtype=0, grad_dtype=0, tau=1.0)
    d.update(kw)
    return L.kan_distill_desc_t(*d.values())


def test_struct_layout(L):
    assert ctypes.sizeof(L.kan_embed_desc_t) == 3 * 8 + 4 * 4
    assert ctypes.sizeof(L.kan_recur_desc_t) == 11 * 8 + 2 * 4
    assert ctypes.sizeof(L.kan_distill_desc_t) == 5 * 8 + 5 * 4 + 4


NAN, INF = float("nan"), float("inf")
EMBED_BAD = [(dict(N=-1), "SHAPE"), (dict(V=0), "SHAPE"), (dict(D=0), "SHAPE"), (dict(N=(1 << 24) + 1), "SHAPE"),
             (dict(V=(1 << 26) + 1), "SHAPE"), (dict(D=(1 << 23) + 1), "SHAPE"), (dict(V=1 << 20, D=1 << 18), "SHAPE"),
             (dict(N=1 << 20, D=1 << 18), "SHAPE"), (dict(dtype=2), "DTYPE"),
             (dict(row_dtype=-1), "DTYPE"), (dict(id_dtype=2), "DTYPE"), (dict(scale=NAN), "UNSUPPORTED"),
             (dict(scale=INF), "UNSUPPORTED")]
RECUR_BAD = [(dict(B=-1), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(D=0), "SHAPE"), (dict(x_row=-1), "SHAPE"),
             (dict(g_seq=1 << 41), "SHAPE"), (dict(B=1 << 23, D=64), "SHAPE"), (dict(dtype=3), "DTYPE"),
             (dict(grad_dtype=-2), "DTYPE"), (dict(T=1 << 31), "SHAPE"),
             (dict(B=1 << 21, T=1 << 20, x_seq=1 << 40), "SHAPE")]
DISTILL_BAD = [(dict(N=-1), "SHAPE"), (dict(N=(1 << 21) + 1), "SHAPE"), (dict(V=0), "SHAPE"), (dict(K=0), "SHAPE"),
               (dict(K=1025), "SHAPE"), (dict(z_row=99), "SHAPE"), (dict(dtype=2), "DTYPE"),
               (dict(teacher_dtype=2), "DTYPE"), (dict(id_dtype=-1), "DTYPE"), (dict(tau=0.0), "UNSUPPORTED"),
               (dict(tau=-1.0), "UNSUPPORTED"), (dict(tau=NAN), "UNSUPPORTED"), (dict(tau=INF), "UNSUPPORTED")]


def calls(L, kind, d):
    """(entry point, its arguments) of every call of an operator, with valid pointers."""
    lib = L.lib()
    if kind == "embed":
        return [(lib.kan_embed_forward, [d, A[0], A[1], A[2], None]),
                (lib.kan_embed_backward, [d, A[0], A[1], A[2], A[3], 1 << 39, None])]
    if kind == "recur":
        return [(lib.kan_recur_forward, [d, A[0], A[1], A[2], A[3], A[4], A[5], A[6], 1 << 39, None]),
                (lib.kan_recur_backward, [d, A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], A[8], A[9], A[10], 1 << 39,
                                          None])]
    return [(lib.kan_distill_forward, [d, A[0], A[1], A[2], A[3], A[4], A[5], A[6], 1 << 39, None]),
            (lib.kan_distill_backward, [d, A[0], A[1], A[2], A[3], A[4], A[5], A[6], None]),
            (lib.kan_distill_step, [d, A[0], A[1], A[2], A[3], A[4], A[5], A[6], 1 << 39, None])]


def size(L, kind, d):
    f = getattr(L.lib(), "kan_%s_workspace_size" % kind)
    return f(d, 0) if kind == "recur" else f(d)


ALL_BAD = [("embed", kw, c) for kw, c in EMBED_BAD] + [("recur", kw, c) for kw, c in RECUR_BAD] + [
    ("distill", kw, c) for kw, c in DISTILL_BAD]


@pytest.mark.parametrize("kind,kw,code", ALL_BAD)
def test_bad_descriptions(L, kind, kw, code):
    d = globals()[kind](L, **kw)
    assert size(L, kind, d) == SIZE_MAX
    for fn, args in calls(L, kind, d):
        assert fn(*args) == getattr(L, "KAN_ERR_" + code)


@pytest.mark.parametrize("kind", ["embed", "recur", "distill"])
def test_null_description(L, kind):
    assert size(L, kind, None) == SIZE_MAX
    for fn, args in calls(L, kind, None):
        assert fn(*args) == L.KAN_ERR_NULL


def test_gradient_descriptions(L):
    """Fields of the gradients are looked at by the calls that write them."""
    lib = L.lib()
    for kw, code in ((dict(dz_row=99), "SHAPE"), (dict(grad_dtype=2), "DTYPE")):
        d = distill(L, **kw)
        assert size(L, "distill", d) != SIZE_MAX
        for fn, args in calls(L, "distill", d)[1:]:
            assert fn(*args) == getattr(L, "KAN_ERR_" + code)
    # rows of dx that overlap each other, and sequences that cut into rows
    for kw in (dict(dx_row=7), dict(dg_seq=40), dict(dx_row=0), dict(dx_row=16, dx_seq=12), dict(dx_seq=0)):
        fn, args = calls(L, "recur", recur(L, **kw))[1]
        assert fn(*args) == L.KAN_ERR_SHAPE
    # a gradient in each of the layouts that are accepted reaches the workspace
    # check: [B, T, D], [T, B, D], halves of one array
    for kw, dx, dg in ((dict(), A[7], A[8]), (dict(dx_row=16, dx_seq=8, dg_row=16, dg_seq=8), A[7], A[8]),
                       (dict(dx_row=16, dx_seq=96, dg_row=16, dg_seq=96), A[7], A[7] + 32)):
        d = recur(L, T=300000, x_seq=8 * 300000, g_seq=8 * 300000,
                  **{k: v * 50000 if k.endswith("seq") and v > 16 else v for k, v in dict(
                      dict(dx_seq=48, dg_seq=48), **kw).items()})
        fn, args = calls(L, "recur", d)[1]
        args[8], args[9], args[12] = dx, dg, 0
        need = lib.kan_recur_workspace_size(d, 1)
        assert need > 0 and fn(*args) == L.KAN_ERR_WORKSPACE


@pytest.mark.parametrize("kind", ["embed", "recur", "distill"])
def test_required_and_misaligned_pointers(L, kind):
    d = globals()[kind](L)
    optional = {"embed": [[], []], "recur": [[2, 3, 5], [2, 3, 6, 7, 8, 9]], "distill": [[3], [3], [3]]}[kind]
    element = {"embed": [[], []], "recur": [[0, 1], [0, 1, 7, 8]], "distill": [[0], [0, 6], [0, 5]]}[kind]
    for (fn, args), opt, el in zip(calls(L, kind, d), optional, element):
        pointers = [i for i, v in enumerate(args[1:]) if v in A and not (isinstance(args[i + 2] if i + 2 < len(args)
                                                                                   else None, int) and
                                                                         args[i + 2] == 1 << 39)]
        for i in pointers:
            if i not in opt:
                bad = list(args)
                bad[1 + i] = None
                assert fn(*bad) == L.KAN_ERR_NULL, (fn.__name__, i)
            bad = list(args)
            bad[1 + i] += 2 if i in el else 8
            assert fn(*bad) == L.KAN_ERR_ALIGN, (fn.__name__, i)


def test_overlaps(L):
    for kind, pairs in (("embed", [[(1, 3), (2, 3)], [(1, 3), (2, 3), (2, 4), (3, 4)]]),
                        ("recur", [[(1, 5), (2, 5), (3, 6), (4, 5), (5, 6)],
                                   [(1, 8), (5, 8), (6, 9), (7, 10), (2, 9), (8, 9), (8, 10)]]),
                        ("distill", [[(1, 5), (3, 6), (5, 6)], [(1, 7), (5, 7), (6, 7)], [(1, 6), (4, 5), (5, 6)]])):
        for (fn, args), some in zip(calls(L, kind, globals()[kind](L)), pairs):
            for i, j in some:
                bad = list(args)
                bad[j] = bad[i]
                assert fn(*bad) == L.KAN_ERR_ALIAS, (fn.__name__, i, j)
    # halves of one array whose columns meet
    d = recur(L, dx_row=15, dx_seq=90, dg_row=15, dg_seq=90)
    fn, args = calls(L, "recur", d)[1]
    args[9] = args[8] + 4 * 7
    assert fn(*args) == L.KAN_ERR_ALIAS


def test_one_gradient_without_the_other(L):
    fn, args = calls(L, "recur", recur(L))[1]
    args[8] = None
    assert fn(*args) == L.KAN_ERR_NULL


def test_workspaces(L):
    lib = L.lib()
    assert size(L, "embed", embed(L, N=0)) == 0 and size(L, "recur", recur(L, B=0)) == 0
    assert size(L, "distill", distill(L, N=0)) == 0
    n = size(L, "embed", embed(L, N=5000, V=700, D=96))
    assert n >= 5000 * 8 + 701 * 4 and n % 256 == 0
    d = embed(L, N=5000, V=700, D=96)
    assert lib.kan_embed_backward(d, A[0], A[1], A[2], A[3], n - 1, None) == L.KAN_ERR_WORKSPACE
    assert lib.kan_embed_backward(d, A[0], A[1], A[2], None, n, None) == L.KAN_ERR_NULL
    assert lib.kan_embed_backward(d, A[0], A[1], A[2], A[3] + 64, n, None) == L.KAN_ERR_ALIGN
    assert lib.kan_recur_workspace_size(recur(L), 2) == SIZE_MAX
    # as many rows as fill the GPU, and a batch of short sequences, need none
    for B, T, D in ((8, 4096, 2048), (64, 197, 768), (1, 1, 1)):
        assert size(L, "recur", recur(L, B=B, T=T, D=D, x_row=D, x_seq=T * D, g_row=D, g_seq=T * D)) == 0
    assert size(L, "recur", recur(L, B=1, T=65536, D=64, x_row=64, g_row=64)) > 0


def test_step_arguments(L):
    lib = L.lib()
    d = recur(L, T=1)
    ok = [d, 4, A[0], A[1], A[2], A[3], A[4], None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.kan_recur_step(*a)

    assert call(_0=recur(L)) == L.KAN_ERR_SHAPE                      # T is 6
    assert call(_0=None) == L.KAN_ERR_NULL
    assert call(_1=-1) == L.KAN_ERR_SHAPE
    assert call(_1=1, _5=None) == L.KAN_ERR_SHAPE                    # fewer states than sequences, no slots
    for i in (2, 3, 4, 6):
        assert call(**{"_%d" % i: None}) == L.KAN_ERR_NULL
    for i, by in ((2, 2), (3, 2), (4, 8), (5, 8), (6, 8)):
        assert call(**{"_%d" % i: ok[i] + by}) == L.KAN_ERR_ALIGN
    assert call(_6=A[2]) == L.KAN_ERR_ALIAS and call(_2=A[2]) == L.KAN_ERR_ALIAS and call(_6=A[0]) == L.KAN_ERR_ALIAS
    assert lib.kan_recur_step(recur(L, B=0, T=1), 0, None, None, None, None, None, None) == L.KAN_OK


def test_empty_calls_launch_nothing(L):
    """No rows: valid without any pointer but the ones that are written."""
    lib = L.lib()
    assert lib.kan_embed_forward(embed(L, N=0), None, A[0], None, None) == L.KAN_OK
    assert lib.kan_recur_forward(recur(L, B=0), *[None] * 7, 0, None) == L.KAN_OK
    assert lib.kan_recur_forward(recur(L, T=0), *[None] * 7, 0, None) == L.KAN_OK
    assert lib.kan_recur_backward(recur(L, B=0), *[None] * 11, 0, None) == L.KAN_OK
    d = distill(L, N=0)
    assert lib.kan_distill_forward(d, *[None] * 7, 0, None) == L.KAN_OK
    assert lib.kan_distill_backward(d, *[None] * 8) == L.KAN_OK
    assert lib.kan_distill_step(d, *[None] * 7, 0, None) == L.KAN_OK
