"""C ABI of the gated delta rule and of the join, no GPU: sizes of the
descriptions, every refusal with its status (pointers are fake addresses, never
dereferenced) and the workspace sizes."""

import ctypes

import pytest

from kan_testutil import ensure_built


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from kolmogorov_arnold_network_amd import _lib
    return _lib


A = [(k + 1) << 40 for k in range(20)]       # fake, 256-aligned device addresses 1 TiB apart
SIZE_MAX = ctypes.c_size_t(-1).value
WS = 1 << 39
NAN, INF = float("nan"), float("inf")
HEADS = dict(q=(96, 16, 8), k=(96, 16, 8), v=(240, 40, 10), dq=(96, 16, 8), dk=(96, 16, 8), dv=(240, 40, 10))


def delta(L, **kw):
    d = dict(B=2, T=6, Hk=2, Hv=4, Dk=8, Dv=10, **HEADS, dtype=0, flags=0, scale=1.0)
    d.update(kw)
    return L.kan_delta_desc_t(*(L.kan_heads_t(*v) if isinstance(v, tuple) else v for v in d.values()))


def join(L, **kw):
    d = dict(N=6, D=20, h_row=20, r_row=24, gate_row=20, dtype=0, res_dtype=0, row_dtype=0, activation=0, flags=3,
             scale=1.0, eps=1e-6)
    d.update(kw)
    return L.kan_join_desc_t(*d.values())


def calls(L, kind, d):
    """(entry point, its arguments) of every call of an operator, with valid pointers."""
    lib = L.lib()
    if kind == "delta":
        return [(lib.kan_delta_forward, [d, *A[:9], A[9], WS, None]),
                (lib.kan_delta_backward, [d, *A[:15], A[15], WS, None])]
    return [(lib.kan_join_forward, [d, *A[:8], None]), (lib.kan_join_backward, [d, *A[:13], A[13], WS, None])]


def size(L, kind, d):
    return L.lib().kan_delta_workspace_size(d, 1) if kind == "delta" else L.lib().kan_join_workspace_size(d)


def test_struct_layout(L):
    assert ctypes.sizeof(L.kan_heads_t) == 24
    assert ctypes.sizeof(L.kan_delta_desc_t) == 6 * 8 + 6 * 24 + 3 * 4 + 4
    assert ctypes.sizeof(L.kan_join_desc_t) == 5 * 8 + 7 * 4 + 4


BAD = [("delta", kw, c) for kw, c in [
    (dict(B=-1), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(Hk=0), "SHAPE"), (dict(Hv=0), "SHAPE"), (dict(Hk=3), "SHAPE"),
    (dict(Dk=0), "SHAPE"), (dict(Dk=129), "SHAPE"), (dict(Dv=0), "SHAPE"), (dict(Dv=1025), "SHAPE"),
    (dict(B=1 << 17), "SHAPE"), (dict(B=1 << 8, T=1 << 20), "SHAPE"), (dict(Hv=1 << 17, Dv=1024), "SHAPE"),
    (dict(q=(-1, 16, 8)), "SHAPE"), (dict(k=(96, (1 << 24) + 1, 8)), "SHAPE"), (dict(v=(240, 40, 1 << 41)), "SHAPE"),
    (dict(dtype=2), "DTYPE"), (dict(dtype=-1), "DTYPE"), (dict(flags=2), "UNSUPPORTED"),
    (dict(scale=NAN), "UNSUPPORTED"), (dict(scale=INF), "UNSUPPORTED")]] + [("join", kw, c) for kw, c in [
        (dict(N=-1), "SHAPE"), (dict(D=0), "SHAPE"), (dict(D=8193), "SHAPE"), (dict(N=(1 << 25) + 1), "SHAPE"),
        (dict(N=(1 << 23) + 1, D=1025), "SHAPE"), (dict(N=(1 << 21) + 1, D=4097), "SHAPE"), (dict(h_row=-1), "SHAPE"),
        (dict(r_row=1 << 41), "SHAPE"), (dict(gate_row=-5), "SHAPE"), (dict(dtype=2), "DTYPE"),
        (dict(res_dtype=-1), "DTYPE"), (dict(row_dtype=7), "DTYPE"), (dict(activation=2), "UNSUPPORTED"),
        (dict(flags=4), "UNSUPPORTED"), (dict(scale=INF), "UNSUPPORTED"), (dict(eps=-1e-9), "UNSUPPORTED"),
        (dict(eps=NAN), "UNSUPPORTED")]]


@pytest.mark.parametrize("kind,kw,code", BAD)
def test_bad_descriptions(L, kind, kw, code):
    d = globals()[kind](L, **kw)
    assert size(L, kind, d) == SIZE_MAX
    for fn, args in calls(L, kind, d):
        assert fn(*args) == getattr(L, "KAN_ERR_" + code)


@pytest.mark.parametrize("kind", ["delta", "join"])
def test_null_description(L, kind):
    assert size(L, kind, None) == SIZE_MAX
    for fn, args in calls(L, kind, None):
        assert fn(*args) == L.KAN_ERR_NULL


# indexes into the pointers of (forward, backward): those that may be NULL, those that need an element's alignment alone
OPTIONAL = {"delta": [[5, 6, 8], [5, 6, 8, 14]], "join": [[1, 2, 3, 4], [3, 4, 5, 9, 10, 11, 12]]}
ELEMENT = {"delta": [[0, 1, 2], [0, 1, 2, 9, 10, 11]], "join": [[0, 1, 2], [0, 5]]}


@pytest.mark.parametrize("kind", ["delta", "join"])
def test_required_and_misaligned_pointers(L, kind):
    d = globals()[kind](L)
    for (fn, args), optional, element in zip(calls(L, kind, d), OPTIONAL[kind], ELEMENT[kind]):
        for i in range(sum(v in A for v in args[1:])):
            bad = list(args)
            bad[1 + i] = None
            if i not in optional and not (kind == "join" and fn.__name__ == "kan_join_backward" and i in (6, 7)):
                assert fn(*bad) == L.KAN_ERR_NULL, (fn.__name__, i)
            bad[1 + i] = args[1 + i] + (2 if i in element else 8)
            assert fn(*bad) == L.KAN_ERR_ALIGN, (fn.__name__, i)


def test_outputs_apart_from_everything(L):
    outs = {"delta": [[7, 8, 9], [9, 10, 11, 12, 13, 14, 15]], "join": [[5, 6, 7], [8, 9, 10, 11, 12, 13]]}
    for kind, both in outs.items():
        for (fn, args), out in zip(calls(L, kind, globals()[kind](L)), both):
            n = sum(v in A for v in args[1:])
            for o in out:
                for i in range(n):
                    if i != o:
                        bad = list(args)
                        bad[1 + o] = bad[1 + i]
                        assert fn(*bad) == L.KAN_ERR_ALIAS, (fn.__name__, o, i)


def _gradients(L, at=None, **kw):
    """Status of a backward call with a workspace of one byte too few: WORKSPACE if the gradients' layout passes so far."""
    d = delta(L, **kw)
    fn, args = calls(L, "delta", d)[1]
    if at is not None:
        args[10], args[11], args[12] = (A[16] + o for o in at)
    args[17] = L.lib().kan_delta_workspace_size(d, 1) - 1
    return fn(*args)


def test_gradients_that_overlap_themselves(L):
    for kw in (dict(dq=(96, 15, 8)), dict(dq=(96, 16, 7)), dict(dk=(95, 16, 8)), dict(dv=(0, 40, 10)),
               dict(dv=(240, 0, 10)), dict(dv=(240, 40, 0)), dict(dq=(7, 16, 96)), dict(dk=(8, 16, 95))):
        assert _gradients(L, **kw) == L.KAN_ERR_SHAPE, kw
    # any order of the dimensions; and the inputs may repeat rows, heads and sequences
    for kw in (dict(q=(0, 0, 0), k=(0, 0, 0), v=(0, 0, 0)), dict(dq=(16, 32, 8), dk=(16, 32, 8)), dict(dq=(8, 16, 96))):
        assert _gradients(L, **kw) == L.KAN_ERR_WORKSPACE, kw


def test_gradients_as_slices_of_rows(L):
    """dq | dk | dv in the rows of one array, and what is not such slices."""
    def status(row=72, at=(0, 64, 128)):
        d = delta(L, dq=(6 * row, row, 8), dk=(6 * row, row, 8), dv=(6 * row, row, 10))
        fn, args = calls(L, "delta", d)[1]
        args[10], args[11], args[12] = (A[16] + o for o in at)
        args[13] = args[1]                        # dg lies on q, the check after the gradients' layouts
        return fn(*args), _gradients(L, at, dq=(6 * row, row, 8), dk=(6 * row, row, 8), dv=(6 * row, row, 10))
    assert status() == (L.KAN_ERR_ALIAS, L.KAN_ERR_WORKSPACE)
    assert status(at=(0, 66, 130))[1] == status(at=(0, 62, 128))[1] == L.KAN_ERR_ALIGN


@pytest.mark.parametrize("row,at", [(72, (0, 60, 128)), (72, (0, 64, 124)), (71, (0, 64, 128)), (72, (64, 0, 60)),
                                    (72, (0, 0, 128))])
def test_gradients_that_are_no_slices(L, row, at):
    d = delta(L, dq=(6 * row, row, 8), dk=(6 * row, row, 8), dv=(6 * row, row, 10))
    fn, args = calls(L, "delta", d)[1]
    args[10], args[11], args[12] = (A[16] + o for o in at)
    assert fn(*args) == L.KAN_ERR_ALIAS


def test_workspaces(L):
    lib = L.lib()
    for p in (0, 1):
        n = lib.kan_delta_workspace_size(delta(L), p)
        assert 0 < n < 1 << 30 and n % 256 == 0
        fn, args = calls(L, "delta", delta(L))[p]
        at = len(args) - 2
        assert fn(*args[:at], n - 1, None) == L.KAN_ERR_WORKSPACE
        assert fn(*args[:at - 1], None, n, None) == L.KAN_ERR_NULL
        assert fn(*args[:at - 1], args[at - 1] + 64, n, None) == L.KAN_ERR_ALIGN
    assert lib.kan_delta_workspace_size(delta(L), 2) == lib.kan_delta_workspace_size(delta(L), -1) == SIZE_MAX
    n = lib.kan_join_workspace_size(join(L))
    fn, args = calls(L, "join", join(L))[1]
    assert n > 0 and fn(*args[:-2], n - 1, None) == L.KAN_ERR_WORKSPACE
    assert lib.kan_join_workspace_size(join(L, N=0)) == 0


def test_join_arguments_that_contradict(L):
    fwd, bwd = calls(L, "join", join(L, flags=1))
    assert fwd[0](*fwd[1]) == L.KAN_ERR_UNSUPPORTED             # x and w_pre without the second norm
    assert bwd[0](*bwd[1]) == L.KAN_ERR_UNSUPPORTED
    fn, args = calls(L, "join", join(L))[1]
    for given, gone in ((11, 6), (12, 7), (13, 8)):             # a gradient of what is not there
        bad = list(args)
        bad[gone] = None
        assert fn(*bad) == L.KAN_ERR_UNSUPPORTED, given


def test_step_arguments(L):
    lib = L.lib()
    d = delta(L, T=1)
    ok = [d, 4, *A[:8], None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.kan_delta_step(*a)
    assert call(_0=delta(L)) == L.KAN_ERR_SHAPE                      # T is 6
    assert call(_0=None) == L.KAN_ERR_NULL
    assert call(_1=-1) == L.KAN_ERR_SHAPE and call(_1=1 << 60) == L.KAN_ERR_SHAPE
    assert call(_1=1, _8=None) == L.KAN_ERR_SHAPE                    # fewer states than sequences, no slots
    for i in (2, 3, 4, 5, 6, 7, 9):
        assert call(**{"_%d" % i: None}) == L.KAN_ERR_NULL
    for i, by in ((2, 2), (3, 2), (4, 2), (5, 8), (6, 8), (7, 8), (8, 8), (9, 8)):
        assert call(**{"_%d" % i: ok[i] + by}) == L.KAN_ERR_ALIGN
    for i in range(2, 9):
        assert call(**{"_9": ok[i]}) == L.KAN_ERR_ALIAS
        assert i == 7 or call(**{"_7": ok[i]}) == L.KAN_ERR_ALIAS
    assert lib.kan_delta_step(delta(L, B=0, T=1), 0, *[None] * 8, None) == L.KAN_OK


def test_empty_calls_launch_nothing(L):
    lib = L.lib()
    for d in (delta(L, B=0), delta(L, T=0)):
        assert lib.kan_delta_forward(d, *[None] * 10, 0, None) == L.KAN_OK
        assert lib.kan_delta_backward(d, *[None] * 16, 0, None) == L.KAN_OK
    assert lib.kan_join_forward(join(L, N=0), *[None] * 8, None) == L.KAN_OK
    assert lib.kan_join_backward(join(L, N=0), *[None] * 14, 0, None) == L.KAN_OK
