"""GPU: the join between two blocks and its backward pass against the float64 oracle.

Tolerances, with e = 2^-24, of each element: a mean is a sum over at most 26
levels (four vectors of four of a thread, ten levels across threads) and its factor a
root and a reciprocal, 16 e; the activation's exp has an argument |g| <= 16 that
rounds to 16 e, the rest of it 8 e; the products and the sum of a value 8 e:
48 e of the values' sizes, of the terms of a sum and not of the sum.  A second
norm over those adds as much: twice.  Sums over N rows add N e of their terms'
sizes.  Outputs in bfloat16 are rounded once more, 2^-8 of the value.
"""

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import delta as O

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
STEP = 48 * E


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _dt(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(torch, N, D, dtype, gap, size=1.0):
    """Rows with a stride of their own; what lies between them is NaN."""
    t = torch.full((N, D + gap), float("nan"), dtype=dtype, device="cuda:0")[:, :D] if gap else \
        torch.empty(N, D, dtype=dtype, device="cuda:0")
    t.copy_(torch.randn(N, D, device="cuda:0").clamp(-16, 16) * size)
    return t


def _half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 0.0


SHAPES = [(1, 1), (3, 2), (2, 3), (1, 4), (7, 31), (9, 64), (5, 127), (64, 128), (33, 129), (8, 255), (6, 256),
          (5, 257), (300, 770), (3, 1024), (4, 1025), (2, 2048), (5, 2049), (3, 4096), (2, 4097), (2, 8191), (3, 8192)]
# (post, pre, residual, gate, weights, activation, scale)
FORMS = [(True, True, True, True, True, "silu", 1.0), (True, True, True, True, False, "sigmoid", 0.3),
         (True, False, False, True, True, "silu", 1.0), (False, True, True, False, True, "silu", -2.0),
         (True, False, True, False, True, "silu", 1.0), (False, True, False, False, True, "silu", 1.0),
         (False, False, True, True, False, "sigmoid", 1.0)]
TYPES = [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("f32", "bf16", "bf16"),
         ("bf16", "f32", "f32"), ("f32", "f32", "bf16")]


def _inputs(torch, N, D, types, form, seed):
    torch.manual_seed(seed)
    post, pre, res, gate, weights, activation, scale = form
    h = _rows(torch, N, D, _dt(torch, types[0]), seed % 3 and 5 * (seed % 3) - 1)
    r = _rows(torch, N, D, _dt(torch, types[1]), 8) if res else None
    g = _rows(torch, N, D, _dt(torch, types[0]), 3, 3.0) if gate else None
    w_post = 1 + 0.3 * torch.randn(D, device="cuda:0") if weights else None
    w_pre = 1 + 0.3 * torch.randn(D, device="cuda:0") if weights and pre else None
    return h, r, g, w_post, w_pre


@pytest.mark.parametrize("N,D", SHAPES)
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forward(env, N, D, form):
    torch, F = env
    for types in (TYPES if D < 1000 else TYPES[form % 3::3]):
        post, pre, _, _, _, activation, scale = FORMS[form]
        h, r, g, w_post, w_pre = _inputs(torch, N, D, types, FORMS[form], N + D + form)
        y, x, stats = F.kan_join_forward(h, r, g, w_post, w_pre, post, pre, activation, scale, 1e-5,
                                         _dt(torch, types[1]), _dt(torch, types[2]))
        wy, wx, n1, n2 = O.join_forward(_np(h), _np(r), _np(g), _np(w_post), _np(w_pre), post, pre, activation, scale,
                                        1e-5)
        size = np.abs(wy - (0 if r is None else _np(r))) + (0 if r is None else np.abs(_np(r)))
        assert y.dtype == _dt(torch, types[1])
        assert (np.abs(_np(y) - wy) <= STEP * size + _half(types[1]) * np.abs(wy) + 1e-37).all()
        assert (np.abs(_np(stats[0]) - n1) <= STEP * n1).all()
        if pre:
            grown = np.sqrt((size ** 2).mean(-1, keepdims=True)) * n2[:, None]         # of n2's relative error
            w = 1 if w_pre is None else np.abs(_np(w_pre))
            tol = 2 * STEP * (w * n2[:, None] * size + np.abs(wx) * (1 + grown))
            assert x.dtype == _dt(torch, types[2])
            assert (np.abs(_np(x) - wx) <= tol + _half(types[2]) * np.abs(wx)).all()
            assert (np.abs(_np(stats[1]) - n2) <= STEP * n2 * (1 + grown[:, 0])).all()
        else:
            assert x is None and (stats[1] == 1).all()
        again = F.kan_join_forward(h, r, g, w_post, w_pre, post, pre, activation, scale, 1e-5, _dt(torch, types[1]),
                                   _dt(torch, types[2]))
        assert torch.equal(y, again[0]) and torch.equal(stats, again[2])


def _sizes(h, y, n1, n2, dy, dx, gate, w_post, w_pre, post, activation, scale):
    """Sums of the terms' sizes behind each gradient: dh, dr, dgate, dw_post, dw_pre."""
    n1, n2 = n1[:, None], n2[:, None]
    d, dw_pre = np.abs(dy) if dy is not None else np.zeros_like(h), None
    if dx is not None:
        z, c = np.abs(y * n2), np.abs(dx)
        dw_pre = (c * z).sum(0)
        c = c * (1 if w_pre is None else np.abs(w_pre))
        d = d + n2 * (c + z * (c * z).mean(-1, keepdims=True))
    t, w = np.abs(h * n1), 1 if w_post is None else np.abs(w_post)
    e, dgate = abs(scale) * d, None
    if gate is not None:
        a, _ = O._act(activation, gate)
        s, _ = O._act("sigmoid", gate)
        # the slope's terms, s + g s (1 - s) or s (1 - s)
        slope = s + np.abs(gate) * s * (1 - s) if activation == "silu" else s * (1 - s)
        dgate, e = e * w * t * slope, e * np.abs(a)
    dw_post = (e * t).sum(0)
    e = e * w
    return (n1 * (e + t * (e * t).mean(-1, keepdims=True)) if post else e), d, dgate, dw_post, dw_pre


@pytest.mark.parametrize("N,D", SHAPES + [(2100, 40), (1030, 300)])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_backward(env, N, D, form):
    torch, F = env
    for types in (TYPES if D < 1000 else TYPES[form % 3::3]):
        post, pre, res, _, _, activation, scale = FORMS[form]
        h, r, g, w_post, w_pre = _inputs(torch, N, D, types, FORMS[form], N + 2 * D + form)
        y, x, stats = F.kan_join_forward(h, r, g, w_post, w_pre, post, pre, activation, scale, 1e-5,
                                         _dt(torch, types[1]), _dt(torch, types[2]))
        dy = torch.randn(N, D, device="cuda:0").to(y.dtype) if not pre or form % 2 == 0 else None
        dx = torch.randn(N, D, device="cuda:0").to(x.dtype) if pre else None
        got = F.kan_join_backward(h, y, stats, dy, dx, g, w_post, w_pre, post, activation, scale, need_dr=res)
        a = [_np(t) for t in (h, y, stats[0], stats[1], dy, dx, g, w_post, w_pre)]
        want = O.join_backward(*a, post, activation, scale)
        sizes = _sizes(*a, post, activation, scale)
        for i, name in enumerate(("dh", "dr", "dgate", "dw_post", "dw_pre")):
            absent = (not res, g is None, w_post is None, w_pre is None)
            if i and absent[i - 1]:
                assert got[i] is None, name
                continue
            tol = 2 * STEP * sizes[i] + (N * E * sizes[i] if i > 2 else 0)
            tol = tol + _half(types[1] if i == 1 else types[0] if i < 3 else "f32") * np.abs(want[i])
            assert (np.abs(_np(got[i]) - want[i]) <= tol + 1e-37).all(), (name, types)
        again = F.kan_join_backward(h, y, stats, dy, dx, g, w_post, w_pre, post, activation, scale, need_dr=res)
        assert all(torch.equal(p, q) for p, q in zip(got, again) if p is not None)


def test_gradients_by_differences(env):
    torch, F = env
    form = FORMS[0]
    h, r, g, w_post, w_pre = _inputs(torch, 40, 150, TYPES[0], form, 3)
    y, x, stats = F.kan_join_forward(h, r, g, w_post, w_pre, eps=1e-5)
    dy, dx = torch.randn_like(y), torch.randn_like(x)
    got = [_np(t) for t in F.kan_join_backward(h, y, stats, dy, dx, g, w_post, w_pre)]
    a = [_np(t) for t in (h, r, g, w_post, w_pre)]
    way_of = np.random.default_rng(0)

    def loss(a):
        y, x, _, _ = O.join_forward(*a, eps=1e-5)
        return (y * _np(dy)).sum() + (x * _np(dx)).sum()
    for i, name in enumerate(("h", "r", "gate", "w_post", "w_pre")):
        way, s = way_of.standard_normal(a[i].shape), 1e-5
        moved = [loss([t + b * way if j == i else t for j, t in enumerate(a)]) for b in (s, -s)]
        size = np.linalg.norm(got[i]) * np.linalg.norm(way)
        assert abs((got[i] * way).sum() - (moved[0] - moved[1]) / (2 * s)) <= (4 * STEP + 40 * E + 1e-7) * size, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_gates_far_out(env, activation, dtype):
    """Gates whose exp overflows or vanishes, up to infinite ones where the activation has a limit."""
    torch, F = env
    t = _dt(torch, dtype)
    gate = torch.tensor([-1e30, -1000.0, -90.0, -40.0, 0.0, 40.0, 90.0, 1000.0, 1e30], device="cuda:0").to(t)[None]
    gate = torch.cat([gate, -gate])
    h = torch.randn(2, 9, device="cuda:0").to(t)
    y, _, stats = F.kan_join_forward(h, None, gate, None, None, True, False, activation)
    wy = O.join_forward(_np(h), None, _np(gate), pre=False, activation=activation)[0]
    # of a vanishing factor only its size matters: below 1e-37 it may be 0, and its exp's argument |g| rounds to |g| e
    tol = (48 + 110) * E * np.abs(wy) + _half(dtype) * np.abs(wy) + 1e-35
    assert (np.abs(_np(y) - wy) <= tol).all()
    dy = torch.randn(2, 9, device="cuda:0").to(t)
    dh, _, dgate, _, _ = F.kan_join_backward(h, y, stats, dy, None, gate, activation=activation)
    assert dgate.isfinite().all() and (dgate[:, [0, -1]].float().abs() <= dgate.new_tensor(1e3).float()).all()
    if activation == "sigmoid":
        inf = torch.tensor([[float("inf"), -float("inf")]], device="cuda:0").to(t)
        y, _, _ = F.kan_join_forward(torch.ones_like(inf), None, inf, None, None, False, False, "sigmoid")
        assert y.tolist() == [[1.0, 0.0]]


def test_sizes_at_the_ends(env):
    """Rows of zeros, of tiny and of huge values, and a NaN that stays in its row."""
    torch, F = env
    h = torch.randn(5, 300, device="cuda:0")
    h[0] = 0
    h[1] *= 1e-15
    h[2] *= 1e15
    y, x, stats = F.kan_join_forward(h, eps=1e-6)
    wy, wx, n1, n2 = O.join_forward(_np(h), eps=1e-6)
    assert (np.abs(_np(y) - wy) <= STEP * np.abs(wy)).all() and (np.abs(_np(x) - wx) <= 4 * STEP * np.abs(wx)).all()
    assert not y[0].any() and not x[0].any()
    h[3, 17] = float("nan")
    bad = F.kan_join_forward(h, eps=1e-6)
    assert bad[0][3].isnan().all() and torch.equal(bad[0][[0, 1, 2, 4]], y[[0, 1, 2, 4]])


def test_empty(env):
    torch, F = env
    h, w = torch.empty(0, 12, device="cuda:0"), torch.ones(12, device="cuda:0")
    y, x, stats = F.kan_join_forward(h, h, h, w, w)
    assert y.shape == x.shape == (0, 12) and stats.shape == (2, 0)
    dh, dr, dgate, dw_post, dw_pre = F.kan_join_backward(h, y, stats, y, x, h, w, w)
    assert dh.shape == dr.shape == dgate.shape == (0, 12) and not dw_post.any() and not dw_pre.any()


def test_rows_past_32_bits(env):
    """Elements past 2^31 of contiguous outputs, and rows further apart than 2^31."""
    torch, F = env
    N, D = (1 << 24) + 9, 128
    h = torch.randn(1 << 12, D, device="cuda:0").to(torch.bfloat16)
    big = h.repeat(N // len(h) + 1, 1)[:N]
    w = 1 + 0.1 * torch.randn(D, device="cuda:0")
    y, x, _ = F.kan_join_forward(big, None, None, w, w)
    wy, wx, _ = F.kan_join_forward(h, None, None, w, w)
    for lo in range(0, N, 1 << 22):
        at = torch.arange(lo, min(N, lo + (1 << 22)), device="cuda:0") % len(h)
        assert torch.equal(y[lo:lo + (1 << 22)], wy[at]) and torch.equal(x[lo:lo + (1 << 22)], wx[at])
    base = torch.empty((1 << 31) + 4 * D, dtype=torch.bfloat16, device="cuda:0")
    far = base.as_strided((2, D), ((1 << 31) + D, 1), D)
    far.copy_(h[:2])
    assert torch.equal(F.kan_join_forward(far, far, far, w, w)[0], F.kan_join_forward(h[:2], h[:2], h[:2], w, w)[0])


@pytest.mark.parametrize("N,D,dtype", [(131072 + 5, 100, "bf16"), (65536 + 1, 256, "f32"), (140001, 31, "f32")])
def test_many_narrow_rows_equal_few(env, N, D, dtype):
    """Threads that have several rows at a time: the same bits as a call of few of the rows."""
    torch, F = env
    dt = _dt(torch, dtype)
    h, r, gate = (_rows(torch, N, D, dt, gap) for gap in (0, 3, 8))
    w, u = torch.rand(D, device="cuda:0"), torch.rand(D, device="cuda:0")
    whole = F.kan_join_forward(h, r, gate, w, u)
    for lo, hi in ((0, 700), (N // 2, N // 2 + 333), (N - 41, N)):
        part = F.kan_join_forward(h[lo:hi], r[lo:hi], gate[lo:hi], w, u)
        assert torch.equal(whole[0][lo:hi], part[0]) and torch.equal(whole[1][lo:hi], part[1])
        assert torch.equal(whole[2][:, lo:hi], part[2])
    assert bool(whole[0].isfinite().all()) and bool(whole[1].isfinite().all())


def test_refusals(env):
    torch, F = env
    h, w = torch.randn(4, 16, device="cuda:0"), torch.ones(16, device="cuda:0")
    y, x, stats = F.kan_join_forward(h)
    for call in (lambda: F.kan_join_forward(h[0]), lambda: F.kan_join_forward(h.half()),
                 lambda: F.kan_join_forward(h.t()), lambda: F.kan_join_forward(h, h[:3]),
                 lambda: F.kan_join_forward(h, None, h.to(torch.bfloat16)),
                 lambda: F.kan_join_forward(h, None, None, w[:15]), lambda: F.kan_join_forward(h, None, None, w.double()),
                 lambda: F.kan_join_forward(h, None, None, None, w, pre=False),
                 lambda: F.kan_join_forward(h, activation="relu"), lambda: F.kan_join_forward(h, eps=-1.0),
                 lambda: F.kan_join_forward(h, scale=float("inf")), lambda: F.kan_join_forward(h, row_dtype=torch.half),
                 lambda: F.kan_join_forward(h, h, res_dtype=torch.bfloat16),
                 lambda: F.kan_join_forward(torch.empty(1, 8193, device="cuda:0")),
                 lambda: F.kan_join_backward(h, y, stats[0], y), lambda: F.kan_join_backward(h, y[:3], stats, y),
                 lambda: F.kan_join_backward(h, y, stats, y, None, None, None, w),
                 lambda: F.kan_join_backward(h, y, stats, y.to(torch.bfloat16))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
