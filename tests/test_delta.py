"""GPU: the gated delta rule, its backward pass and its step of one row against the
float64 oracle.

Tolerances, with e = 2^-24, of the largest row error against the largest row
norm: a chunk's result is a chain of five products of a depth of at most 128
(the state's answer, the triangular solve, its correction, the rows' answer and
the state's update), each off by sqrt(128) e of its own norm; keys of a norm of
at most 1 and rates up to 1 let no error grow, and independent errors of the
chunks add like the root of their number: 5 sqrt(128) e sqrt(chunks).  The
backward pass chains the forward's values with two such chains of its own: three
times that.  Outputs in bfloat16 are rounded once more, 2^-8 of each value, and
what the kernels keep in two planes of bfloat16 for them adds 2^-16.

A gradient through x / |x| is n (d - u (u . d)), n = 1 / |x|, u = n x: the
difference of two terms of at most n |d| each, whose errors, of at least e n |d|,
stay when the terms cancel (with one key feature they cancel to 1e-6 of their size).
Gradients of q and k that are made unit vectors are therefore held against the
larger of their own rows and n |d|, with d the gradient of u.

A row of one sequence with one key and one value feature is a chain of scalars with
sums of two terms: v - S'k, S' + ku, dhT + q dy, dS - k du and dS u - S' dw.  A
rounding of a term stays when they cancel, and there is no other element whose
size the error could be held against, so it is held against the sizes of the
terms (with more features the rest of a row keeps its size: a key takes away one
direction of it).
"""

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import delta as O

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


@pytest.fixture(autouse=True)
def seeded(env):
    env[0].manual_seed(0)


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _dt(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _layout(torch, q, k, v, layout):
    """The same values as arrays of their own, slices of one array's rows (at aligned and at
    odd columns, with NaN between them), or heads before rows."""
    if layout == "apart":
        return q, k, v
    if layout == "heads":
        return tuple(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    B, T = q.shape[:2]
    pad = 0 if layout == "packed" else 3
    flat = [t.flatten(2) for t in (q, k, v)]
    p = torch.full((B, T, sum(t.shape[2] + pad for t in flat) + pad), float("nan"), dtype=q.dtype, device=q.device)
    out, at = [], pad
    for t, whole in zip(flat, (q, k, v)):
        p[..., at:at + t.shape[2]] = t
        out.append(p[..., at:at + t.shape[2]].unflatten(-1, whole.shape[2:]))
        at += t.shape[2] + pad
    return tuple(out)


def _draw(torch, B, T, Hk, Hv, Dk, Dv, dtype, layout, seed, unit=False, decay=0.3):
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, device="cuda:0", generator=gen)
    q, k, v = rand(B, T, Hk, Dk), rand(B, T, Hk, Dk), rand(B, T, Hv, Dv)
    if not unit:
        k = k / (k.norm(dim=-1, keepdim=True) * 1.01)
    g = -decay * torch.rand(B, T, Hv, device="cuda:0", generator=gen) ** 2
    beta = torch.rand(B, T, Hv, device="cuda:0", generator=gen)
    return (*_layout(torch, *(t.to(_dt(torch, dtype)) for t in (q, k, v)), layout), g, beta)


def _error(got, want, terms=None):
    """The largest row error over the largest row norm (of want, or of its terms if they are larger)."""
    got, want = (np.asarray(t, np.float64).reshape(-1, t.shape[-1]) if t.ndim > 3 else np.asarray(t, np.float64).reshape(-1, 1)
                 for t in (got, want))
    assert got.shape == want.shape and np.isfinite(got).all()
    size = max(np.sqrt((np.atleast_1d(t) ** 2).sum(-1)).max(initial=0) for t in ((want,) if terms is None else (want, terms)))
    error = np.sqrt(((got - want) ** 2).sum(-1)).max(initial=0)
    return error / size if size > 0 else error


def _tol(T, dtype=None, back=False):
    t = 5 * np.sqrt(128) * E * np.sqrt(max(1, -(-T // 64))) * (3 if back else 1)
    return t + (2.0 ** -8 + 2.0 ** -16 if dtype == "bf16" else 0)


def _scalars(q, k, v, h0, dy, dhT, unit):
    """Sizes of the terms behind y, hT and the gradients where every array has one element (|k|, beta, exp(g) <= 1)."""
    q, k, v, h0, dy, dhT = (0.0 if t is None else float(np.abs(t).max(initial=0)) for t in (q, k, v, h0, dy, dhT))
    nq, nk = (1 / np.sqrt(x * x + O.UNIT_EPS) if unit else 1.0 for x in (q, k))
    w, d = v + h0, dhT + q * nq * dy
    return dict(y=q * nq * (h0 + w), hT=h0 + w, dq=nq * dy * (h0 + w), dk=nk * d * (w + h0), dv=d, dg=2 * d * h0, dbeta=d * w,
                dh0=2 * d)


def _lengths(torch, B, T):
    n = [T, T // 2, 0, T + 9, -2, 1, max(T - 1, 0)]
    return torch.tensor([n[(i + (B == 1)) % 7] for i in range(B)], dtype=torch.int32, device="cuda:0")


# (B, T, Hk, Hv, Dk, Dv): one row to long ones, a chunk's edges, one column to all, shared heads, groups of
# columns that are and are not whole, enough heads for two blocks of columns a head, few for cut sequences
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 1, 1, 2, 5, 3), (1, 2, 2, 2, 16, 16), (3, 7, 1, 3, 33, 31), (2, 63, 2, 2, 32, 64),
          (2, 64, 1, 4, 64, 16), (1, 65, 2, 4, 128, 128), (2, 82, 2, 2, 104, 72), (3, 127, 3, 3, 8, 200),
          (2, 128, 1, 1, 128, 33), (2, 129, 1, 2, 65, 65), (5, 190, 2, 6, 48, 80), (1, 300, 1, 1, 24, 1024),
          (2, 257, 4, 4, 128, 64), (130, 66, 1, 2, 16, 40), (3, 700, 1, 2, 127, 17), (1, 2049, 1, 1, 40, 24),
          (1, 1600, 1, 2, 128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["apart", "packed", "odd", "heads"])
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SHAPES)
def test_forward(env, B, T, Hk, Hv, Dk, Dv, layout, dtype):
    torch, F = env
    unit = layout in ("packed", "odd")
    args = _draw(torch, B, T, Hk, Hv, Dk, Dv, dtype, layout, B + 3 * T + Dk, unit)
    h0 = torch.randn(B, Hv, Dk, Dv, device="cuda:0") if layout != "apart" else None
    lengths = _lengths(torch, B, T) if layout in ("odd", "heads") else None
    scale = 0.5 if layout == "heads" else None
    y = torch.full((B, T, Hv, Dv), float("nan"), dtype=args[0].dtype, device="cuda:0")
    _, hT = F.kan_delta_forward(*args, h0, lengths, scale, unit, out=y)
    wy, wh = O.delta_forward(*map(_np, args), _np(h0), None if lengths is None else lengths.tolist(), scale, unit)
    terms = _scalars(*map(_np, (*args[:3], h0, None, None)), unit) if B * T * Dk * Dv == 1 else {}
    assert _error(_np(y), wy, terms.get("y")) <= _tol(T, dtype) and _error(_np(hT), wh, terms.get("hT")) <= _tol(T)
    if lengths is not None:
        for b, n in enumerate(lengths.tolist()):
            assert not y[b, max(n, 0):].any()
            assert n > 0 or torch.equal(hT[b], h0[b])
    again = F.kan_delta_forward(*args, h0, lengths, scale, unit)
    assert torch.equal(y, again[0]) and torch.equal(hT, again[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["apart", "packed", "odd", "heads"])
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SHAPES)
def test_backward(env, B, T, Hk, Hv, Dk, Dv, layout, dtype):
    torch, F = env
    unit = layout in ("packed", "odd")
    args = _draw(torch, B, T, Hk, Hv, Dk, Dv, dtype, layout, B + 5 * T + Dk, unit)
    state = (B, Hv, Dk, Dv)
    h0 = torch.randn(state, device="cuda:0") if layout != "apart" else None
    dhT = torch.randn(state, device="cuda:0") if layout != "packed" else None
    lengths = _lengths(torch, B, T) if layout in ("odd", "heads") else None
    dy = torch.randn(B, T, Hv, Dv, device="cuda:0").to(args[0].dtype)
    grads = _layout(torch, *(torch.full_like(t, float("nan")).contiguous() for t in args[:3]), layout)
    got = F.kan_delta_backward(*args, dy, h0, lengths, dhT, None, unit, True, *grads)
    assert all(a is b for a, b in zip(got, grads))
    want = O.delta_backward(*map(_np, args), _np(dy), _np(h0), None if lengths is None else lengths.tolist(), _np(dhT),
                            None, unit)
    terms = _scalars(*map(_np, (*args[:3], h0, dy, dhT)), unit) if B * T * Dk * Dv == 1 else {}
    if unit and not terms:               # n d of q and k
        u, n = zip(*(O._unit(_np(t), True) for t in args[:2]))
        plain = O.delta_backward(*u, *map(_np, args[2:]), _np(dy), _np(h0),
                                 None if lengths is None else lengths.tolist(), _np(dhT))
        terms = {"dq": n[0] * plain[0], "dk": n[1] * plain[1]}
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want):
        assert _error(_np(a), b, terms.get(name)) <= _tol(T, dtype if name in ("dq", "dk", "dv") else None, True), name
    if lengths is not None:
        for b, n in enumerate(lengths.tolist()):
            assert not any(t[b, max(n, 0):].any() for t in got[:5])
    again = F.kan_delta_backward(*args, dy, h0, lengths, dhT, None, unit, True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [96, 1300])
def test_gradients_by_differences(env, T, dtype):
    """<gradient, direction> against the oracle's loss along the direction, for each input."""
    torch, F = env
    args = list(_draw(torch, 2, T, 1, 2, 24, 40, dtype, "apart", T))
    h0, dhT = (torch.randn(2, 2, 24, 40, device="cuda:0") for _ in range(2))
    dy = torch.randn(2, T, 2, 40, device="cuda:0").to(args[0].dtype)
    got = [_np(t) for t in F.kan_delta_backward(*args, dy, h0, None, dhT)]
    x = [_np(t) for t in (*args, h0)]
    r = np.random.default_rng(T)

    def loss(x):
        y, hT = O.delta_forward(*x)
        return (y * _np(dy)).sum() + (hT * _np(dhT)).sum()
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        way = r.standard_normal(x[i].shape) * (0.1 if i in (3, 4) else 1.0)
        s = 1e-5                         # central differences: s^2 of the third derivative, 2^-53 / s of the loss
        moved = [loss([t + a * way if j == i else t for j, t in enumerate(x)]) for a in (s, -s)]
        want = (moved[0] - moved[1]) / (2 * s)
        size = np.linalg.norm(got[i]) * np.linalg.norm(way)
        assert abs((got[i] * way).sum() - want) <= (_tol(T, dtype if i < 3 else None, True) + 1e-6) * size, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 1), (3, 1, 3, 33, 31), (4, 2, 4, 128, 128), (2, 1, 2, 104, 72),
                                           (5, 3, 3, 64, 1000), (2, 2, 2, 7, 129)])
@pytest.mark.parametrize("unit", [False, True])
def test_steps_equal_the_oracle(env, B, Hk, Hv, Dk, Dv, dtype, unit):
    """Rows one at a time, with the states in a pool whose other entries stay as they are."""
    torch, F = env
    T, S = 9, B + 3
    args = _draw(torch, B, T, Hk, Hv, Dk, Dv, dtype, "odd" if unit else "apart", Dk + Dv, unit)
    pool = torch.randn(S, Hv, Dk, Dv, device="cuda:0")
    slots = torch.randperm(S)[:B].to(torch.int32).cuda()
    before, h0 = pool.clone(), pool[slots.long()].clone()
    y = torch.stack([F.kan_delta_step(*(t[:, i] for t in args[:3]), args[3][:, i].contiguous(), args[4][:, i].contiguous(),
                                      pool, slots, unit=unit) for i in range(T)], 1)
    wy, wh = O.delta_forward(*map(_np, args), _np(h0), unit=unit)
    assert _error(_np(y), wy) <= _tol(T, dtype) and _error(_np(pool[slots.long()]), wh) <= _tol(T)
    rest = [i for i in range(S) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_step_without_slots_and_with_slots_outside(env):
    torch, F = env
    q, k, v, g, beta = (t[:, 0].contiguous() for t in _draw(torch, 4, 1, 1, 2, 16, 24, "f32", "apart", 1))
    pool = torch.randn(6, 2, 16, 24, device="cuda:0")
    a, b = pool.clone(), pool.clone()
    ya = F.kan_delta_step(q, k, v, g, beta, a)
    yb = F.kan_delta_step(q, k, v, g, beta, b, torch.tensor([0, -1, 6, 3], dtype=torch.int32, device="cuda:0"))
    assert torch.equal(a[4:], pool[4:]) and torch.equal(b[[1, 2, 4, 5]], pool[[1, 2, 4, 5]])
    assert torch.equal(a[[0, 3]], b[[0, 3]]) and torch.equal(ya[[0, 3]], yb[[0, 3]]) and not yb[1:3].any()


def test_forward_in_parts_and_steps(env):
    """A sequence cut anywhere, its state handed on, and its end step by step."""
    torch, F = env
    args = _draw(torch, 2, 411, 2, 4, 64, 48, "f32", "packed", 5, unit=True)
    y, hT = F.kan_delta_forward(*args, unit=True)
    h, rows = None, []
    for lo, hi in ((0, 1), (1, 64), (64, 230), (230, 402)):
        part, h = F.kan_delta_forward(*(t[:, lo:hi] if t.dim() == 4 else t[:, lo:hi].contiguous() for t in args), h,
                                      unit=True)
        rows.append(part)
    for i in range(402, 411):
        rows.append(F.kan_delta_step(*(t[:, i] for t in args[:3]), args[3][:, i].contiguous(),
                                     args[4][:, i].contiguous(), h, unit=True)[:, None])
    assert _error(_np(torch.cat(rows, 1)), _np(y)) <= 2 * _tol(411) and _error(_np(h), _np(hT)) <= 2 * _tol(411)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1e-4, 4.0, 60.0, float("inf")])
def test_decays(env, decay, dtype):
    """From a state that never fades to one that a row wipes out; products of decays underflow inside a chunk."""
    torch, F = env
    args = _draw(torch, 2, 150, 1, 2, 32, 48, dtype, "apart", 3)
    gen = torch.Generator(device="cuda:0").manual_seed(4)
    pick = torch.rand(args[3].shape, device="cuda:0", generator=gen)
    g = torch.where(pick < 0.2, torch.full_like(pick, -decay), -decay * 1e-2 * pick if decay < 1e9 else -pick)
    beta = torch.where(pick > 0.9, torch.zeros_like(pick), args[4])
    h0, dhT = (torch.randn(2, 2, 32, 48, device="cuda:0") for _ in range(2))
    dy = torch.randn(2, 150, 2, 48, device="cuda:0").to(args[0].dtype)
    a = (*args[:3], g, beta)
    y, hT = F.kan_delta_forward(*a, h0)
    wy, wh = O.delta_forward(*map(_np, a), _np(h0))
    assert _error(_np(y), wy) <= _tol(150, dtype) and _error(_np(hT), wh) <= _tol(150)
    got = F.kan_delta_backward(*a, dy, h0, None, dhT)
    want = O.delta_backward(*map(_np, a), _np(dy), _np(h0), None, _np(dhT))
    for i, (x, w) in enumerate(zip(got, want)):
        assert _error(_np(x), w) <= _tol(150, dtype if i < 3 else None, True), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_past_a_length_may_hold_anything(env, dtype):
    torch, F = env
    args = _draw(torch, 4, 200, 1, 2, 64, 72, dtype, "apart", 6)
    lengths = torch.tensor([100, 64, 0, 1], dtype=torch.int32, device="cuda:0")
    dy = torch.randn(4, 200, 2, 72, device="cuda:0").to(args[0].dtype)
    clean = F.kan_delta_forward(*args, None, lengths), F.kan_delta_backward(*args, dy, None, lengths)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t in (*args, dy):
            for b, n in enumerate(lengths.tolist()):
                t[b, n:] = bad
        again = F.kan_delta_forward(*args, None, lengths), F.kan_delta_backward(*args, dy, None, lengths)
        for one, two in zip(clean, again):
            assert all(torch.equal(a, b) for a, b in zip(one, two) if a is not None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", [0, 1, 2, 3, 4])
def test_a_nan_stays_in_its_sequence(env, which, dtype):
    """It shows in its row's answer and its last state, and in no other sequence and no earlier chunk."""
    torch, F = env
    args = _draw(torch, 3, 200, 1, 1, 32, 48, dtype, "apart", 7)
    y0, h0 = F.kan_delta_forward(*args)
    args[which][1, 130] = float("nan")
    y, h = F.kan_delta_forward(*args)
    assert torch.equal(y[[0, 2]], y0[[0, 2]]) and torch.equal(h[[0, 2]], h0[[0, 2]])
    assert torch.equal(y[1, :128], y0[1, :128]) and y[1, 130].isnan().all()
    assert which == 0 or h[1].isnan().all()


def test_empty(env):
    torch, F = env
    for B, T in ((0, 5), (2, 0), (0, 0)):
        args = _draw(torch, B, T, 1, 2, 16, 24, "f32", "apart", 1)
        h0, dhT = (torch.randn(B, 2, 16, 24, device="cuda:0") for _ in range(2))
        y, hT = F.kan_delta_forward(*args, h0)
        assert y.shape == (B, T, 2, 24) and torch.equal(hT, h0)
        assert not F.kan_delta_forward(*args)[1].any()
        got = F.kan_delta_backward(*args, torch.empty_like(y), h0, None, dhT)
        assert torch.equal(got[5], dhT)
    q, k, v, g, beta = (t[:, 0] for t in _draw(torch, 0, 1, 1, 2, 16, 24, "f32", "apart", 1))
    pool = torch.ones(3, 2, 16, 24, device="cuda:0")
    assert F.kan_delta_step(q, k, v, g, beta, pool).shape == (0, 2, 24) and (pool == 1).all()


@pytest.mark.parametrize("seq,row", [(2 ** 31 + 40, 96), (130 * 2 ** 24, 2 ** 24)])
def test_strides_past_32_bits(env, seq, row):
    """Sequences, and rows of one sequence, further apart than 2^31 elements."""
    torch, F = env
    B, T, D = 2, 130, 32
    base = torch.empty((B - 1) * seq + (T - 1) * row + 3 * D, dtype=torch.bfloat16, device="cuda:0")
    grad = torch.empty_like(base)

    def views(t):
        return [t.as_strided((B, T, 1, D), (seq, row, D, 1), i * D) for i in range(3)]
    args = _draw(torch, B, T, 1, 1, D, D, "bf16", "apart", 8)
    far = views(base)
    for a, b in zip(far, args):
        a.copy_(b)
    dy = torch.randn(B, T, 1, D, device="cuda:0").to(torch.bfloat16)
    near = F.kan_delta_forward(*args), F.kan_delta_backward(*args, dy)
    got = F.kan_delta_forward(*far, *args[3:])
    assert all(torch.equal(a, b) for a, b in zip(near[0], got))
    dq, dk, dv = views(grad)
    F.kan_delta_backward(*far, *args[3:], dy, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip(near[1][:3], (dq, dk, dv)))


def test_a_pool_past_32_bits(env):
    torch, F = env
    pool = torch.empty(2 ** 17 + 50, 1, 128, 128, device="cuda:0")       # 2^31 elements and more
    slots = torch.tensor([2 ** 17 + 49, 0, 2 ** 17], dtype=torch.int32, device="cuda:0")
    h0 = torch.randn(3, 1, 128, 128, device="cuda:0")
    pool[slots.long()] = h0
    args = [t[:, 0].contiguous() for t in _draw(torch, 3, 1, 1, 1, 128, 128, "f32", "apart", 9)]
    y = F.kan_delta_step(*args, pool, slots)
    assert torch.equal(y, F.kan_delta_step(*args, h0)) and torch.equal(pool[slots.long()], h0)


def test_refusals(env):
    torch, F = env
    q, k, v, g, beta = _draw(torch, 2, 6, 2, 4, 16, 24, "f32", "apart", 1)
    dy = torch.zeros_like(v)
    for call in (lambda: F.kan_delta_forward(q[0], k, v, g, beta),
                 lambda: F.kan_delta_forward(q, k[:, :5], v, g, beta),
                 lambda: F.kan_delta_forward(q, k, v[:, :5].contiguous(), g[:, :5].contiguous(), beta[:, :5].contiguous()),
                 lambda: F.kan_delta_forward(q, k.to(torch.bfloat16), v, g, beta),
                 lambda: F.kan_delta_forward(q.half(), k.half(), v.half(), g, beta),
                 lambda: F.kan_delta_forward(q, k, v[:, :, :3], g[..., :3].contiguous(), beta[..., :3].contiguous()),
                 lambda: F.kan_delta_forward(q, k, v, g.double(), beta),
                 lambda: F.kan_delta_forward(q, k, v, g, beta.cpu()),
                 lambda: F.kan_delta_forward(q, k, v, g.transpose(1, 2), beta),
                 lambda: F.kan_delta_forward(q.transpose(2, 3), k.transpose(2, 3), v, g, beta),
                 lambda: F.kan_delta_forward(q, k, v, g, beta, torch.zeros(2, 4, 24, 16, device="cuda:0")),
                 lambda: F.kan_delta_forward(q, k, v, g, beta, None, torch.zeros(2, dtype=torch.int64, device="cuda:0")),
                 lambda: F.kan_delta_forward(q, k, v, g, beta, scale=float("nan")),
                 lambda: F.kan_delta_forward(torch.zeros(1, 2, 1, 129, device="cuda:0"),
                                             torch.zeros(1, 2, 1, 129, device="cuda:0"),
                                             torch.zeros(1, 2, 1, 4, device="cuda:0"),
                                             torch.zeros(1, 2, 1, device="cuda:0"), torch.zeros(1, 2, 1, device="cuda:0")),
                 lambda: F.kan_delta_backward(q, k, v, g, beta, dy.to(torch.bfloat16)),
                 lambda: F.kan_delta_backward(q, k, v, g, beta, dy, dq=torch.empty_like(q)),
                 lambda: F.kan_delta_backward(q, k, v, g, beta, dy, dq=q, dk=torch.empty_like(k), dv=torch.empty_like(v)),
                 lambda: F.kan_delta_backward(q, k, v, g, beta, dy, dq=dy[..., :16], dk=dy[..., 8:], dv=dy.clone()),
                 lambda: F.kan_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), beta[:, 0].contiguous(),
                                          torch.zeros(1, 4, 16, 24, device="cuda:0")),
                 lambda: F.kan_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), beta[:, 0].contiguous(),
                                          torch.zeros(2, 4, 24, 16, device="cuda:0"))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
