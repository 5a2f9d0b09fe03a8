"""GPU: the gated recurrence, its backward pass and its single-row step against
the float64 oracle.

Tolerances, with e = 2^-24: a gate is exp, a sum and a reciprocal; the exp's
argument |g| <= 16 rounds to 16 e, the rest to about 8 e more, so u and f are
within 24 e relative.  An error du of a gate moves h by its share of
|x - h|, and the shares of all steps add to at most 1: 24 e (max |x| + max |h|).
Each step rounds h once; over a memory of M = min(T, 1 / min u) steps such
roundings add at most like 8 sqrt(M) e max |h|.  A gradient multiplies two or
three such factors: three times the bound, at the gradient's own scale.
bf16 gradients round once more, 2^-8 relative.
"""

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import token as O

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


def _dt(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy()


def _draw(torch, B, T, D, dtype, layout, seed, gate=(2.0, 1.5)):
    """x and g as separate arrays, halves of one array, or sequences inside rows."""
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(seed)
    dt = _dt(torch, dtype)
    p = torch.randn(B, T, 2 * D, device="cuda:0", generator=gen)
    p[..., D:] = (p[..., D:] * gate[1] + gate[0]).clamp(-16, 16)
    p = p.to(dt)
    if layout == "packed":
        return p[..., :D], p[..., D:]
    if layout == "rows":                  # [T, B, D] in memory
        q = p.transpose(0, 1).contiguous()
        return q[..., :D].contiguous().transpose(0, 1), q[..., D:].contiguous().transpose(0, 1)
    return p[..., :D].contiguous(), p[..., D:].contiguous()


def _bound(g, x, h, T):
    u = O.sigmoid(-g.astype(np.float64))
    mem = min(T, 1.0 / u.min()) if u.size else 1
    return EPS * (24 * (np.abs(x).max(initial=0) + np.abs(h).max(initial=0)) +
                  8 * np.sqrt(mem) * np.abs(h).max(initial=0))


SHAPES = [(1, 1, 1), (2, 1, 5), (1, 2, 64), (3, 7, 3), (2, 63, 8), (2, 64, 4), (1, 65, 100), (2, 255, 33),
          (1, 256, 16), (1, 257, 64), (3, 300, 770), (2, 513, 36), (1, 1025, 70), (4, 2049, 12), (1, 9000, 24)]


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["apart", "packed", "rows"])
def test_forward(env, B, T, D, dtype, layout):
    torch, F = env
    x, g = _draw(torch, B, T, D, dtype, layout, B + T + D)
    h0 = torch.randn(B, D, device="cuda:0") if T % 2 else None
    lengths = None
    if layout != "apart":
        lengths = torch.tensor([T, 0, T // 2, -3][:B] if B > 1 else [max(T - 1, 0)], dtype=torch.int32, device="cuda:0")
    y = torch.full((B, T, D), float("nan"), device="cuda:0")
    y, hT = F.kan_recur_forward(x, g, h0, lengths, out=y)
    wy, wh = O.recur_forward(_np(x), _np(g), _np(h0), None if lengths is None else lengths.tolist())
    tol = _bound(_np(g), _np(x), np.concatenate([wy.reshape(-1, D), wh]), T)
    assert np.abs(y.double().cpu().numpy() - wy).max() <= tol
    assert np.abs(hT.double().cpu().numpy() - wh).max() <= tol
    again = F.kan_recur_forward(x, g, h0, lengths)
    assert torch.equal(y, again[0]) and torch.equal(hT, again[1])


def _gradient_tolerances(x, g, wy, h0, dx, dg, dh0, T, grad):
    h = wy if h0 is None else np.concatenate([wy.reshape(-1), h0.reshape(-1)])
    # the running gradient del = dx / u is at most as large as its bound here
    u = O.sigmoid(-g.astype(np.float64))
    with np.errstate(divide="ignore", invalid="ignore"):
        d = np.nan_to_num(dx / u)
    mem = min(T, 1.0 / u.min())
    r = 3 * EPS * (24 + 8 * np.sqrt(mem)) * max(np.abs(d).max(), np.abs(dh0).max())
    size = np.abs(x).max() + np.abs(h).max()
    return (r + (2.0 ** -8 * np.abs(dx).max() if grad == "bf16" else 0),
            r * size + (2.0 ** -8 * np.abs(dg).max() if grad == "bf16" else 0), r)


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("layout", ["apart", "packed"])
def test_backward(env, B, T, D, dtype, grad, layout):
    torch, F = env
    x, g = _draw(torch, B, T, D, dtype, layout, B + 2 * T + D)
    ragged = layout == "packed"
    h0 = torch.randn(B, D, device="cuda:0") if T % 2 == 0 else None
    dhT = torch.randn(B, D, device="cuda:0") if T % 3 == 0 or ragged else None
    dy = torch.randn(B, T, D, device="cuda:0")
    lengths = torch.tensor([T, 0, T // 2, T + 5][:B] if B > 1 else [max(T - 1, 0)], dtype=torch.int32,
                           device="cuda:0") if ragged else None
    y, _ = F.kan_recur_forward(x, g, h0, lengths)
    gt = _dt(torch, grad)
    if layout == "packed":
        dp = torch.full((B, T, 2 * D), float("nan"), dtype=gt, device="cuda:0")
        dx, dg = dp[..., :D], dp[..., D:]
    else:
        dx, dg = (torch.full((B, T, D), float("nan"), dtype=gt, device="cuda:0") for _ in range(2))
    dh0 = F.kan_recur_backward(x, g, y, dy, h0, lengths, dhT, need_dh0=True, dx=dx, dg=dg)[2]
    ln = None if lengths is None else lengths.tolist()
    want = O.recur_backward(_np(x), _np(g), _np(dy), _np(h0), ln, _np(dhT))
    wy = O.recur_forward(_np(x), _np(g), _np(h0), ln)[0]
    tols = _gradient_tolerances(_np(x), _np(g), wy, _np(h0), *want, T, grad)
    for got, w, tol in zip((dx, dg, dh0), want, tols):
        assert np.abs(got.double().cpu().numpy() - w).max() <= tol
    dx2, dg2, dh2 = F.kan_recur_backward(x, g, y, dy, h0, lengths, dhT, need_dh0=True, grad_dtype=gt)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2) and torch.equal(dh0, dh2)


def test_gradient_by_differences(env):
    """The kernels' own forward at x, g, h0 moved by +-h along a direction: a
    central difference (error h^2 / 6 of the third derivative, h = 1e-2, and
    the forward's rounding over 2h) within 2e-3 of the gradient's size."""
    torch, F = env
    torch.manual_seed(2)
    B, T, D = 2, 90, 20
    x, g = torch.randn(B, T, D, device="cuda:0"), torch.randn(B, T, D, device="cuda:0") + 1
    h0, dy, dhT = torch.randn(B, D, device="cuda:0"), torch.randn(B, T, D, device="cuda:0"), torch.randn(
        B, D, device="cuda:0")
    y, _ = F.kan_recur_forward(x, g, h0)
    grads = F.kan_recur_backward(x, g, y, dy, h0, None, dhT)

    def loss(*a):
        yy, hT = F.kan_recur_forward(*a)
        return float((yy.double() * dy).sum() + (hT.double() * dhT).sum())

    for k in range(3):
        way = torch.randn_like((x, g, h0)[k])
        hi, lo = [x, g, h0], [x, g, h0]
        hi[k], lo[k] = hi[k] + 1e-2 * way, lo[k] - 1e-2 * way
        want = (loss(*hi) - loss(*lo)) / 2e-2
        got = float((grads[k].double() * way).sum())
        assert abs(got - want) <= 2e-3 * float((grads[k] * way).abs().sum().clamp(min=1)) ** 0.5 * 10


def test_what_lies_past_a_length_is_not_used(env):
    torch, F = env
    B, T, D = 3, 700, 40
    x, g = _draw(torch, B, T, D, "f32", "apart", 9)
    dy = torch.randn(B, T, D, device="cuda:0")
    lengths = torch.tensor([311, 0, 512], dtype=torch.int32, device="cuda:0")
    h0 = torch.randn(B, D, device="cuda:0")
    y, hT = F.kan_recur_forward(x, g, h0, lengths)
    grads = F.kan_recur_backward(x, g, y, dy, h0, lengths, hT)
    inside = torch.arange(T, device="cuda:0")[None, :, None] < lengths[:, None, None]
    for junk in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min):
        bad = [torch.where(inside, t, junk) for t in (x, g, dy, y)]
        y2, hT2 = F.kan_recur_forward(bad[0], bad[1], h0, lengths)
        assert torch.equal(y, y2) and torch.equal(hT, hT2)
        again = F.kan_recur_backward(bad[0], bad[1], bad[3], bad[2], h0, lengths, hT)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
    assert torch.equal(hT[1], h0[1]) and not y[1].any() and torch.equal(grads[2][1], hT[1])


@pytest.mark.parametrize("g", [100.0, -100.0, float("inf"), -float("inf"), 3.0e38, -3.0e38])
def test_saturated_gates(env, g):
    """A gate at its end keeps the state exactly, or replaces it exactly; at
    +-100 the other side's share is e^-100, below half an ulp."""
    torch, F = env
    x = torch.randn(2, 600, 10, device="cuda:0")
    h0 = torch.randn(2, 10, device="cuda:0")
    y, _ = F.kan_recur_forward(x, torch.full_like(x, g), h0)
    assert torch.equal(y, x if g < 0 else h0[:, None].expand_as(x))


def test_long_memories_keep_their_digits(env):
    """Gates of 1 - 2^-13: with x constant the state tends to x as 1 - f^t; over
    20000 steps (2.4 memories) each step's rounding adds less than
    2^-25 |x| sqrt(memory) * 8."""
    torch, F = env
    T = 20000
    g = np.log(2.0 ** 13 - 1)
    x = torch.full((1, T, 8), 3.0, device="cuda:0")
    gt = torch.full_like(x, g)
    y, _ = F.kan_recur_forward(x, gt)
    u = O.sigmoid(-np.float64(np.float32(g)))
    want = 3.0 * -np.expm1(np.arange(1, T + 1) * np.log1p(-u))
    tol = 3.0 * EPS * (24 + 4 * np.sqrt(2.0 ** 13))
    assert np.abs(y.double().cpu().numpy() - want[None, :, None]).max() <= tol


@pytest.mark.parametrize("B,T,D", [(2, 300, 36), (1, 3000, 8), (1, 5000, 3), (3, 700, 130)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_states_are_forgotten_exactly(env, B, T, D, dtype):
    """Single inputs and gradients of 3e7 among values around 1: what is left of
    them n rows on is a product of n shares, each within 24 e and rounded in at
    most 4 e more, so a row is within (28 T + 64) e of the sum of its
    contributions' sizes, whatever the largest value of the sequence.  What lies
    in earlier segments may be dropped once 2^-64 of it is left.  dg has three
    such factors."""
    torch, F = env
    x, g = _draw(torch, B, T, D, dtype, "apart", B + 3 * T + D, gate=(0.0, 1.5))
    dy = torch.randn(B, T, D, device="cuda:0")
    x[:, 40::97] = 3e7
    dy[:, 60::97] = -3e7
    h0 = torch.randn(B, D, device="cuda:0") * 3e7
    dhT = torch.randn(B, D, device="cuda:0") * 3e7
    y, hT = F.kan_recur_forward(x, g, h0)
    dx, dg, dh0 = F.kan_recur_backward(x, g, y, dy, h0, dhT=dhT)
    ax, ag, ad, ah, at = _np(x), _np(g), _np(dy), _np(h0), _np(dhT)
    wy, wh = O.recur_forward(ax, ag, ah)
    wdx, wdg, wdh = O.recur_backward(ax, ag, ad, ah, dhT=at)
    sy, sh = O.recur_forward(np.abs(ax), ag, np.abs(ah))
    sdx, _, sdh = O.recur_backward(ax, ag, np.abs(ad), ah, dhT=np.abs(at))
    f = O.sigmoid(ag.astype(np.float64))
    before = np.concatenate([np.abs(ah)[:, None], sy[:, :-1]], 1)
    sdg = f * sdx * (before + np.abs(ax))
    r = (28 * T + 64) * EPS

    def close(got, want, size, k=1):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= k * r * size + 2.0 ** -64 * size.max()).all()

    close(y, wy, sy)
    close(hT, wh, sh)
    close(dx, wdx, sdx)
    close(dh0, wdh, sdh)
    close(dg, wdg, sdg, 3)


def test_broadcast_inputs(env):
    """Stride 0: one gate for all rows and sequences."""
    torch, F = env
    x = torch.randn(3, 70, 12, device="cuda:0")
    g = torch.randn(12, device="cuda:0")
    a = F.kan_recur_forward(x, g.expand_as(x))
    b = F.kan_recur_forward(x, g.expand_as(x).contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("B,S,D", [(1, 1, 1), (5, 9, 3), (4, 4, 64), (64, 256, 770), (300, 301, 10), (3, 7, 4096)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step(env, B, S, D, dtype):
    torch, F = env
    x, g = _draw(torch, B, 1, D, dtype, "packed", B + D)
    x, g = x[:, 0], g[:, 0]
    state = torch.randn(S, D, device="cuda:0")
    before = state.clone()
    slots = torch.randperm(S, device="cuda:0")[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, S
    y = F.kan_recur_step(x, g, state, slots)
    h = _np(before)
    wy = np.zeros((B, D))
    wstate = h.astype(np.float64)
    for b, k in enumerate(slots.tolist()):
        if 0 <= k < S:
            wy[b] = O.recur_forward(_np(x)[b][None, None], _np(g)[b][None, None], h[k][None])[1][0]
            wstate[k] = wy[b]
    tol = _bound(_np(g), _np(x), h, 1)
    assert np.abs(y.double().cpu().numpy() - wy).max() <= tol
    assert np.abs(state.double().cpu().numpy() - wstate).max() <= tol
    used = [k for k in slots.tolist() if 0 <= k < S]
    rest = [k for k in range(S) if k not in used]
    assert torch.equal(state[rest], before[rest])


def test_steps_equal_the_sequence(env):
    """Row by row through the step and as one sequence: within two forward bounds."""
    torch, F = env
    B, T, D = 5, 40, 70
    x, g = _draw(torch, B, T, D, "f32", "apart", 4)
    y, hT = F.kan_recur_forward(x, g)
    state = torch.zeros(B, D, device="cuda:0")
    rows = torch.stack([F.kan_recur_step(x[:, t], g[:, t], state) for t in range(T)], 1)
    tol = 2 * _bound(_np(g), _np(x), _np(y), T)
    assert float((rows - y).abs().max()) <= tol and float((state - hT).abs().max()) <= tol


def test_empty(env):
    torch, F = env
    dev = "cuda:0"
    for shape in ((0, 5, 4), (2, 0, 4)):
        x = torch.empty(shape, device=dev)
        h0 = torch.randn(shape[0], 4, device=dev)
        y, hT = F.kan_recur_forward(x, x, h0)
        assert y.shape == shape and torch.equal(hT, h0)
        dx, dg, dh0 = F.kan_recur_backward(x, x, y, y, h0, dhT=h0)
        assert dx.shape == shape and torch.equal(dh0, h0)
    y, hT = F.kan_recur_forward(torch.empty(2, 0, 4, device=dev), torch.empty(2, 0, 4, device=dev))
    assert not hT.any()
    assert F.kan_recur_step(torch.empty(0, 4, device=dev), torch.empty(0, 4, device=dev),
                            torch.empty(3, 4, device=dev)).shape == (0, 4)


def test_refusals(env):
    torch, F = env
    from kolmogorov_arnold_network_amd import _lib as L
    dev = "cuda:0"
    x, g = torch.zeros(2, 6, 8, device=dev), torch.zeros(2, 6, 8, device=dev)
    for bad in (dict(x=x.half()), dict(g=g.bfloat16()), dict(g=g[:, :5]), dict(x=x[0], g=g[0]), dict(x=x.cpu()),
                dict(x=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(h0=torch.zeros(2, 7, device=dev)),
                dict(lengths=torch.zeros(2, dtype=torch.int64, device=dev)),
                dict(lengths=torch.zeros(3, dtype=torch.int32, device=dev)),
                dict(out=torch.zeros(2, 6, 9, device=dev))):
        with pytest.raises(ValueError):
            F.kan_recur_forward(**dict(dict(x=x, g=g), **bad))
    y = torch.zeros_like(x)
    for bad in (dict(dx=y.clone()), dict(dy=y.bfloat16()), dict(dhT=torch.zeros(6, 8, device=dev)),
                dict(dx=y.half(), dg=y.half())):
        with pytest.raises(ValueError):
            F.kan_recur_backward(**dict(dict(x=x, g=g, y=y, dy=y), **bad))
    one = torch.zeros(2, 6, 8, device=dev)
    for dx, dg, status in ((one, one, L.KAN_ERR_ALIAS), (x, one, L.KAN_ERR_ALIAS),
                           (torch.zeros(8, device=dev).expand(2, 6, 8), one, L.KAN_ERR_SHAPE)):
        with pytest.raises(L.KanError) as e:
            F.kan_recur_backward(x, g, y, one + 1, dx=dx, dg=dg)
        assert e.value.status == status
    # halves that overlap by one channel
    p = torch.zeros(2, 6, 15, device=dev)
    with pytest.raises(L.KanError) as e:
        F.kan_recur_backward(x, g, y, one + 1, dx=p[..., :8], dg=p[..., 7:])
    assert e.value.status == L.KAN_ERR_ALIAS
    for bad in (dict(state=torch.zeros(2, 7, device=dev)), dict(slots=torch.zeros(2, device=dev)),
                dict(state=torch.zeros(2, 8, device=dev).bfloat16())):
        with pytest.raises(ValueError):
            F.kan_recur_step(**dict(dict(x=x[:, 0], g=g[:, 0], state=torch.zeros(2, 8, device=dev)), **bad))
    with pytest.raises(L.KanError) as e:
        F.kan_recur_step(x[:, 0], g[:, 0], torch.zeros(1, 8, device=dev))         # fewer states than sequences
    assert e.value.status == L.KAN_ERR_SHAPE
