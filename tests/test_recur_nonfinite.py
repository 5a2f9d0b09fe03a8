"""GPU: infinities and NaN among the recurrence's states, against the float64
oracle's ``f h + u x``: an infinite state stays one, and a value that float32
holds comes out finite (tolerance 32 e of |h| + |x|: a gate within 24 e, two
products and a sum)."""

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import token as O

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


def _np(t):
    return t.detach().double().cpu().numpy()


def test_step_with_infinite_and_huge_states(env):
    torch, F = env
    h = torch.tensor([INF, -INF, INF, -INF, 1.0, 2.0, 3e38, -3e38, 3e38, INF, float("nan"), 1.0], device="cuda:0")
    x = torch.tensor([1.0, 2.0, -3.0, 3e38, INF, -INF, -3e38, 3e38, 3e38, INF, 1.0, float("nan")], device="cuda:0")
    for gate in (-9.0, -1.0, 0.0, 0.5, 4.0, 11.0):
        g = torch.full((1, 12), gate, device="cuda:0")
        state = h[None].clone()
        y = F.kan_recur_step(x[None], g, state)
        assert torch.equal(y.nan_to_num(7.0), state.nan_to_num(7.0))
        with np.errstate(all="ignore"):
            want = O.recur_forward(_np(x)[None, None], _np(g)[None], _np(h)[None])[1][0]
        got = _np(y)[0]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        far = np.isinf(want)
        assert np.array_equal(got[far], want[far])
        near = np.isfinite(want)
        size = np.abs(_np(h)) + np.abs(_np(x))
        assert (np.abs(got - want)[near] <= 32 * EPS * size[near]).all()


@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 3, 5), (3, 70, 64), (2, 600, 36), (2, 1300, 3)])
@pytest.mark.parametrize("gate", [-1.0, 0.0, 3.0])
def test_an_infinite_state_stays(env, B, T, D, gate):
    """h0 infinite in every third channel: so is each row (shares of 1/4 to 19/20,
    so that no float32 product of a tile's shares is 0 before row 60), and the
    others are what they are without it."""
    torch, F = env
    print("states", B, T, D, gate, flush=True)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(T)
    x = torch.randn(B, T, D, device="cuda:0", generator=gen)
    g = torch.full_like(x, gate)
    h0 = torch.randn(B, D, device="cuda:0", generator=gen)
    plain, _ = F.kan_recur_forward(x, g, h0)
    h0[:, ::3] = INF
    h0[:, ::6] = -INF
    y, hT = F.kan_recur_forward(x, g, h0)
    n = min(T, 60)
    assert torch.equal(y[:, :n, ::3], h0[:, None, ::3].expand(B, n, -1))
    assert not torch.isfinite(y[:, :, ::3]).any() and not torch.isfinite(hT[:, ::3]).any()
    rest = [c for c in range(D) if c % 3]
    assert torch.equal(y[..., rest], plain[..., rest])


@pytest.mark.parametrize("T", [64, 700])
def test_an_infinite_gradient_stays(env, T):
    torch, F = env
    torch.manual_seed(T)
    x, g = torch.randn(2, T, 40, device="cuda:0"), torch.randn(2, T, 40, device="cuda:0") * 0.3 + 2
    dy, dhT = torch.randn(2, T, 40, device="cuda:0"), torch.randn(2, 40, device="cuda:0")
    y, _ = F.kan_recur_forward(x, g)
    h0 = torch.zeros(2, 40, device="cuda:0")
    plain = F.kan_recur_backward(x, g, y, dy, h0, dhT=dhT)
    dhT[:, ::4] = INF
    dx, dg, dh0 = F.kan_recur_backward(x, g, y, dy, h0, dhT=dhT)
    n = min(T, 60)
    assert (dx[:, T - n:, ::4] == INF).all()
    assert not torch.isfinite(dx[..., ::4]).any() and not torch.isfinite(dh0[:, ::4]).any()
    rest = [c for c in range(40) if c % 4]
    assert all(torch.equal(a[..., rest], b[..., rest]) for a, b in zip((dx, dg, dh0), plain))


# segments of one tile, which are read whole, and of several, which are not
LONG = [(1, 9000, 24), (1, 5000, 3), (2, 4000, 130), (1, 3000, 770), (3, 2500, 66), (1, 70000, 24), (1, 66000, 64),
        (1, 8192, 1024), (2, 8192, 770)]


@pytest.mark.parametrize("B,T,D", LONG)
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_not_finite_reaches_the_end_of_its_sequence(env, B, T, D, bad, dtype):
    """One bad input (gradient) near the start (end) of a sequence that is cut into
    segments, with gates that forget within a segment: the rows of its channel
    that are finite are those of the oracle, and the other channels keep their
    values (within 1e-5 of the largest, as without it)."""
    torch, F = env
    from kolmogorov_arnold_network_amd import _lib as L
    print("long", B, T, D, bad, dtype, flush=True)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(T + D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.randn(B, T, D, device="cuda:0", generator=gen).to(dt)
    g = torch.randn(B, T, D, device="cuda:0", generator=gen).to(dt)
    dy = torch.randn(B, T, D, device="cuda:0", generator=gen)
    lengths = torch.full((B,), T - 7, dtype=torch.int32, device="cuda:0")
    for p in (L.KAN_PASS_FORWARD, L.KAN_PASS_BACKWARD):
        assert F.kan_recur_workspace_size(F.recur_desc(x, g, dy, dy), p) > 0        # in segments
    h0 = torch.zeros(B, D, device="cuda:0")
    y, hT = F.kan_recur_forward(x, g, h0, lengths)
    plain = (y, hT) + F.kan_recur_backward(x, g, y, dy, h0, lengths)
    c = D - 1
    bx, bdy = x.clone(), dy.clone()
    bx[B - 1, 11, c] = bad
    bdy[B - 1, T - 20, c] = bad
    yb, hTb = F.kan_recur_forward(bx, g, h0, lengths)
    got = (yb, hTb) + F.kan_recur_backward(x, g, y, bdy, h0, lengths)
    with np.errstate(all="ignore"):
        ab, ag, n = _np(bx[B - 1:, :, c:]), _np(g[B - 1:, :, c:]), [T - 7]
        want = O.recur_forward(ab, ag, None, n) + O.recur_backward(_np(x[B - 1:, :, c:]), ag, _np(bdy[B - 1:, :, c:]),
                                                                   None, n)
    for a, b, w in zip(got, plain, want):
        assert np.array_equal(np.isfinite(_np(a)[B - 1, ..., c]), np.isfinite(w)[0, ..., 0])
        clean = torch.ones_like(a, dtype=torch.bool)
        clean[B - 1, ..., c] = False
        assert float((a - b)[clean].abs().max()) <= 1e-5 * float(b.abs().max())


def test_a_cut_sequence_shows_what_a_whole_one_does(env):
    """The same rows alone (in segments) and in a batch that is not cut."""
    torch, F = env
    from kolmogorov_arnold_network_amd import _lib as L
    torch.manual_seed(5)
    x, g = torch.randn(300, 2600, 24, device="cuda:0"), torch.randn(300, 2600, 24, device="cuda:0")
    x[0, 40, 3], g[0, 90, 7], x[0, 1700, 9] = INF, float("nan"), -INF
    size = [F.kan_recur_workspace_size(F.recur_desc(a, a), L.KAN_PASS_FORWARD) for a in (x, x[:1])]
    assert size[0] == 0 and size[1] > 0
    y, hT = F.kan_recur_forward(x, g)
    y1, hT1 = F.kan_recur_forward(x[:1], g[:1])
    assert torch.equal(torch.isfinite(y[:1]), torch.isfinite(y1))
    assert torch.equal(torch.isfinite(hT[:1]), torch.isfinite(hT1))
    assert torch.isfinite(hT1).sum() == 21
