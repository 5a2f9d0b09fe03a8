"""GPU: gates far from 0, relatively, and the recurrence's gradient by differences.

A gate's smaller share is v / (1 + v) with v = exp(-|g|): |g| log2 e rounds to
|g| e in the exponent (e = 2^-24; log2 e itself to a quarter of that), exp, sum,
reciprocal and product add a few ulp.  So it is within (1.3 |g| + 12) e of its
own size, as long as float32 holds it (|g| <= 80: e^-80 = 1.8e-35).
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


def test_shares_of_large_gates(env):
    """x = 1 on a state of 0 gives u, x = 0 on a state of 1 gives f."""
    torch, F = env
    g = torch.linspace(0.0, 80.0, 4001, device="cuda:0")[None]
    one, zero = torch.ones_like(g), torch.zeros_like(g)
    want = O.sigmoid(-g.double().cpu().numpy()[0])
    tol = (1.3 * g.double().cpu().numpy()[0] + 12) * EPS * want
    up = F.kan_recur_step(one, g, zero.clone()), F.kan_recur_forward(one[:, None], g[:, None])[1]
    left = F.kan_recur_step(zero, -g, one.clone()), F.kan_recur_forward(zero[:, None], -g[:, None], one)[1]
    for y in up + left:
        assert (np.abs(y.double().cpu().numpy()[0] - want) <= tol).all()


@pytest.mark.parametrize("T,D", [(40, 33), (300, 20)])
def test_large_gates_of_a_sequence(env, T, D):
    """Gates of +-16 .. 40 in turn at random: a row is within the sum of its
    contributions' errors, each of at most T shares (1.3 40 + 12) e."""
    torch, F = env
    torch.manual_seed(T)
    x = torch.randn(2, T, D, device="cuda:0")
    sign = torch.where(torch.rand(2, T, D, device="cuda:0") < 0.02, -1.0, 1.0)
    g = (16 + 24 * torch.rand(2, T, D, device="cuda:0")) * sign
    ax, ag = x.cpu().numpy(), g.cpu().numpy()
    y, hT = F.kan_recur_forward(x, g)
    wy, wh = O.recur_forward(ax, ag)
    sy, sh = O.recur_forward(np.abs(ax), ag)
    # shares near 1 are within e; those near 0 within 64 e; roundings of a row's sum
    tol = (64 + 4 * T) * EPS
    assert (np.abs(y.double().cpu().numpy() - wy) <= tol * sy).all()
    assert (np.abs(hT.double().cpu().numpy() - wh) <= tol * sh).all()


def test_gradient_by_differences_of_its_terms_size(env):
    """Central differences of the kernels' own forward at h = 1e-2.  x and h0 enter
    linearly; for g the third derivative leaves at most h^2 / 6 * 6 |way|^2 of a
    term.  The forward's rounding, 64 e of its rows twice over 2 h, against dy:
    in all 1e-3 of the terms' sizes and 64 e / h of the outputs'."""
    torch, F = env
    torch.manual_seed(2)
    B, T, D = 2, 90, 20
    x, g = torch.randn(B, T, D, device="cuda:0"), torch.randn(B, T, D, device="cuda:0") + 1
    h0, dy, dhT = torch.randn(B, D, device="cuda:0"), torch.randn(B, T, D, device="cuda:0"), torch.randn(
        B, D, device="cuda:0")
    y, hT = F.kan_recur_forward(x, g, h0)
    grads = F.kan_recur_backward(x, g, y, dy, h0, None, dhT)

    def loss(*a):
        yy, h = F.kan_recur_forward(*a)
        return float((yy.double() * dy).sum() + (h.double() * dhT).sum())

    outputs = float((y * dy).abs().sum() + (hT * dhT).abs().sum())
    for k in range(3):
        way = torch.randn_like((x, g, h0)[k])
        hi, lo = [x, g, h0], [x, g, h0]
        hi[k], lo[k] = hi[k] + 1e-2 * way, lo[k] - 1e-2 * way
        want = (loss(*hi) - loss(*lo)) / 2e-2
        terms = grads[k].double() * way
        assert abs(float(terms.sum()) - want) <= 1e-3 * float(terms.abs().sum()) + 64 * EPS / 1e-2 * outputs
