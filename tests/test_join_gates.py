"""GPU: digits of the join's gate where it is far from zero.

With e = 2^-24 and no norm, act(g) h is off by: the exponential, whose argument keeps
the digits of g and which the hardware gives to 2 e, and its correction e; the sum
and the reciprocal 3 e; the share, its product with g and that with h 3 e: 9 e of
the value.  The slope is a sum of two such terms, 10 e of each, and takes three more
products.  Values below 2^-126 may be 0.
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


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("D", [100, 770, 2048])
def test_gates_far_from_zero(env, activation, D):
    torch, F = env
    gen = torch.Generator(device="cuda:0").manual_seed(D)
    h, g, dy = torch.randn(3, 9, D, device="cuda:0", generator=gen)
    g = (torch.rand(9, D, device="cuda:0", generator=gen) * 2 - 1) * 80
    y, _, stats = F.kan_join_forward(h, None, g, post=False, pre=False, activation=activation)
    gd, hd = _np(g), _np(h)
    act, slope = O._act(activation, gd)
    want = act * hd
    assert (np.abs(_np(y) - want) <= 9 * E * np.abs(want) + 2.0 ** -120).all(), (np.abs(_np(y) / want - 1)).max() / E
    dh, _, dgate, _, _ = F.kan_join_backward(h, y, stats, dy, None, g, post=False, activation=activation)
    want = act * _np(dy)
    assert (np.abs(_np(dh) - want) <= 9 * E * np.abs(want) + 2.0 ** -120).all()
    s = O._act("sigmoid", gd)[0]
    o = O._act("sigmoid", -gd)[0]        # 1 - s
    terms = s + np.abs(gd) * s * o if activation == "silu" else s * o
    want = slope * _np(dy) * hd
    assert (np.abs(_np(dgate) - want) <= 13 * E * terms * np.abs(_np(dy) * hd) + 2.0 ** -120).all()


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_gates_at_the_ends(env, activation):
    """Infinite gates, those past the exponential's range, and NaN."""
    torch, F = env
    inf = float("inf")
    g = torch.tensor([[inf, 3e38, 200.0, 128.0, 100.0, -100.0, -128.0, -200.0, -3e38, 0.0, -0.0, float("nan")]],
                     device="cuda:0")
    h = torch.ones_like(g)
    y, _, _ = F.kan_join_forward(h, None, g, post=False, pre=False, activation=activation)
    y = _np(y)[0]
    want = [inf, 3e38, 200.0, 128.0, 100.0] if activation == "silu" else [1.0] * 5
    assert y[:5] == pytest.approx(want) and np.abs(y[5:9]).max() < 1e-36
    assert (y[9:11] == (0.0 if activation == "silu" else 0.5)).all() and np.isnan(y[11])
    low = F.kan_join_forward(h[:, :1].contiguous(), None, torch.full((1, 1), -inf, device="cuda:0"), post=False,
                             pre=False, activation="sigmoid")[0]
    assert (low == 0).all()
