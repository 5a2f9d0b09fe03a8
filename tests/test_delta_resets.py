"""GPU: a decay that wipes out the state and growth (g > 0) after it, in one chunk of
rows, against the float64 oracle and the step of one row.

Tolerances are those of the delta rule's tests: 5 sqrt(128) 2^-24 of the largest row
norm for each chunk, three times that backward, and 2^-8 for bfloat16 outputs.  Rows
before the decay are as large as the state that it wipes out, those after it are
not, so that the two are held to their own norms.  What is below the least float32
is 0.
"""

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import delta as O

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
LARGE = 1e30


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol):
    want = want.astype(np.float32).astype(np.float64)
    got, want = (t.reshape(-1, t.shape[-1]) if t.ndim > 3 else t.reshape(-1, 1) for t in (got, want))
    assert np.isfinite(got).all()
    size, off = np.linalg.norm(want, axis=-1).max(), np.linalg.norm(got - want, axis=-1).max()
    assert off <= tol * size, (off, size)


def _draw(torch, at, g_reset, dtype, T=100):
    """Row `at` wipes the state out, the two rows behind it let what is left grow by exp(70)."""
    B, H, Dk, Dv = 2, 2, 40, 48
    gen = torch.Generator(device="cuda:0").manual_seed(at + T)

    def rand(*shape):
        return torch.randn(*shape, device="cuda:0", generator=gen)
    q, k, v = rand(B, T, H, Dk), rand(B, T, H, Dk), rand(B, T, H, Dv)
    k = k / (k.norm(dim=-1, keepdim=True) * 1.01)
    g, beta = -0.1 * rand(B, T, H).abs(), torch.sigmoid(rand(B, T, H))
    g[:, at], g[:, at + 1:at + 3], beta[:, at:at + 3] = g_reset, 35.0, 0.0
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return [q.to(dt), k.to(dt), v.to(dt), g, beta, LARGE * rand(B, H, Dk, Dv)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g_reset", [-300.0, -1e30, -float("inf")])
@pytest.mark.parametrize("at", [0, 20, 61, 64, 97])
def test_growth_after_a_reset(env, at, g_reset, dtype):
    torch, F = env
    args = _draw(torch, at, g_reset, dtype)
    y, hT = F.kan_delta_forward(*args)
    wy, wh = O.delta_forward(*map(_np, args))
    tol = 5 * np.sqrt(128) * E * np.sqrt(2)
    out = tol + (2.0 ** -8 if dtype == "bf16" else 0)
    _close(_np(y)[:, at:], wy[:, at:], out)
    _close(_np(hT), wh, tol)
    state, rows = args[5].clone(), []
    for t in range(y.shape[1]):
        rows.append(F.kan_delta_step(*(x[:, t].contiguous() for x in args[:5]), state))
    _close(_np(torch.stack(rows[at:], 1)), wy[:, at:], out)
    _close(_np(state), wh, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g_reset", [-300.0, -1e30, -float("inf")])
def test_gradients_with_growth_after_a_reset(env, g_reset, dtype):
    torch, F = env
    args = _draw(torch, 0, g_reset, dtype)
    dy = torch.randn(2, 100, 2, 48, device="cuda:0").to(args[0].dtype)
    dhT = torch.randn(2, 2, 40, 48, device="cuda:0")
    got = F.kan_delta_backward(*args[:5], dy, args[5], None, dhT)
    want = O.delta_backward(*map(_np, args[:5]), _np(dy), _np(args[5]), None, _np(dhT))
    tol = 15 * np.sqrt(128) * E * np.sqrt(2)
    for i, (a, b) in enumerate(zip(got, want)):
        _close(_np(a), b, tol + (2.0 ** -8 if dtype == "bf16" and i < 3 else 0))


def test_decays_below_the_least_float_are_exact(env):
    """g = -140 and growth by 70 in the same chunk leave exp(-70) of a large state."""
    torch, F = env
    args = _draw(torch, 0, -140.0, "f32")
    y, hT = F.kan_delta_forward(*args)
    wy, wh = O.delta_forward(*map(_np, args))
    tol = 5 * np.sqrt(128) * E * np.sqrt(2)
    _close(_np(y), wy, tol)
    _close(_np(hT), wh, tol)
