"""The gated delta rule with many heads, whose scans have blocks of four groups of 16
state columns, at every padded width of keys: forward and backward against the
float64 oracle (GPU), and that the shapes here are laid out so (host).

The tolerances are those of the delta rule's tests, of the largest row error against
the largest row norm: 5 sqrt(128) 2^-24 sqrt(chunks), three times that backward, and
2^-8 for bfloat16 outputs.  A few sequences are repeated through the batch: the
oracle walks through those, and every repetition has to be equal bit by bit.
"""

import os
import subprocess

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import delta as O
from test_host_sanitize import CSRC, HERE, ROOT, _hipcc

E = 2.0 ** -24
KINDS = 5                            # different sequences of a batch

# (B, T, Hk, Hv, Dk, Dv): keys padded to 32, 64 and 128, whole pieces of eight and odd ones, values of
# one block of columns, of more and of a part of one, shared heads
SHAPES = [(128, 70, 2, 2, 32, 64), (128, 130, 2, 2, 64, 64), (130, 129, 1, 2, 128, 64), (64, 100, 2, 4, 33, 33),
          (65, 130, 1, 2, 65, 130), (32, 128, 4, 4, 128, 128), (130, 65, 1, 2, 96, 72), (130, 129, 2, 2, 127, 40),
          (43, 64, 3, 6, 63, 57)]


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


def test_shapes_have_four_groups(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "delta_groups")
    cmd = [cc, "--offload-host-only", "-std=c++17", "-O1", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o", out,
           os.path.join(CSRC, "kan_delta_api.cpp"), os.path.join(HERE, "host", "delta_groups.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    shapes = [",".join(map(str, (*s, dtype))) for s in SHAPES for dtype in (0, 1)]
    res = subprocess.run([out, *shapes], capture_output=True, text=True, timeout=60)
    plans = [tuple(map(int, line.split())) for line in res.stdout.splitlines()]
    assert res.returncode == 0 and len(plans) == len(shapes)
    assert all(p[1:] == (4, 1, 4, 1) for p in plans), plans
    assert {p[0] for p in plans} == {32, 64, 128}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(torch, B, T, Hk, Hv, Dk, Dv, dtype, layout):
    gen = torch.Generator(device="cuda:0").manual_seed(B + T + Dk + Dv)
    pick = torch.arange(B, device="cuda:0") % KINDS

    def rand(*shape):
        return torch.randn(KINDS, *shape, device="cuda:0", generator=gen)[pick]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = rand(T, Hk, Dk), rand(T, Hk, Dk), rand(T, Hv, Dv)
    k = k / (k.norm(dim=-1, keepdim=True) * 1.01)
    q, k, v, dy = (t.to(dt) for t in (q, k, v, rand(T, Hv, Dv)))
    if layout == "slices":               # at odd columns of one array's rows, with NaN between them
        p = torch.full((B, T, 2 * Hk * Dk + Hv * Dv + 12), float("nan"), dtype=dt, device="cuda:0")
        out, at = [], 3
        for t in (q, k, v):
            p[..., at:at + t.shape[2] * t.shape[3]] = t.flatten(2)
            out.append(p[..., at:at + t.shape[2] * t.shape[3]].unflatten(-1, t.shape[2:]))
            at += t.shape[2] * t.shape[3] + 3
        q, k, v = out
    g, beta = -0.3 * rand(T, Hv).abs(), torch.sigmoid(rand(T, Hv))
    lengths = torch.tensor([T, T // 2, 0, 1, T - 1], dtype=torch.int32, device="cuda:0")[pick]
    return (q, k, v, g, beta), dy, rand(Hv, Dk, Dv), rand(Hv, Dk, Dv), lengths


def _check(got, want, tol, name):
    """The sequences of the oracle's, and each repetition of them."""
    for b in range(KINDS, got.shape[0], KINDS):
        n = min(KINDS, got.shape[0] - b)
        assert bool((got[b:b + n] == got[:n]).all()), (name, b)
    got = _np(got[:KINDS])
    got, want = (t.reshape(-1, t.shape[-1]) if t.ndim > 3 else t.reshape(-1, 1) for t in (got, want))
    assert np.isfinite(got).all(), name
    size, off = np.linalg.norm(want, axis=-1).max(), np.linalg.norm(got - want, axis=-1).max()
    assert off <= tol * size, (name, off / size)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["apart", "slices"])
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SHAPES)
def test_forward_and_backward(env, B, T, Hk, Hv, Dk, Dv, layout, dtype):
    torch, F = env
    args, dy, h0, dhT, lengths = _inputs(torch, B, T, Hk, Hv, Dk, Dv, dtype, layout)
    n = None if layout == "apart" else lengths
    some = [t[:KINDS] for t in (*args, dy, h0, dhT)]
    few = None if n is None else n[:KINDS].tolist()
    tol, half = 5 * np.sqrt(128) * E * np.sqrt(-(-T // 64)), 2.0 ** -8 if dtype == "bf16" else 0.0
    got = F.kan_delta_forward(*args, h0, n)
    want = O.delta_forward(*map(_np, some[:5]), _np(some[6]), few)
    _check(got[0], want[0], tol + half, "y")
    _check(got[1], want[1], tol, "hT")
    got = F.kan_delta_backward(*args, dy, h0, n, dhT)
    want = O.delta_backward(*map(_np, some[:5]), _np(some[5]), _np(some[6]), few, _np(some[7]))
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want):
        _check(a, b, 3 * tol + (half if name in ("dq", "dk", "dv") else 0), name)
