"""The recurrence's segments: a channel's run is stored by one block, so that
results are the same on every call where the last channels share a lane with
those of the block before.

A CPU walk over the channels of blocks and lanes (``host/recur_lanes_check.cpp``),
and on the GPU the same bits from repeated calls on inputs whose runs end at
different rows in neighbouring blocks.
"""

import os
import subprocess

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import token as O
from test_host_sanitize import CSRC, HERE, ROOT, _hipcc


def test_every_channel_has_one_block(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "recur_lanes_check")
    cmd = [cc, "--offload-host-only", "-std=c++17", "-O2", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o",
           out, os.path.join(HERE, "host", "recur_lanes_check.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    res = subprocess.run([out], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.startswith("ok "), res.stdout + res.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("D", [65, 66, 67, 130, 770])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_repeat_themselves(D, dtype):
    """Inputs and gradients of 1e18 at a few rows and 0 elsewhere, so that what
    2^-64 leaves of them is all that a row has; gates of the first channels
    forget in a few rows, those of the last ones hardly.  A row within (28 T +
    64) e of its contributions' sizes, or 2^-64 of the largest dropped."""
    ensure_built()
    import torch
    from kolmogorov_arnold_network_amd import _lib as L
    from kolmogorov_arnold_network_amd import functional as F
    T = 6000 if D < 500 else 2500
    print("channels", D, dtype, flush=True)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, dy = torch.zeros(1, T, D, device="cuda:0"), torch.zeros(1, T, D, device="cuda:0")
    x[:, 5::701], dy[:, 9::701] = 1e18, -1e18
    g = torch.randn(1, T, D, device="cuda:0", generator=gen) * 0.5
    g[..., D - 3:] += 4.0                                     # about 50 rows
    x, g = x.to(dt), g.to(dt)
    for p in (L.KAN_PASS_FORWARD, L.KAN_PASS_BACKWARD):
        assert F.kan_recur_workspace_size(F.recur_desc(x, g, dy, dy), p) > 0        # in segments
    y, hT = F.kan_recur_forward(x, g)
    dx, dg, _ = F.kan_recur_backward(x, g, y, dy)
    for _ in range(8):
        assert all(torch.equal(a, b) for a, b in zip((y, hT), F.kan_recur_forward(x, g)))
        assert all(torch.equal(a, b) for a, b in zip((dx, dg), F.kan_recur_backward(x, g, y, dy)[:2]))
    ax, ag, ad = (v.float().cpu().numpy() for v in (x, g, dy))
    wy, _ = O.recur_forward(ax, ag)                           # all of one sign: also the contributions' sizes
    sdx, _, _ = O.recur_backward(ax, ag, np.abs(ad))
    r = (28 * T + 64) * 2.0 ** -24
    for got, size, want in ((y, wy, wy), (dx, sdx, -sdx)):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= r * size + 2.0 ** -64 * size.max() + 1e-37).all()
