"""The distillation's gradient: each element is stored by one thread, so that the
teacher's entries come out the same whatever the order in which stores land.

A CPU walk over the kernels' store loops (``host/distill_rows_check.cpp``), and
on the GPU the same bits from repeated calls on every path, with entries at a
row's head, tail and parts, against the float64 oracle.  Tolerance of an
element: float32 results as in ``test_distill``, (3 R + 8 + V / 256 + 16) e of
q + p with R the range of the logits, plus 2^-8 where dz is bf16.
"""

import os
import subprocess

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import token as O
from test_host_sanitize import CSRC, HERE, ROOT, _hipcc

EPS = 2.0 ** -24


def test_every_element_has_one_thread(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "distill_rows_check")
    cmd = [cc, "--offload-host-only", "-std=c++17", "-O2", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o",
           out, os.path.join(HERE, "host", "distill_rows_check.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    res = subprocess.run([out], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.startswith("ok "), res.stdout + res.stderr


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


# rows of more than one wave, stored plainly and (past 128 MiB) as streamed data, cut and whole
SHAPES = [(3, 5001, 64), (40, 9001, 300), (300, 20003, 128), (4, 131075, 200), (2100, 50021, 128), (2700, 50021, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,K", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_entries_come_out_the_same_on_every_call(env, N, V, K, dtype):
    torch, F = env
    print("rows", N, V, K, dtype, flush=True)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(N + V + K)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z = (torch.randn(N, V, device="cuda:0", generator=gen) * 2.5).to(dt)
    ids = torch.randint(0, V, (N, K), device="cuda:0", generator=gen)
    ids[:, 0], ids[:, 1] = 0, V - 1                       # head and tail
    ids[:, 2:6] = torch.arange(V // 2, V // 2 + 4, device="cuda:0")      # one vector
    ids[1, 6:9] = 7                                       # one id three times
    t = torch.randn(N, K, device="cuda:0", generator=gen) * 2
    dloss = torch.rand(N, device="cuda:0", generator=gen) + 0.5
    _, lse = F.kan_distill_forward(z, ids, t)
    got = F.kan_distill_backward(z, ids, t, lse, dloss, grad_dtype=dt)
    step = F.kan_distill_step(z, ids, t, grad_dtype=dt)[1]
    again = torch.empty_like(got)
    for _ in range(4):
        again.fill_(float("nan"))
        assert torch.equal(F.kan_distill_backward(z, ids, t, lse, dloss, out=again), got)
        again.fill_(float("nan"))
        assert torch.equal(F.kan_distill_step(z, ids, t, out=again)[1], step)
    rows = [0, 1, N // 2, N - 1]
    nz, nt = z[rows].float().cpu().numpy(), t[rows].cpu().numpy()
    want = O.distill(nz, ids[rows].cpu().numpy(), nt, 1.0, None, np.ones(len(rows)))[2]
    R = min(88.0, max(np.ptp(nz), np.ptp(nt)) + np.log(V))
    q = np.exp(nz.astype(np.float64) - O.distill(nz, ids[rows].cpu().numpy(), nt, 1.0)[1][:, None])
    at = np.zeros_like(q)
    np.put_along_axis(at, ids[rows].cpu().numpy(), 1.0, 1)
    tol = (3 * R + 24 + V / 256) * EPS * (q + at) * 1.1 + (2.0 ** -8 + EPS) * np.abs(want) * (dtype == "bf16") + 1e-38
    scale = dloss[rows].double().cpu().numpy()[:, None]
    assert (np.abs(step[rows].double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(got[rows].double().cpu().numpy() / scale - want) <= 1.1 * tol + 4 * EPS * (np.abs(nz).max() + 30) * q).all()
