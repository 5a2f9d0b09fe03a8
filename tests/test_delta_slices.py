"""Gradients of the gated delta rule that are slices of one array: which layouts are
taken (host, with launchers that do nothing; every answer is checked against the
sets of elements themselves) and that they are written in full and nothing else (GPU)."""

import os
import subprocess

import numpy as np
import pytest

from kan_testutil import ensure_built
from test_host_sanitize import CSRC, HERE, ROOT, _hipcc

# (B, T, Hk, Hv, Dk, Dv), then place and strides of dq, dk and dv
APART = [
    ((2, 6, 2, 4, 8, 10), (0, 432, 72, 8), (16, 432, 72, 8), (32, 432, 72, 10)),          # in a row
    ((2, 6, 4, 4, 8, 10), (0, 624, 104, 26), (8, 624, 104, 26), (16, 624, 104, 26)),      # in a head
    ((2, 6, 4, 4, 10, 8), (18, 672, 112, 28), (8, 672, 112, 28), (0, 672, 112, 28)),
    ((2, 6, 4, 4, 8, 8), (0, 576, 32, 8), (192, 576, 32, 8), (384, 576, 32, 8)),          # in a sequence
    ((3, 5, 2, 2, 4, 4), (0, 8, 72, 4), (24, 8, 72, 4), (48, 8, 72, 4)),                  # sequences inside rows
    ((2, 6, 4, 4, 8, 8), (0, 8, 48, 288), (16, 8, 48, 288), (32, 8, 48, 288)),            # sequences inside rows inside heads
    ((1, 6, 1, 1, 8, 8), (0, 7, 24, 3), (8, 5, 24, 1), (16, 0, 24, 0)),                   # strides of one entry
]
OVERLAPPING = [
    ((2, 6, 4, 4, 8, 10), (0, 600, 100, 25), (8, 600, 100, 25), (16, 600, 100, 25)),      # 26 columns a head
    ((2, 6, 4, 4, 8, 10), (0, 624, 104, 26), (7, 624, 104, 26), (16, 624, 104, 26)),
    ((2, 6, 2, 4, 8, 10), (0, 432, 72, 8), (16, 432, 72, 8), (31, 432, 72, 10)),
    ((2, 6, 4, 4, 8, 8), (0, 576, 32, 8), (191, 576, 32, 8), (384, 576, 32, 8)),
    ((2, 6, 4, 4, 8, 8), (0, 568, 32, 8), (192, 568, 32, 8), (384, 568, 32, 8)),
    ((2, 6, 4, 4, 8, 10), (0, 624, 104, 26), (8, 624, 104, 26), (18, 624, 104, 26)),
    ((2, 6, 4, 4, 8, 8), (0, 576, 32, 8), (192, 576, 32, 8), (0, 576, 32, 8)),
]


def _elements(shape, place, which):
    B, T, Hk, Hv, Dk, Dv = shape
    at, seq, row, head = place
    H, D = (Hv, Dv) if which == 2 else (Hk, Dk)
    return {at + b * seq + t * row + h * head + c for b in range(B) for t in range(T) for h in range(H) for c in range(D)}


def test_layouts(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not found")
    for cases, apart in ((APART, True), (OVERLAPPING, False)):
        for shape, *places in cases:
            sets = [_elements(shape, p, i) for i, p in enumerate(places)]
            assert (len(set.union(*sets)) == sum(map(len, sets))) == apart, (shape, places)
    out = str(tmp_path / "delta_slices")
    cmd = [cc, "--offload-host-only", "-std=c++17", "-O1", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o", out,
           os.path.join(CSRC, "kan_delta_api.cpp"), os.path.join(HERE, "host", "delta_slices.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    r = np.random.default_rng(0)
    drawn = []                           # layouts whose refusal is the sets' own, or caution, but never their acceptance
    for _ in range(400):
        B, T, H, D = (int(n) for n in r.integers(1, 4, 4))
        dims = [(B, 0), (T, 1), (H, 2), (3, 3)]
        stride, strides = D + int(r.integers(0, 2)), [0] * 4
        for n, i in [dims[i] for i in r.permutation(4)]:
            strides[i] = stride
            stride = max(1, stride * n - int(r.integers(0, 3)) * int(r.integers(0, 2)))
        drawn.append(((B, T, H, H, D, D), *((i * strides[3], *strides[:3]) for i in range(3))))
    cases = APART + OVERLAPPING + drawn
    res = subprocess.run([out, *(",".join(map(str, (*s, *a, *b, *c))) for s, a, b, c in cases)], capture_output=True,
                         text=True, timeout=60)
    got = [int(line) for line in res.stdout.split()]
    assert res.returncode == 0 and len(got) == len(cases)
    from kolmogorov_arnold_network_amd import _lib as L
    assert got[:len(APART)] == [L.KAN_OK] * len(APART)
    assert got[len(APART):len(APART) + len(OVERLAPPING)] == [L.KAN_ERR_ALIAS] * len(OVERLAPPING)
    taken = 0
    for (shape, *places), status in zip(drawn, got[len(APART) + len(OVERLAPPING):]):
        sets = [_elements(shape, p, i) for i, p in enumerate(places)]
        assert status in (L.KAN_OK, L.KAN_ERR_ALIAS, L.KAN_ERR_SHAPE)
        if status == L.KAN_OK:
            taken += 1
            assert len(set.union(*sets)) == sum(map(len, sets)), (shape, places)
    assert taken > 100


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("axis", [1, 2, 3])
@pytest.mark.parametrize("D", [24, 33])
def test_gradients_beside_each_other(dtype, axis, D):
    """In a sequence, a row or a head of one array, with columns between them that stay as they were."""
    ensure_built()
    import torch
    from kolmogorov_arnold_network_amd import functional as F
    B, T, H = 3, 70, 2
    torch.manual_seed(D + axis)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, dy = (torch.randn(B, T, H, D, device="cuda:0").to(dt) for _ in range(4))
    g, beta = -torch.rand(B, T, H, device="cuda:0"), torch.rand(B, T, H, device="cuda:0")
    want = F.kan_delta_backward(q, k, v, g, beta, dy, unit=True)
    shape = [B, T, H]
    shape.insert(axis, 4)
    p = torch.full((*shape, D + 1), 7.0, dtype=dt, device="cuda:0")
    dq, dk, dv = (p.select(axis, i)[..., :D] for i in (0, 2, 3))
    got = F.kan_delta_backward(q, k, v, g, beta, dy, unit=True, dq=dq, dk=dk, dv=dv)
    assert got[0] is dq and all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))
    assert (p.select(axis, 1) == 7).all() and (p[..., D] == 7).all()
