"""The recurrence's kernels by launch plan: each of 4, 8, 16 and 32 lanes along
the channels, whole sequences and segments, of several tiles and a remainder,
and large outputs that are stored as streamed data.

A CPU test pins the plans that the shapes take (``host/recur_plan_print.cpp``),
so that the shapes go on covering them.  On the GPU every value is compared
with the recurrence in float64, one row after the other.

Tolerances as in ``test_recur``, e = 2^-24: with |g| <= 4 a gate is within 24 e
and a memory M = min(T, 1 / min u) rows; a row within e (24 (max |x| + max |h|)
+ 8 sqrt(M) max |h|), a gradient within three times the same at its own scale,
and 2^-8 relative more where it is stored in bf16.
"""

import os
import subprocess

import pytest

from kan_testutil import ensure_built
from test_host_sanitize import CSRC, HERE, ROOT, _hipcc

EPS = 2.0 ** -24

# B, T, D, dtype, gradient's dtype, x and g in one array; then for forward and
# backward: channels of a lane, lanes, segments, rows of a segment and of a tile,
# streamed stores
SHAPES = [
    (96, 2100, 3, "f32", "f32", False, (1, 4, 2, 1536, 512, False), (1, 4, 2, 1536, 512, False)),
    (200, 1700, 3, "bf16", "bf16", True, (1, 4, 1, 1700, 512, False), (1, 4, 1, 1700, 512, False)),
    (200, 1700, 4, "bf16", "bf16", True, (4, 4, 1, 1700, 512, False), (4, 4, 1, 1700, 512, False)),
    (2, 1800, 2048, "f32", "f32", False, (4, 4, 1, 1800, 512, False), (4, 4, 1, 1800, 512, False)),
    (1, 66000, 130, "f32", "f32", True, (4, 8, 86, 768, 256, False), (4, 8, 86, 768, 256, False)),
    (1, 66000, 130, "bf16", "bf16", False, (4, 8, 86, 768, 256, False), (4, 8, 86, 768, 256, False)),
    (5, 900, 1024, "bf16", "bf16", False, (4, 8, 1, 900, 256, False), (4, 8, 1, 900, 256, False)),
    (1, 1100, 32, "f32", "f32", True, (4, 8, 1, 1100, 256, False), (4, 8, 1, 1100, 256, False)),
    (1, 66000, 33, "f32", "bf16", False, (4, 16, 172, 384, 128, False), (4, 16, 172, 384, 128, False)),
    (1, 66000, 64, "bf16", "f32", True, (4, 16, 172, 384, 128, False), (4, 16, 172, 384, 128, False)),
    (8, 450, 2048, "bf16", "bf16", True, (4, 16, 1, 450, 128, False), (4, 16, 1, 450, 128, False)),
    (24, 450, 770, "f32", "f32", False, (4, 16, 1, 450, 128, False), (4, 16, 1, 450, 128, False)),
    (1, 33000, 66, "bf16", "bf16", True, (4, 32, 172, 192, 64, False), (4, 32, 172, 192, 64, False)),
    (1, 33000, 100, "f32", "f32", False, (4, 32, 172, 192, 64, False), (4, 32, 172, 192, 64, False)),
    (24, 300, 770, "bf16", "f32", True, (4, 32, 1, 300, 64, False), (4, 16, 1, 300, 128, False)),
    (48, 200, 770, "f32", "f32", False, (4, 32, 1, 200, 64, False), (4, 32, 1, 200, 64, False)),
    # past 128 MiB, rows on cache lines
    (8, 2176, 2048, "f32", "f32", True, (4, 16, 1, 2176, 128, True), (4, 16, 1, 2176, 128, True)),
    (8, 2055, 2048, "bf16", "f32", False, (4, 16, 1, 2055, 128, True), (4, 16, 1, 2055, 128, True)),
    (8, 4103, 2048, "bf16", "bf16", True, (4, 16, 1, 4103, 128, True), (4, 16, 1, 4103, 128, True)),
    (8, 4352, 2048, "f32", "bf16", False, (4, 16, 1, 4352, 128, True), (4, 16, 1, 4352, 128, True)),
    (64, 520, 1024, "f32", "f32", False, (4, 32, 1, 520, 64, True), (4, 32, 1, 520, 64, True)),
    (1, 33000, 1024, "f32", "f32", False, (4, 32, 58, 576, 64, True), (4, 32, 58, 576, 64, True)),
    (1, 33000, 1024, "bf16", "f32", True, (4, 32, 58, 576, 64, True), (4, 32, 58, 576, 64, True)),
    (1, 66000, 1024, "bf16", "bf16", True, (4, 32, 61, 1088, 64, True), (4, 32, 61, 1088, 64, True)),
    (1, 66000, 1024, "f32", "bf16", True, (4, 32, 61, 1088, 64, True), (4, 32, 61, 1088, 64, True)),
]


def test_plans_of_the_shapes(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "recur_plan_print")
    cmd = [cc, "--offload-host-only", "-std=c++17", "-O1", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o", out,
           os.path.join(HERE, "host", "recur_plan_print.cpp"), os.path.join(CSRC, "kan_token_api.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    args = [str(v) for B, T, D, dt, gt, packed, _, _ in SHAPES
            for v in (B, T, D, int(dt == "bf16"), int(gt == "bf16"), int(packed))]
    res = subprocess.run([out] + args, capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stderr
    lines = [tuple(map(int, line.split())) for line in res.stdout.splitlines()]
    assert len(lines) == 2 * len(SHAPES)
    for (B, T, D, dt, gt, packed, fwd, bwd), *got in zip(SHAPES, lines[::2], lines[1::2]):
        for want, (vec, lanes, waves, segs, rows, tile, on_lines), size in zip(
                (fwd, bwd), got, (4, 2 if gt == "bf16" else 4)):
            streamed = bool(on_lines) and lanes in (16, 32) and B * T * D * size >= 1 << 27
            assert (vec, lanes, segs, rows, tile, streamed) == want, (B, T, D, dt, gt, packed)
            assert waves == 8 and (rows > 2 * tile)
    kinds = {(dt, s[1], s[2] > 1, s[5]) for _, _, _, dt, _, _, *both in SHAPES for s in both if s[0] == 4}
    assert {(dt, lanes, cut, False) for dt in ("f32", "bf16") for lanes in (8, 16, 32) for cut in (False, True)} <= kinds
    assert {(dt, 4, False, False) for dt in ("f32", "bf16")} <= kinds
    assert {(dt, lanes, False, True) for dt in ("f32",) for lanes in (16, 32)} <= kinds


def _reference(torch, x, g, h0, lengths, dy, dhT):
    """Rows, last state and gradients in float64, time first."""
    B, T, D = x.shape
    inside = (torch.arange(T, device=x.device)[:, None] < lengths.clamp(0, T)[None, :])[..., None]
    x, g, dy = (v.double().transpose(0, 1) for v in (x, g, dy))
    u, f = (torch.where(inside, torch.sigmoid(v), r).contiguous() for v, r in ((-g, 0.0), (g, 1.0)))
    dy = torch.where(inside, dy, 0.0)
    h = torch.empty(T + 1, B, D, dtype=torch.float64, device=x.device)
    c = torch.empty_like(h)
    h[0], c[T] = h0, dhT
    ux, fdy = u * x, f * dy
    for t in range(T):
        torch.addcmul(ux[t], f[t], h[t], out=h[t + 1])
    for t in range(T - 1, -1, -1):
        torch.addcmul(fdy[t], f[t], c[t + 1], out=c[t])
    delta = dy + c[1:]
    return dict(y=torch.where(inside, h[1:], 0.0), hT=h[T], dx=u * delta, dg=f * u * (h[:-1] - x) * delta, dh0=c[0],
                delta=float(delta.abs().max()), least=float(torch.where(inside, u, 1.0).min()))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%dx%d-%s-%s" % s[:5])
def test_every_plan_against_float64(shape):
    ensure_built()
    import torch
    from kolmogorov_arnold_network_amd import functional as F
    B, T, D, dt, gt, packed, _, _ = shape
    print("shape", shape[:6], flush=True)
    dt, gt = (torch.bfloat16 if v == "bf16" else torch.float32 for v in (dt, gt))
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(T + D)
    p = torch.randn(B, T, 2 * D, device="cuda:0", generator=gen)
    p[..., D:].add_(1.0).clamp_(-4, 4)
    p = p.to(dt)
    x, g = (p[..., :D], p[..., D:]) if packed else (p[..., :D].contiguous(), p[..., D:].contiguous())
    h0, dhT = (torch.randn(B, D, device="cuda:0", generator=gen) for _ in range(2))
    dy = torch.randn(B, T, D, device="cuda:0", generator=gen)
    lengths = torch.full((B,), T, dtype=torch.int32, device="cuda:0")
    if B > 1:
        lengths[1::2] = torch.randint(-1, T + 1, (B // 2,), device="cuda:0", generator=gen).int()
        lengths[-1] = 0
    else:
        lengths[0] = T - 39
    y = torch.full((B, T, D), float("nan"), device="cuda:0")
    y, hT = F.kan_recur_forward(x, g, h0, lengths, out=y)
    dp = torch.full((B, T, 2 * D) if packed else (2, B, T, D), float("nan"), dtype=gt, device="cuda:0")
    dx, dg = (dp[..., :D], dp[..., D:]) if packed else dp
    dh0 = F.kan_recur_backward(x, g, y, dy, h0, lengths, dhT, dx=dx, dg=dg)[2]
    again = F.kan_recur_forward(x, g, h0, lengths)
    assert torch.equal(y, again[0]) and torch.equal(hT, again[1])
    first = dx.clone(), dg.clone(), dh0
    more = F.kan_recur_backward(x, g, y, dy, h0, lengths, dhT, dx=dx, dg=dg)
    assert all(torch.equal(a, b) for a, b in zip(first, more))
    r = _reference(torch, x, g, h0, lengths, dy, dhT)
    size = float(x.float().abs().max()), max(float(r["y"].abs().max()), float(h0.abs().max()))
    root = 8 * min(T, 1.0 / r["least"]) ** 0.5
    near = EPS * (24 * sum(size) + root * size[1])
    del_near = 3 * EPS * (24 + root) * max(r["delta"], float(r["dh0"].abs().max()))
    half = 2.0 ** -8 if gt == torch.bfloat16 else 0.0
    for name, got, tol, rounded in (("y", y, near, 0.0), ("hT", hT, near, 0.0), ("dx", dx, del_near, half),
                                    ("dg", dg, del_near * sum(size), half), ("dh0", dh0, del_near, 0.0)):
        want = r[name] if got.dim() == 2 else r[name].transpose(0, 1)
        err = (got.double() - want).abs_().sub_(want.abs(), alpha=rounded)
        assert not torch.isnan(got).any() and float(err.max()) <= tol, (name, float(err.max()), tol)
