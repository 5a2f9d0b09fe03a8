"""GPU: distillation from a teacher's top logits against the float64 oracle.

Tolerances, with e = 2^-24: an exponent x = (z - m) / tau rounds to |x| e in its
difference, product and conversion to base 2 (3 |x| e in all) and exp2 adds an
ulp or two, so a probability is within E = (3 R + 8) e relative, R the range of
z / tau and t / tau that still counts (at most 88: smaller terms vanish).  A sum
of V terms, added in float32 by many threads and then across them, is within
(V / 256 + 16) e relative.  The loss is a mean of terms of size R; the gradient
of q - p with both within that.  bf16 gradients round once more, 2^-8 relative.
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


def _np(t):
    if t is None:
        return None
    return t.detach().cpu().numpy() if not t.dtype.is_floating_point else t.detach().float().cpu().numpy()


def _case(torch, N, V, K, dtype, seed, pad=0, idt=None, tdt=None):
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(seed)
    z = torch.randn(N, V + pad, device="cuda:0", generator=gen) * 3
    z = z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)[:, :V]
    ids = torch.randint(-1, V + 1, (N, K), device="cuda:0", generator=gen)
    ids[:, 0] = torch.randint(0, V, (N,), device="cuda:0", generator=gen)
    t = torch.randn(N, K, device="cuda:0", generator=gen) * 2
    w = torch.rand(N, device="cuda:0", generator=gen) + 0.5
    return z, ids.to(idt or torch.int64), t.to(tdt or torch.float32), w


def _tol(z, t, V, tau):
    z = z[np.isfinite(z)] / tau
    t = t[np.isfinite(t)] / tau
    R = min(88.0, max(np.ptp(z) if z.size else 0, np.ptp(t) if t.size else 0) + np.log(V))
    return ((3 * R + 8) + V / 256 + 16) * EPS, R


def _check(torch, F, z, ids, t, w, tau, grad, weight=True):
    nz, ni, nt, nw = _np(z), _np(ids), _np(t), _np(w) if weight else None
    N, V = z.shape
    wt = w if weight else None
    dl = torch.rand(N, device="cuda:0") + 0.5
    loss, lse = F.kan_distill_forward(z, ids, t, tau, weight=wt)
    wl, wlse, wd = O.distill(nz, ni, nt, tau, nw, _np(dl))
    E, R = _tol(nz, nt, V, tau)
    scale = (1.0 if nw is None else np.abs(nw)) * tau * tau
    got = loss.double().cpu().numpy()
    fin = np.isfinite(wl)
    assert (got[~fin] == wl[~fin]).all()
    assert (np.abs(got - wl)[fin] <= (E * scale * (R + 1) * 2 * np.ones(N))[fin]).all()
    g, finite = lse.double().cpu().numpy(), np.isfinite(wlse)
    assert (g[~finite] == wlse[~finite]).all()
    assert (np.abs(g - wlse)[finite] <= 2 * EPS * (np.abs(wlse[finite]) + np.abs(nz[np.isfinite(nz)]).max(initial=0) / tau
                                                   + 1) + E).all()
    gt = torch.bfloat16 if grad == "bf16" else torch.float32
    dz = F.kan_distill_backward(z, ids, t, lse, dl, tau, weight=wt, grad_dtype=gt)
    f = ((1.0 if nw is None else np.abs(nw)) * tau * _np(dl))[:, None]
    q = np.exp(np.minimum(nz.astype(np.float64) / tau - np.where(finite, wlse, 0)[:, None], 0))
    dE = E + 2 * EPS * (np.abs(wlse[finite]).max(initial=0) + np.abs(nz[np.isfinite(nz)]).max(initial=0) / tau)
    at = np.zeros((N, V))
    for b in range(N):
        for i in ni[b]:
            if 0 <= i < V:
                at[b, i] = 1.0
    tol = f * dE * (q + at) * 1.1 + (2.0 ** -8 + EPS) * np.abs(wd) * (grad == "bf16") + 1e-38
    assert (np.abs(dz.double().cpu().numpy() - wd) <= tol).all()
    out = torch.full((N, V), float("nan"), dtype=gt, device="cuda:0")
    loss2, dz2 = F.kan_distill_step(z, ids, t, tau, weight=wt, out=out)
    assert (np.abs(loss2.double().cpu().numpy() - wl)[fin] <= (E * scale * (R + 1) * 2 * np.ones(N))[fin]).all()
    dl1 = _np(dl)[:, None]
    assert (np.abs(dz2.double().cpu().numpy() - wd / dl1) <= tol / dl1).all()
    again = F.kan_distill_step(z, ids, t, tau, weight=wt, grad_dtype=gt)
    assert torch.equal(loss2, again[0]) and torch.equal(dz2, again[1])


@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 1), (2, 5, 7), (5, 64, 3), (4, 255, 16), (3, 1000, 64),
                                   (7, 1025, 33), (2, 4096, 256), (3, 8191, 5), (2, 8192, 1024), (1, 32003, 16),
                                   (2, 70001, 20), (1, 131072, 8), (2, 140001, 4), (300, 517, 9), (2100, 40, 4)])
@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_against_the_oracle(env, N, V, K, dtype, grad):
    torch, F = env
    tau = (1.0, 2.0, 0.5)[(N + V) % 3]
    idt = torch.int32 if V % 2 else torch.int64
    z, ids, t, w = _case(torch, N, V, K, dtype, N + V + K, pad=(V % 3) * 5, idt=idt,
                         tdt=torch.bfloat16 if K % 2 else torch.float32)
    _check(torch, F, z, ids, t, w, tau, grad, weight=N != 3)


@pytest.mark.parametrize("V", [40, 3001, 70003])
def test_masked_logits(env, V):
    """-inf and the type's lowest value among the student's logits; a teacher
    that wants a masked token makes the loss infinite and the gradient stay
    finite, and rows of only -inf, or of only the lowest value, are defined."""
    torch, F = env
    z, ids, t, w = _case(torch, 6, V, 4, "f32", V)
    ids = torch.arange(4, device="cuda:0").repeat(6, 1)
    z[0, 5:] = -float("inf")
    z[1, 5:] = torch.finfo(torch.float32).min
    z[2] = -float("inf")
    z[3] = torch.finfo(torch.float32).min
    z[4, 1] = -float("inf")
    t[5, 2:] = -float("inf")
    loss, lse = F.kan_distill_forward(z, ids, t, 1.0)
    wl, wlse, wd = O.distill(_np(z), _np(ids), _np(t), 1.0)
    E = _tol(_np(z[5:]), _np(t[5:, :2]), V, 1.0)[0] * 80
    for b in (0, 1, 3, 5):
        assert abs(float(loss[b]) - wl[b]) <= E
    assert float(loss[2]) == 0 and float(lse[2]) == -float("inf") and float(loss[4]) == float("inf")
    for dz in (F.kan_distill_backward(z, ids, t, lse, torch.ones(6, device="cuda:0")), F.kan_distill_step(z, ids, t)[1]):
        got = dz.double().cpu().numpy()
        rows = [0, 1, 2, 4, 5]                    # row 3: z / tau - lse has no digits left at 3e38
        assert np.abs(got[rows] - wd[rows]).max() <= E
        assert not got[2].any() and not got[0, 5:].any()
    assert np.abs(F.kan_distill_step(z, ids, t)[1][3].double().cpu().numpy() - wd[3]).max() <= E


@pytest.mark.parametrize("V,N", [(50, 4), (9000, 4), (9000, 600), (70003, 4)])
def test_rows_without_weight_are_not_read(env, V, N):
    """Junk in a row of weight 0 reaches neither its loss nor its gradient (its
    lse is that of its logits all the same)."""
    torch, F = env
    z, ids, t, w = _case(torch, N, V, 5, "f32", 3)
    w[1] = 0
    z[1], t[1] = float("nan"), float("inf")
    loss, lse = F.kan_distill_forward(z, ids, t, 2.0, weight=w)
    dz = F.kan_distill_backward(z, ids, t, lse, torch.ones(N, device="cuda:0"), 2.0, weight=w)
    l2, dz2 = F.kan_distill_step(z, ids, t, 2.0, weight=w)
    for a in (loss[1], dz[1], l2[1], dz2[1]):
        assert not a.any()
    assert all(bool(torch.isfinite(a).all()) for a in (loss, dz, l2, dz2))
    lse[1] = 0
    assert bool(torch.isfinite(lse).all())
    z[1] = 1.5
    lse = F.kan_distill_forward(z, ids, t, 2.0, weight=w)[1]
    assert abs(float(lse[1]) - (0.75 + np.log(V))) <= 1e-5


@pytest.mark.parametrize("V,N", [(50, 3), (9000, 3), (9000, 600), (140001, 3)])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_nan_and_inf_show(env, V, N, bad):
    """A NaN or +inf among a row's logits makes that row's loss NaN, and only that row's."""
    torch, F = env
    z, ids, t, w = _case(torch, N, V, 5, "f32", 4)
    z[1, V // 2] = float(bad)
    for loss in (F.kan_distill_forward(z, ids, t)[0], F.kan_distill_step(z, ids, t)[0]):
        assert bool(torch.isnan(loss[1])) and bool(torch.isfinite(loss[[0, 2]]).all())


def test_absent_teachers(env):
    torch, F = env
    z, ids, t, w = _case(torch, 5, 300, 6, "f32", 5)
    ids[0], ids[1] = -1, 300
    t[2] = -float("inf")
    t[0, 3], t[1, 2] = float("nan"), float("inf")      # of absent entries: ignored
    ids[3] = 7                                          # one token, six times
    ids[4, 1:] = (1 << 33) + 5                          # past 32 bits: absent
    loss, lse = F.kan_distill_forward(z, ids, t)
    dz = F.kan_distill_step(z, ids, t)[1]
    assert not loss[:3].any() and not dz[:3].any() and bool(torch.isfinite(lse).all())
    wl, _, wd = O.distill(_np(z), _np(ids), _np(t), 1.0)
    E = _tol(_np(z), _np(t[3:]), 300, 1.0)[0] * 40
    assert np.abs(loss.double().cpu().numpy() - wl).max() <= E and np.abs(dz.double().cpu().numpy() - wd).max() <= E


def test_gradient_by_differences(env):
    """The forward at z moved by +-h along a direction (h = 1e-2: h^2 / 6 of the
    third derivative, and 2^-24 of the loss over 2h) within 1e-3 of the terms."""
    torch, F = env
    z, ids, t, w = _case(torch, 4, 60, 6, "f32", 6)
    loss, lse = F.kan_distill_forward(z, ids, t, 2.0, weight=w)
    dz = F.kan_distill_backward(z, ids, t, lse, torch.ones(4, device="cuda:0"), 2.0, weight=w)
    way = torch.randn_like(z)
    hi, lo = (F.kan_distill_forward(z + s * 1e-2 * way, ids, t, 2.0, weight=w)[0].double() for s in (1, -1))
    want = (hi - lo) / 2e-2
    got = (dz.double() * way).sum(1)
    assert float((got - want).abs().max()) <= 1e-3 * float((dz * way).abs().sum(1).max())


def test_a_gradient_row_sums_to_zero_and_rows_are_untouched_outside(env):
    """q and p both sum to 1; a strided dz leaves what lies between its rows."""
    torch, F = env
    z, ids, t, w = _case(torch, 9, 1003, 12, "bf16", 7)
    wide = torch.full((9, 1010), 5.0, device="cuda:0")
    F.kan_distill_step(z, ids, t, out=wide[:, :1003])
    assert (wide[:, 1003:] == 5).all()
    assert float(wide[:, :1003].double().sum(1).abs().max()) <= 40 * EPS * 30


@pytest.mark.parametrize("V,dtype", [(20485, "f32"), (40965, "bf16"), (20485, "bf16"), (122885, "f32"), (122885, "bf16")])
@pytest.mark.parametrize("N", [2, 40, 70])
def test_a_part_that_ends_in_the_next_ones_head(env, V, dtype, N):
    """Vocabularies a few elements past a whole number of a row's parts: with rows
    that start inside a cache line the last part is empty, and the row's tail,
    with the teacher's entries in it, belongs to the part before it."""
    torch, F = env
    z, ids, t, w = _case(torch, N, V, 12, dtype, V + N)
    ids = torch.arange(V - 12, V, device="cuda:0").repeat(N, 1)
    _check(torch, F, z, ids, t, w, 1.0, dtype)


def test_rows_cut_over_blocks(env):
    """Few rows of a large vocabulary: masks, empty rows and weights as elsewhere."""
    test_masked_logits(env, 131075)
    test_rows_without_weight_are_not_read(env, 131075, 4)
    for bad in ("nan", "inf"):
        test_nan_and_inf_show(env, 131075, 3, bad)


def test_empty(env):
    torch, F = env
    z, ids, t = (torch.empty(0, n, device="cuda:0") for n in (10, 3, 3))
    ids = ids.long()
    loss, lse = F.kan_distill_forward(z, ids, t)
    assert loss.shape == lse.shape == (0,)
    assert F.kan_distill_step(z, ids, t)[1].shape == (0, 10)
    assert F.kan_distill_backward(z, ids, t, lse, lse).shape == (0, 10)


def test_refusals(env):
    torch, F = env
    from kolmogorov_arnold_network_amd import _lib as L
    z, ids, t, w = _case(torch, 4, 20, 3, "f32", 8)
    for bad in (dict(z=z.half()), dict(z=z.cpu()), dict(z=z[0]), dict(z=z.t()), dict(ids=ids[:3]),
                dict(ids=ids.float()), dict(t=t[:, :2]), dict(t=t.half()), dict(weight=w[:2]),
                dict(weight=w.double())):
        with pytest.raises(ValueError):
            F.kan_distill_forward(**dict(dict(z=z, ids=ids, t=t), **bad))
        with pytest.raises(ValueError):
            F.kan_distill_step(**dict(dict(z=z, ids=ids, t=t), **bad))
    for bad in (dict(lse=w[:3]), dict(dloss=w.double()), dict(out=torch.empty(4, 19, device="cuda:0"))):
        with pytest.raises(ValueError):
            F.kan_distill_backward(**dict(dict(z=z, ids=ids, t=t, lse=w, dloss=w), **bad))
    for tau in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(L.KanError) as e:
            F.kan_distill_forward(z, ids, t, tau)
        assert e.value.status == L.KAN_ERR_UNSUPPORTED
    many = torch.zeros(4, 1025, dtype=torch.int64, device="cuda:0")
    with pytest.raises(L.KanError) as e:                # more teacher logits than a row may have
        F.kan_distill_forward(z, many, many.float())
    assert e.value.status == L.KAN_ERR_SHAPE
    with pytest.raises(L.KanError) as e:
        F.kan_distill_step(z, ids, t, out=z)
    assert e.value.status == L.KAN_ERR_ALIAS
