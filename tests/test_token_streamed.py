"""GPU: the token-side kernels of large calls, whose outputs or inputs pass 128
MiB and are stored or read as streamed data, and the embedding's long chunks,
against float64.

Tolerances as in ``test_embed`` and ``test_distill``, e = 2^-24: a token's sum
of n rows within (n + 2) e of its terms' sizes; probabilities within E = (3 R +
24 + V / 256) e relative, R the range of the logits over tau.
"""

import numpy as np
import pytest

from kan_testutil import ensure_built

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    yield torch, F
    torch.cuda.empty_cache()


def _gen(torch, seed):
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(seed)
    return gen


@pytest.mark.parametrize("N,D,table,row", [(33000, 2048, "bf16", "bf16"), (16500, 2050, "f32", "f32"),
                                           (16500, 2050, "bf16", "f32"), (70001, 999, "f32", "bf16")])
def test_lookup_of_large_outputs(env, N, D, table, row):
    """One product, rounded once: the same bits as in torch's elementwise operations."""
    torch, F = env
    print("lookup", N, D, table, row, flush=True)
    dts = dict(f32=torch.float32, bf16=torch.bfloat16)
    gen = _gen(torch, N)
    E = torch.randn(5003, D, device="cuda:0", generator=gen).to(dts[table])
    ids = torch.randint(-1, 5004, (N,), device="cuda:0", generator=gen)
    y = F.kan_embed_forward(ids, E, 1.75, row_dtype=dts[row])
    assert y.numel() * y.element_size() >= 1 << 27
    inside = (ids >= 0) & (ids < 5003)
    want = torch.where(inside[:, None], E[ids.clamp(0, 5002)].float() * 1.75, 0.0).to(dts[row])
    assert torch.equal(y, want)


@pytest.mark.parametrize("N,V,D,row", [(262144 + 37, 5003, 100, "f32"), (262144, 70000, 512, "bf16"),
                                       (33000, 3001, 2050, "f32")])
def test_gradient_in_long_chunks(env, N, V, D, row):
    """N / 64 * ceil(D / 256) >= 4096: chunks of 64 rows, a token with half of all rows among them."""
    torch, F = env
    print("gradient", N, V, D, row, flush=True)
    assert N // 64 * ((D + 255) // 256) >= 4096
    gen = _gen(torch, V)
    ids = ((V + 1.0) ** torch.rand(N, device="cuda:0", generator=gen).double()).long().sub_(1).clamp_(0, V - 1)
    ids[torch.rand(N, device="cuda:0", generator=gen) < 0.4] = V // 2
    ids[::17] = -1
    dy = torch.randn(N, D, device="cuda:0", generator=gen).to(torch.bfloat16 if row == "bf16" else torch.float32)
    dE = F.kan_embed_backward(ids, dy, V, 0.5, out=torch.full((V, D), float("nan"), device="cuda:0"))
    assert torch.equal(dE, F.kan_embed_backward(ids, dy, V, 0.5))
    keep = ids >= 0
    want, size = torch.zeros(2, V, D, dtype=torch.float64, device="cuda:0")
    want.index_add_(0, ids[keep], dy[keep].double() * 0.5)
    size.index_add_(0, ids[keep], dy[keep].double().abs() * 0.5)
    n = torch.bincount(ids[keep], minlength=V)[:, None]
    assert bool(((dE.double() - want).abs() <= (n + 2) * EPS * size).all())


@pytest.mark.parametrize("N,V,K,dtype", [(512, 70001, 16, "f32"), (2100, 20003, 16, "f32"), (9000, 4001, 16, "f32"),
                                         (600, 60001, 300, "f32"), (1100, 70003, 64, "bf16"), (20000, 4000, 8, "bf16")])
def test_distillation_of_large_logits(env, N, V, K, dtype):
    torch, F = env
    print("distillation", N, V, K, dtype, flush=True)
    gen = _gen(torch, V)
    dt, tau = torch.bfloat16 if dtype == "bf16" else torch.float32, 2.0
    z = (torch.randn(N, V, device="cuda:0", generator=gen) * 3).to(dt)
    assert z.numel() * z.element_size() >= 1 << 27
    ids = torch.rand(N, V, device="cuda:0", generator=gen).topk(K, 1).indices
    t = torch.randn(N, K, device="cuda:0", generator=gen) * 2
    w = torch.rand(N, device="cuda:0", generator=gen) + 0.5
    dloss = torch.rand(N, device="cuda:0", generator=gen) + 0.5
    loss, lse = F.kan_distill_forward(z, ids, t, tau, weight=w)
    dz = F.kan_distill_backward(z, ids, t, lse, dloss, tau, weight=w, grad_dtype=dt)
    loss2, dz2 = F.kan_distill_step(z, ids, t, tau, weight=w, grad_dtype=dt)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse), F.kan_distill_forward(z, ids, t, tau, weight=w)))
    zd, td, wd = z.double() / tau, t.double() / tau, w.double()
    R = min(88.0, max(float(zd.max() - zd.min()), float(td.max() - td.min())) + np.log(V))
    E = (3 * R + 24 + V / 256) * EPS
    want_lse = torch.logsumexp(zd, 1)
    p = torch.softmax(td, 1)
    want = wd * tau * tau * (p * (torch.log_softmax(td, 1) - zd.gather(1, ids) + want_lse[:, None])).sum(1)
    for got in (loss, loss2):
        assert bool(((got.double() - want).abs() <= E * wd * tau * tau * (R + 1) * 2).all())
    most = float(zd.abs().max())
    assert bool(((lse.double() - want_lse).abs() <= 2 * EPS * (want_lse.abs() + most + 1) + E).all())
    q = zd.sub_(want_lse[:, None]).exp_()
    at = torch.zeros_like(q).scatter_(1, ids, 1.0).add_(q)
    q.scatter_add_(1, ids, -p)
    dE = E + 2 * EPS * (float(want_lse.abs().max()) + most)
    for got, scale in ((dz, wd * tau * dloss.double()), (dz2, wd * tau)):
        err = (got.double() / scale[:, None]).sub_(q).abs_()
        if dtype == "bf16":
            err.sub_(q.abs(), alpha=2.0 ** -8 + EPS)
        assert bool((err <= at * (dE * 1.1) + 1e-37).all())
