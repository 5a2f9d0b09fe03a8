"""GPU: the token-side operators on arrays past 2^31 elements and 2^32 bytes.

Rows are independent, so the last rows of a large array are compared with the
same rows alone (another plan or alignment: the sums' rounding differs).
"""

import pytest

from kan_testutil import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    yield torch, F
    torch.cuda.empty_cache()


def test_embedding_table_past_32_bits(env):
    torch, F = env
    V, D = 600_000, 4096                            # 2.46e9 elements
    E = torch.empty(V, D, dtype=torch.bfloat16, device="cuda:0")
    last = torch.randn(1000, D, device="cuda:0").to(torch.bfloat16)
    E[-1000:] = last
    ids = torch.arange(V - 1000, V, device="cuda:0").repeat(3)
    assert torch.equal(F.kan_embed_forward(ids, E), last.repeat(3, 1))
    del E
    dy = torch.ones(3000, D, device="cuda:0")
    dE = F.kan_embed_backward(ids, dy, V)
    assert bool((dE[-1000:] == 3).all()) and not dE[-1001].any() and not dE[0].any()
    assert float(dE[300_000:300_100].abs().sum()) == 0


def test_recurrence_past_32_bits(env):
    """Few sequences (cut into segments) and a strided, packed input of 4.4e9 elements."""
    torch, F = env
    B, T, D = 2, 550_000, 2000
    p = torch.empty(B, T, 2 * D, dtype=torch.bfloat16, device="cuda:0")
    for b in range(B):
        p[b].normal_()
    p[..., D:].add_(2)
    y, hT = F.kan_recur_forward(p[..., :D], p[..., D:])
    # memories are a few hundred rows: the last ones alone, from a state of zero
    tail = p[1:, -6000:].contiguous()
    y2, h2 = F.kan_recur_forward(tail[..., :D], tail[..., D:])
    assert float((y[1, -1000:] - y2[0, -1000:]).abs().max()) <= 2e-6
    assert torch.equal(hT, y[:, -1]) and float((hT[1] - h2[0]).abs().max()) <= 2e-6
    dy = torch.zeros(B, T, D, device="cuda:0")
    dy[1, -6000:].normal_()
    dp = torch.empty_like(p)
    F.kan_recur_backward(p[..., :D], p[..., D:], y, dy, dx=dp[..., :D], dg=dp[..., D:])
    dx2, dg2, _ = F.kan_recur_backward(tail[..., :D], tail[..., D:], y[1:, -6000:].contiguous(),
                                       dy[1:, -6000:].contiguous(), grad_dtype=torch.bfloat16)
    for a, b in ((dp[1, -5000:, :D], dx2[0, -5000:]), (dp[1, -5000:, D:], dg2[0, -5000:])):
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())


def test_distillation_past_32_bits(env):
    torch, F = env
    N, V, K = 17_000, 131_075, 8                    # 2.2e9 logits
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda:0")
    for i in range(0, N, 1000):
        z[i:i + 1000].normal_()
    ids = torch.randint(0, V, (N, K), device="cuda:0")
    t = torch.randn(N, K, device="cuda:0")
    loss, dz = F.kan_distill_step(z, ids, t, 2.0, grad_dtype=torch.bfloat16)
    l2, dz2 = F.kan_distill_step(z[-7:].contiguous(), ids[-7:].contiguous(), t[-7:].contiguous(), 2.0,
                                 grad_dtype=torch.bfloat16)
    assert float((loss[-7:] - l2).abs().max()) <= 1e-5 * float(l2.abs().max())
    assert float((dz[-7:].float() - dz2.float()).abs().max()) <= 2.0 ** -7 * float(dz2.float().abs().max())
    fl, lse = F.kan_distill_forward(z, ids, t, 2.0)
    assert float((fl - loss).abs().max()) <= 1e-5 * float(loss.abs().max())
    F.kan_distill_backward(z, ids, t, lse, torch.ones(N, device="cuda:0"), 2.0, out=dz)
    assert float((dz[-7:].float() - dz2.float()).abs().max()) <= 2.0 ** -7 * float(dz2.float().abs().max())
