"""GPU: what the token-side modules have no gradient of is refused, not left out:
the distillation's teacher and weights, and second derivatives."""

import pytest

from kan_testutil import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import kolmogorov_arnold_network_amd as kan
    return torch, kan


def _case(torch):
    torch.manual_seed(0)
    z = torch.randn(4, 30, device="cuda:0", requires_grad=True)
    ids = torch.randint(0, 30, (4, 3), device="cuda:0")
    return z, ids, torch.randn(4, 3, device="cuda:0"), torch.rand(4, device="cuda:0")


@pytest.mark.parametrize("which", ["t", "weight"])
def test_distillation_refuses_gradients_that_it_does_not_have(env, which):
    torch, kan = env
    z, ids, t, w = _case(torch)
    loss = kan.KANDistillLoss(2.0)
    want = loss(z, ids, t, w).detach()
    (t if which == "t" else w).requires_grad_()
    with pytest.raises(ValueError):
        loss(z, ids, t, w)
    with torch.no_grad():                             # nothing to differentiate
        assert torch.equal(loss(z, ids, t, w), want)
    assert torch.equal(loss(z, ids, t.detach(), w.detach()).detach(), want)
    rows = kan.DistillFunction.apply(z, ids, t, 2.0, w)
    with pytest.raises(ValueError):
        rows.sum().backward()


def test_second_derivatives_are_refused(env):
    torch, kan = env
    z, ids, t, w = _case(torch)
    emb = kan.KANEmbedding(30, 6, device="cuda:0")
    p = torch.randn(2, 9, 8, device="cuda:0", requires_grad=True)
    for out, x in (((emb(ids) ** 2).sum(), emb.table),
                   ((kan.RecurFunction.apply(p, None, None)[0] ** 2).sum(), p),
                   ((kan.DistillFunction.apply(z, ids, t, 2.0, w) ** 2).sum(), z)):
        (first,) = torch.autograd.grad(out, x, create_graph=True)
        assert bool(torch.isfinite(first).all()) and bool(first.any())
        with pytest.raises(RuntimeError, match="once_differentiable"):
            first.sum().backward()
