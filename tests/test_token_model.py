"""GPU: the token-side modules through autograd, and the example that runs them together."""

import os
import sys

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import token as O

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import kolmogorov_arnold_network_amd as kan
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import token_distillation
    return torch, kan, token_distillation


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("table,row", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float32", "bfloat16")])
def test_embedding_module(env, table, row):
    """Sums of at most 12 rows of float32 (13 e), one more rounding where the
    table, and with it the gradient, is bf16 (2^-8)."""
    torch, kan, _ = env
    torch.manual_seed(0)
    m = kan.KANEmbedding(11, 24, scale=1.5, dtype=getattr(torch, table), row_dtype=getattr(torch, row), device="cuda:0")
    ids = torch.randint(-1, 11, (3, 20), device="cuda:0")
    y = m(ids)
    assert y.shape == (3, 20, 24) and y.dtype == getattr(torch, row)
    dy = torch.randn(3, 20, 24, device="cuda:0").to(y.dtype)
    y.backward(dy)
    assert m.table.grad.dtype == m.table.dtype
    flat, d = ids.flatten().cpu().numpy(), _np(dy).reshape(-1, 24)
    want = O.embed_backward(flat, d, 11, 1.5)
    tol = 2.0 ** -24 * 30 * O.embed_backward(flat, np.abs(d), 11, 1.5) + (
        2.0 ** -8 * np.abs(want) if table == "bfloat16" else 0)
    assert (np.abs(_np(m.table.grad) - want) <= tol).all()


def test_recurrence_module_gradients(env):
    """Through the layer, the recurrence and both outputs, against the oracle's
    gradients of the recurrence pulled through the layer's own backward."""
    torch, kan, _ = env
    torch.manual_seed(1)
    m = kan.KANRecurrence(10, 6, grid_size=5, grid_range=(-3.0, 3.0), device="cuda:0")
    x = torch.randn(2, 30, 10, device="cuda:0", requires_grad=True)
    h0 = torch.randn(2, 6, device="cuda:0", requires_grad=True)
    lengths = torch.tensor([30, 17], dtype=torch.int32, device="cuda:0")
    y, hT = m(x, h0, lengths)
    dy, dh = torch.randn_like(y), torch.randn_like(hT)
    torch.autograd.backward([y, hT], [dy, dh])
    p = m.layer(x.detach())
    q = _np(p)
    dx, dg, dh0 = O.recur_backward(q[..., :6], q[..., 6:], _np(dy), _np(h0), lengths.tolist(), _np(dh))
    assert np.abs(_np(h0.grad) - dh0).max() <= 1e-5 * np.abs(dh0).max()
    x2 = x.detach().clone().requires_grad_()
    m2 = m.layer
    m2.zero_grad()
    m2(x2).backward(torch.tensor(np.concatenate([dx, dg], -1), device="cuda:0", dtype=torch.float32))
    assert float((x.grad - x2.grad).abs().max()) <= 1e-5 * float(x2.grad.abs().max())


def test_recurrence_module_uses_only_what_is_asked_for(env):
    torch, kan, _ = env
    m = kan.KANRecurrence(8, 4, device="cuda:0")
    x = torch.rand(3, 5, 8, device="cuda:0", requires_grad=True)
    m(x)[1].sum().backward()                     # only the last state
    assert bool(x.grad.any())
    x.grad = None
    m(x)[0].sum().backward()                     # only the rows
    assert bool(x.grad.any())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_distillation_module(env, dtype):
    """The loss through autograd equals the one-call step, and the weights' rows
    count as they should (same kernels: the rounding of two exponentials)."""
    torch, kan, _ = env
    torch.manual_seed(2)
    z = (torch.randn(2, 5, 300, device="cuda:0") * 2).to(getattr(torch, dtype)).requires_grad_()
    ids = torch.randint(0, 300, (2, 5, 7), device="cuda:0")
    t = torch.randn(2, 5, 7, device="cuda:0")
    w = torch.rand(2, 5, device="cuda:0")
    w[0, 2] = 0
    loss = kan.KANDistillLoss(2.0)(z, ids, t, w)
    loss.backward()
    rows, dz = kan.kan_distill_step(z.detach().view(-1, 300), ids.view(-1, 7), t.view(-1, 7), 2.0, weight=w.view(-1) / 10)
    assert z.grad.dtype == z.dtype
    assert abs(float(loss.detach() - rows.sum())) <= 1e-5 * float(rows.abs().sum())
    tol = 1e-5 * dz.abs().max() + (2.0 ** -8 * dz.abs() if dtype == "bfloat16" else 0)
    assert bool(((z.grad.float().view(-1, 300) - dz).abs() <= tol).all()) and not z.grad[0, 2].any()
    none = kan.KANDistillLoss(2.0, reduction="none")(z, ids, t, w)
    assert none.shape == (2, 5) and abs(float((none.sum() - 10 * loss).detach())) <= 1e-4
    with pytest.raises(ValueError):
        kan.KANDistillLoss(2.0)(z, ids[:1], t, w)


@pytest.mark.parametrize("autograd", [False, True])
def test_example_learns_its_teacher(env, autograd):
    """A uniform student of 200 tokens loses about log 200 minus the teacher's
    entropy; sixty steps take off more than a third of what it starts with."""
    torch, kan, ex = env
    r = ex.main(steps=60, autograd=autograd, quiet=True)
    assert all(np.isfinite(r["losses"])) and r["losses"][-1] < 0.65 * r["losses"][0]
    out = r["generated"]
    assert out.shape == (4, 13) and int(out.min()) >= 0 and int(out.max()) < 200


def test_token_by_token_equals_the_sequence(env):
    """Logits of the step and of the whole sequence: the same sums in another
    order, float32 through three spline layers (each 1e-5 of its range)."""
    torch, kan, ex = env
    torch.manual_seed(3)
    model = ex.TokenModel(50, 32, device="cuda:0")
    ids = torch.randint(0, 50, (3, 20), device="cuda:0")
    with torch.no_grad():
        z = model(ids)
        state = torch.zeros(5, 32, device="cuda:0")
        slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda:0")
        rows = torch.stack([model.step(ids[:, t], state, slots) for t in range(20)], 1)
    assert float((z - rows).abs().max()) <= 5e-5 * float(z.abs().max())
    assert not state[[0, 3]].any()
