"""GPU: the delta rule's and the join's modules through autograd, and a model over
tokens that runs them together with the other operators."""

import os
import sys

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import delta as O

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
    return None if t is None else t.detach().double().cpu().numpy()


def test_delta_module_gradients(env):
    """Both outputs, pulled through the layers' own backward from the oracle's gradients
    (1e-5: the backward's tolerance of two chunks, through a layer)."""
    torch, kan, _ = env
    torch.manual_seed(1)
    m = kan.KANDeltaRule(10, 4, 8, 12, key_heads=2, grid_size=5, grid_range=(-3.0, 3.0), device="cuda:0")
    x = torch.randn(2, 90, 10, device="cuda:0", requires_grad=True)
    h0 = torch.randn(2, 4, 8, 12, device="cuda:0", requires_grad=True)
    lengths = torch.tensor([90, 17], dtype=torch.int32, device="cuda:0")
    y, hT = m(x, h0, lengths)
    assert y.shape == (2, 90, 48) and hT.shape == h0.shape
    dy, dh = torch.randn_like(y), torch.randn_like(hT)
    torch.autograd.backward([y, hT], [dy, dh])
    x2 = x.detach().clone().requires_grad_()
    p, (g, beta) = m.layer(x2), m._gates(x2)
    q, k, v = kan.DeltaFunction._slices(p, 2, 8, 4, 12)
    dq, dk, dv, dg, db, dh0 = O.delta_backward(*map(_np, (q, k, v, g, beta)), _np(dy).reshape(2, 90, 4, 12), _np(h0),
                                               lengths.tolist(), _np(dh), unit=True)
    assert np.abs(_np(h0.grad) - dh0).max() <= 1e-5 * np.abs(dh0).max()
    got = {n: t.grad.clone() for n, t in m.named_parameters()}
    m.zero_grad()
    dp = np.concatenate([t.reshape(2, 90, -1) for t in (dq, dk, dv)], -1)
    torch.autograd.backward([p, g, beta], [torch.tensor(t, device="cuda:0", dtype=torch.float32) for t in (dp, dg, db)])
    assert float((x.grad - x2.grad).abs().max()) <= 1e-5 * float(x2.grad.abs().max())
    for n, t in m.named_parameters():
        assert float((got[n] - t.grad).abs().max()) <= 1e-5 * float(t.grad.abs().max()), n


def test_delta_module_uses_only_what_is_asked_for(env):
    torch, kan, _ = env
    m = kan.KANDeltaRule(8, 2, 4, 4, device="cuda:0")
    x = torch.rand(3, 5, 8, device="cuda:0", requires_grad=True)
    m(x)[1].sum().backward()                     # only the last state
    assert bool(x.grad.any())
    x.grad = None
    m(x)[0].sum().backward()                     # only the rows, whose gradient is an expanded one
    assert bool(x.grad.any())
    y, hT = m(x, torch.zeros(1, 2, 4, 4, device="cuda:0").expand(3, 2, 4, 4))
    assert torch.equal(y, m(x)[0])
    with pytest.raises(ValueError):
        kan.KANDeltaRule(8, 3, 4, 4, key_heads=2)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pre", [True, False])
def test_join_module_gradients(env, dtype, pre):
    """Against the oracle at the stored rows; 2e-5 of the largest value, and bf16's rounding."""
    torch, kan, _ = env
    torch.manual_seed(2)
    dt = getattr(torch, dtype)
    m = kan.KANJoin(40, pre=pre, scale=0.5, device="cuda:0")
    with torch.no_grad():
        for w in m.parameters():
            w.add_(0.3 * torch.randn_like(w))
    h, r, gate = (torch.randn(3, 7, 40, device="cuda:0").to(dt).requires_grad_() for _ in range(3))
    out = m(h, r, gate)
    y, x = out if pre else (out, None)
    dy, dx = torch.randn_like(y), None if x is None else torch.randn_like(x)
    torch.autograd.backward([y] + [x] * pre, [dy] + [dx] * pre)
    flat = [None if t is None else _np(t).reshape(-1, 40) for t in (h, r, gate, y, dy, dx)]
    wp, wq = _np(m.w_post), _np(m.w_pre)
    wy, wx, n1, n2 = O.join_forward(*flat[:3], wp, wq, True, pre, scale=0.5)
    half = 2.0 ** -8 if dtype == "bfloat16" else 0

    def close(got, want, half=half):
        want = want.reshape(tuple(got.shape))
        assert (np.abs(_np(got) - want) <= 2e-5 * np.abs(want).max() + half * np.abs(want)).all()
    close(y, wy)
    if pre:
        close(x, wx)
    want = O.join_backward(flat[0], flat[3], n1, n2, flat[4], flat[5], flat[2], wp, wq, scale=0.5)
    for t, w in zip((h, r, gate), want):
        assert t.grad.dtype == t.dtype
        close(t.grad, w)
    close(m.w_post.grad, want[3], 0)
    if pre:
        close(m.w_pre.grad, want[4], 0)


def test_join_module_inputs(env):
    """Absent and strided inputs, unused outputs, shapes that do not belong together."""
    torch, kan, _ = env
    m = kan.KANJoin(6, device="cuda:0")
    h = torch.randn(5, 4, 6, device="cuda:0", requires_grad=True)
    y, x = m(h.transpose(0, 1))
    assert y.shape == x.shape == (4, 5, 6)
    x.sum().backward()                                # only the second norm
    assert bool(m.w_pre.grad.any()) and bool(h.grad.isfinite().all())
    m.zero_grad()
    m(h)[0].sum().backward()                          # only the sum
    assert m.w_pre.grad is None and bool(m.w_post.grad.any())
    wide = torch.randn(5, 4, 12, device="cuda:0")
    assert torch.equal(m(wide[..., 6:], wide[..., :6])[0],
                       m(wide[..., 6:].contiguous(), wide[..., :6].contiguous())[0])
    with pytest.raises(ValueError):
        m(h, h[:1])
    with pytest.raises(ValueError):
        kan.KANJoin(6, activation="relu")


def test_second_derivatives_are_refused(env):
    torch, kan, _ = env
    p = torch.randn(2, 9, 2 * 4 + 5, device="cuda:0", requires_grad=True)
    g, beta = -torch.rand(2, 9, 1, device="cuda:0"), torch.rand(2, 9, 1, device="cuda:0")
    h = torch.randn(3, 6, device="cuda:0", requires_grad=True)
    m = kan.KANJoin(6, device="cuda:0")
    for out, x in (((kan.DeltaFunction.apply(p, g, beta, None, None, (1, 4, 1, 5))[0] ** 2).sum(), p),
                   ((m(h)[1] ** 2 * torch.arange(6, device="cuda:0")).sum(), h)):
        (first,) = torch.autograd.grad(out, x, create_graph=True)
        assert bool(torch.isfinite(first).all()) and bool(first.any())
        with pytest.raises(RuntimeError, match="once_differentiable"):
            first.sum().backward()


@pytest.mark.parametrize("autograd", [False, True])
def test_example_runs(env, autograd):
    torch, kan, ex = env
    r = ex.main(steps=3, autograd=autograd, quiet=True, mixer="delta")
    assert all(np.isfinite(r["losses"]))
    out = r["generated"]
    assert out.shape == (4, 13) and int(out.min()) >= 0 and int(out.max()) < 200
    assert not r["state"][[1, 3, 4, 6]].any() and bool(r["state"][[0, 2, 5, 7]].any(-1).any(-1).all())


class _Plain:
    """The mixer and the join in float64 elementwise operations that autograd differentiates."""

    @staticmethod
    def mix(torch, m, x, lengths):
        Hk, Dk, Hv, Dv = m._shape()
        p = m.layer(x).double()
        g, beta = (t.double() for t in m._gates(x))
        n = Hk * Dk
        q, k = (t.unflatten(-1, (Hk, Dk)).repeat_interleave(Hv // Hk, 2) for t in (p[..., :n], p[..., n:2 * n]))
        q, k = (t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
        v, rows = p[..., 2 * n:].unflatten(-1, (Hv, Dv)), []
        S = torch.zeros(len(x), Hv, Dk, Dv, dtype=torch.float64, device=x.device)
        for t in range(x.shape[1]):
            inside = (t < lengths)[:, None, None]
            D = g[:, t].exp()[..., None, None] * S
            u = beta[:, t, :, None] * (v[:, t] - (D * k[:, t, :, :, None]).sum(2))
            new = D + k[:, t, :, :, None] * u[:, :, None, :]
            rows.append(torch.where(inside, Dk ** -0.5 * (new * q[:, t, :, :, None]).sum(2), 0.0))
            S = torch.where(inside[..., None], new, S)
        return torch.stack(rows, 1).flatten(2).float()

    @staticmethod
    def join(m, h, r):
        h, r = h.double(), r.double()
        y = r + m.w_post * h / (h.pow(2).mean(-1, keepdim=True) + m.eps).sqrt()
        return y.float(), (m.w_pre * y / (y.pow(2).mean(-1, keepdim=True) + m.eps).sqrt()).float()


def test_model_gradients_equal_those_with_plain_operators(env):
    """Every parameter's gradient of a model of embedding, delta rule, join, layers and distillation
    against the same model around plain float64 operators (float32 through three spline layers, each 1e-5
    of its range, and the operators' own 1e-5: 1e-4 of the gradient's norm)."""
    torch, kan, ex = env
    torch.manual_seed(3)
    model = ex.DeltaTokenModel(50, 32, device="cuda:0")
    ids = torch.randint(0, 50, (3, 80), device="cuda:0")
    lengths = torch.tensor([80, 33, 65], dtype=torch.int32, device="cuda:0")
    top = torch.randint(0, 50, (3, 80, 5), device="cuda:0")
    t, w = torch.randn(3, 80, 5, device="cuda:0"), (torch.arange(80, device="cuda:0")[None] < lengths[:, None]).float()
    z = model(ids, lengths)
    kan.KANDistillLoss(reduction="sum")(z, top, t, w).backward()
    got = {n: p.grad.clone() for n, p in model.named_parameters()}
    model.zero_grad()
    x = model.embed(ids)
    y, rows = _Plain.join(model.join, _Plain.mix(torch, model.mix, x, lengths), x)
    z2 = model.head(y + model.channels(rows))
    assert float((z - z2).detach().abs().max()) <= 5e-5 * float(z2.detach().abs().max())
    kan.KANDistillLoss(reduction="sum")(z2, top, t, w).backward()
    for n, p in model.named_parameters():
        assert bool(p.grad.any()), n
        assert float((got[n] - p.grad).norm()) <= 1e-4 * float(p.grad.norm()), n


def test_token_by_token_equals_the_sequence(env):
    """Logits of the step and of the whole sequence: the same sums in another
    order, float32 through three spline layers (each 1e-5 of its range)."""
    torch, kan, ex = env
    torch.manual_seed(4)
    model = ex.DeltaTokenModel(50, 32, device="cuda:0")
    ids = torch.randint(0, 50, (3, 70), device="cuda:0")
    with torch.no_grad():
        z = model(ids)
        state = model.state(5)
        slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda:0")
        rows = torch.stack([model.step(ids[:, t], state, slots) for t in range(70)], 1)
    assert float((z - rows).abs().max()) <= 5e-5 * float(z.abs().max())
    assert not state[[0, 3]].any()
