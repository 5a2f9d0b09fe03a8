"""GPU: the token-side operators on views of larger tensors: data that starts
off 16 bytes, in the wrappers, in the modules and in gradients that autograd
hands on; strided and expanded views in the modules.  Results equal those of
copies, bit for bit."""

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


def _off(torch, t, by=1):
    """The values of ``t`` in a tensor that starts ``by`` elements into its storage."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)[by:]
    out = flat.view(t.shape)
    out.copy_(t)
    assert out.is_contiguous() and out.data_ptr() % 16 != 0
    return out


def _same(torch, a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("idt", ["int32", "int64"])
def test_embedding(env, dtype, idt):
    torch, kan = env
    torch.manual_seed(0)
    dt = getattr(torch, dtype)
    ids = torch.randint(-1, 40, (33,), device="cuda:0").to(getattr(torch, idt))
    E, dy = torch.randn(40, 21, device="cuda:0").to(dt), torch.randn(33, 21, device="cuda:0").to(dt)
    want = kan.kan_embed_forward(ids, E), kan.kan_embed_backward(ids, dy, 40)
    assert _same(torch, want, (kan.kan_embed_forward(_off(torch, ids), E), kan.kan_embed_backward(_off(torch, ids), dy, 40)))
    assert torch.equal(want[0], kan.kan_embed_forward(ids, _off(torch, E)))
    assert torch.equal(want[1], kan.kan_embed_backward(ids, _off(torch, dy), 40))


def test_recurrence(env):
    torch, kan = env
    torch.manual_seed(1)
    x, g, dy = (torch.randn(3, 50, 7, device="cuda:0") for _ in range(3))
    h0, dhT = torch.randn(3, 7, device="cuda:0"), torch.randn(3, 7, device="cuda:0")
    lengths = torch.tensor([50, 0, 31], dtype=torch.int32, device="cuda:0")
    y, hT = kan.kan_recur_forward(x, g, h0, lengths)
    grads = kan.kan_recur_backward(x, g, y, dy, h0, lengths, dhT)
    o = lambda t: _off(torch, t)  # noqa: E731
    for a, b, n in ((x, h0, o(lengths)), (x, o(h0), lengths), (o(x), h0, lengths)):
        assert _same(torch, (y, hT), kan.kan_recur_forward(a, g, b, n))
    for k in range(5):
        args = [y, dy, h0, lengths, dhT]
        args[k] = o(args[k])
        assert _same(torch, grads, kan.kan_recur_backward(x, g, *args))
    state = torch.randn(9, 7, device="cuda:0")
    slots = torch.tensor([4, 2, 7], dtype=torch.int32, device="cuda:0")
    s1, s2 = state.clone(), state.clone()
    assert torch.equal(kan.kan_recur_step(x[:, 0], g[:, 0], s1, slots), kan.kan_recur_step(x[:, 0], g[:, 0], s2, o(slots)))
    assert torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_distillation(env, dtype):
    torch, kan = env
    torch.manual_seed(2)
    z = torch.randn(9, 301, device="cuda:0").to(getattr(torch, dtype))
    t, w, dl = torch.randn(9, 5, device="cuda:0"), torch.rand(9, device="cuda:0"), torch.rand(9, device="cuda:0")
    ids = torch.randint(0, 301, (9, 5), device="cuda:0")
    loss, lse = kan.kan_distill_forward(z, ids, t, 2.0, weight=w)
    dz = kan.kan_distill_backward(z, ids, t, lse, dl, 2.0, weight=w)
    step = kan.kan_distill_step(z, ids, t, 2.0, weight=w)
    o = lambda v: _off(torch, v)  # noqa: E731
    for a in ((o(ids), t, w), (ids, o(t), w), (ids, t, o(w))):
        assert _same(torch, (loss, lse), kan.kan_distill_forward(z, a[0], a[1], 2.0, weight=a[2]))
        assert torch.equal(dz, kan.kan_distill_backward(z, a[0], a[1], lse, dl, 2.0, weight=a[2]))
        assert _same(torch, step, kan.kan_distill_step(z, a[0], a[1], 2.0, weight=a[2]))
    assert torch.equal(dz, kan.kan_distill_backward(z, ids, t, o(lse), o(dl), 2.0, weight=w))


def test_modules_on_slices(env):
    """The next-token slices of a batch, a run of a state pool's slots."""
    torch, kan = env
    torch.manual_seed(3)
    tokens = torch.randint(0, 50, (8, 13), device="cuda:0")
    emb = kan.KANEmbedding(50, 9, device="cuda:0")
    assert torch.equal(emb(tokens[3]), emb(tokens[3].clone()))
    assert torch.equal(emb(tokens.flatten()[1:]), emb(tokens.flatten()[1:].clone()))
    rec = kan.KANRecurrence(9, 5, grid_range=(-4.0, 4.0), device="cuda:0")
    lengths = torch.tensor([0, 12, 5, 7], dtype=torch.int32, device="cuda:0")
    h0 = torch.randn(4, 5, device="cuda:0")
    x = emb(tokens[:3, 1:])
    assert _same(torch, rec(x, h0[1:], lengths[1:]), rec(x, h0[1:].clone(), lengths[1:].clone()))
    loss = kan.KANDistillLoss(2.0, "none")
    z, t = torch.randn(8, 13, 50, device="cuda:0"), torch.randn(8, 13, 3, device="cuda:0")
    ids, w = torch.randint(0, 50, (8, 13, 3), device="cuda:0"), torch.rand(8, 13, device="cuda:0")
    assert torch.equal(loss(z[1], ids[1], t[1], w[1]), loss(z[1], ids[1].clone(), t[1].clone(), w[1].clone()))


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("D,dtype", [(770, "bfloat16"), (33, "float32"), (5, "float32")])
def test_backward_through_cat(env, rows, D, dtype):
    """A part of ``torch.cat`` gets a view of the whole gradient, wherever it starts."""
    torch, kan = env
    torch.manual_seed(4)
    emb = kan.KANEmbedding(20, D, dtype=getattr(torch, dtype), device="cuda:0")
    first = torch.randn(rows, D, device="cuda:0").to(emb.table.dtype)
    ids = torch.randint(0, 20, (11,), device="cuda:0")
    dy = torch.randn(rows + 11, D, device="cuda:0").to(emb.table.dtype)
    torch.cat([first.requires_grad_(), emb(ids)]).backward(dy)
    want = kan.kan_embed_backward(ids, dy[rows:].clone(), 20, emb.scale)
    assert torch.equal(emb.table.grad, want.to(emb.table.dtype))


def test_losses_and_states_through_cat(env):
    torch, kan = env
    torch.manual_seed(5)
    z = torch.randn(6, 40, device="cuda:0", requires_grad=True)
    ids, t = torch.randint(0, 40, (6, 3), device="cuda:0"), torch.randn(6, 3, device="cuda:0")
    rows = kan.KANDistillLoss(reduction="none")(z, ids, t)
    dl = torch.rand(7, device="cuda:0")
    torch.cat([torch.zeros(1, device="cuda:0", requires_grad=True), rows]).backward(dl)
    lse = kan.kan_distill_forward(z.detach(), ids, t)[1]
    assert torch.equal(z.grad, kan.kan_distill_backward(z.detach(), ids, t, lse, dl[1:].clone()))
    rec = kan.KANRecurrence(4, 3, grid_range=(-4.0, 4.0), device="cuda:0")
    x = torch.randn(1, 5, 4, device="cuda:0", requires_grad=True)
    for k in range(2):
        out = rec(x)[k].reshape(-1)
        torch.cat([torch.zeros(1, device="cuda:0", requires_grad=True), out]).sum().backward()
        assert bool(torch.isfinite(x.grad).all()) and bool(x.grad.any())
        x.grad = None


def test_one_initial_state_for_all_sequences(env):
    """A learned state, expanded over the batch: its gradient is the sequences' sum."""
    torch, kan = env
    torch.manual_seed(6)
    rec = kan.KANRecurrence(4, 6, grid_range=(-4.0, 4.0), device="cuda:0")
    x = torch.randn(5, 8, 4, device="cuda:0")
    lengths = torch.tensor([8, 1, 0, 1, 3, 1, 8, 1, 5, 1], dtype=torch.int32, device="cuda:0")[::2]
    first = torch.randn(6, device="cuda:0", requires_grad=True)
    y, hT = rec(x, first.expand(5, 6), lengths)
    whole = first.detach().expand(5, 6).contiguous().requires_grad_()
    y2, hT2 = rec(x, whole, lengths.contiguous())
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    dy, dh = torch.randn_like(y), torch.randn_like(hT)
    torch.autograd.backward([y, hT], [dy, dh])
    torch.autograd.backward([y2, hT2], [dy, dh])
    assert torch.equal(first.grad, whole.grad.sum(0))
    s1 = torch.randn(6, 6, device="cuda:0")
    s2 = s1.clone()
    slots = torch.tensor([4, 9, 0, 9, 3, 9], dtype=torch.int32, device="cuda:0")[::2]
    assert torch.equal(rec.step(x[:3, 0], s1, slots), rec.step(x[:3, 0], s2, slots.contiguous())) and torch.equal(s1, s2)


@pytest.mark.parametrize("layout", ["columns", "one row", "vocabulary first"])
def test_logits_of_any_strides(env, layout):
    torch, kan = env
    torch.manual_seed(7)
    loss = kan.KANDistillLoss(2.0)
    if layout == "columns":
        z = torch.randn(40, 6, device="cuda:0", requires_grad=True)
        view = z.t()
    elif layout == "one row":
        z = torch.randn(40, device="cuda:0", requires_grad=True)
        view = z.expand(6, 40)
    else:
        z = torch.randn(2, 40, 3, device="cuda:0", requires_grad=True)
        view = z.transpose(1, 2)
    lead = view.shape[:-1]
    ids, t = torch.randint(0, 40, (*lead, 3), device="cuda:0"), torch.randn(*lead, 3, device="cuda:0")
    w = torch.rand(*lead, device="cuda:0")
    got = loss(view, ids, t, w)
    copy = view.detach().contiguous().requires_grad_()
    want = loss(copy, ids, t, w)
    assert torch.equal(got, want)
    got.backward()
    want.backward()
    back = {"columns": lambda v: v.t(), "one row": lambda v: v.sum(0), "vocabulary first": lambda v: v.transpose(1, 2)}
    assert torch.equal(z.grad, back[layout](copy.grad))
