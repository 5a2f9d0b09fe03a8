"""GPU: the delta rule and the join on views of larger tensors: data that starts off 16
bytes in the wrappers and in gradients that autograd hands on, expanded and
transposed views in the modules.  Results equal those of copies, bit for bit."""

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
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_delta(env, dtype):
    torch, kan = env
    torch.manual_seed(0)
    q, k, v, dy = (torch.randn(3, 130, 2, 32, device="cuda:0").to(getattr(torch, dtype)) for _ in range(4))
    g, beta = -torch.rand(3, 130, 2, device="cuda:0"), torch.rand(3, 130, 2, device="cuda:0")
    h0, dhT = torch.randn(3, 2, 32, 32, device="cuda:0"), torch.randn(3, 2, 32, 32, device="cuda:0")
    n = torch.tensor([130, 0, 77], dtype=torch.int32, device="cuda:0")
    args = [q, k, v, g, beta, h0, n]
    want = kan.kan_delta_forward(*args, unit=True)
    back = [q, k, v, g, beta, dy, h0, n, dhT]
    grads = kan.kan_delta_backward(*back, unit=True)
    for i in range(len(args)):
        assert _same(torch, want, kan.kan_delta_forward(*(_off(torch, t) if j == i else t for j, t in enumerate(args)),
                                                        unit=True)), i
    for i in range(len(back)):
        assert _same(torch, grads, kan.kan_delta_backward(*(_off(torch, t) if j == i else t for j, t in enumerate(back)),
                                                          unit=True)), i
    row = [t[:, 0].contiguous() for t in args[:5]]
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda:0")
    first = h0.clone()
    y = kan.kan_delta_step(*row, first, slots)
    for i in range(6):
        state = h0.clone()
        moved = [_off(torch, t) if j == i else t for j, t in enumerate([*row, slots])]
        assert torch.equal(y, kan.kan_delta_step(*moved[:5], state, moved[5])) and torch.equal(state, first), i
    # outputs and the pool are where the caller wants them: they must be aligned
    with pytest.raises(Exception):
        kan.kan_delta_step(*row, _off(torch, h0), slots)
    with pytest.raises(Exception):
        kan.kan_delta_forward(*args, out=_off(torch, v))


def test_gradients_may_start_anywhere(env):
    torch, kan = env
    torch.manual_seed(1)
    q, k, v, dy = (torch.randn(2, 70, 1, 24, device="cuda:0").bfloat16() for _ in range(4))
    g, beta = -torch.rand(2, 70, 1, device="cuda:0"), torch.rand(2, 70, 1, device="cuda:0")
    want = kan.kan_delta_backward(q, k, v, g, beta, dy)
    base = torch.full((2, 70, 80), 7.0, dtype=torch.bfloat16, device="cuda:0")
    dq, dk, dv = (base[..., None, o:o + 24] for o in (1, 27, 54))
    kan.kan_delta_backward(q, k, v, g, beta, dy, dq=dq, dk=dk, dv=dv)
    assert _same(torch, want, (dq, dk, dv))
    assert bool((base[..., [0, 25, 26, 51, 52, 53, 78, 79]] == 7).all())        # nothing else was written


def test_outputs_stay_inside(env):
    """Memory on both sides of y, hT's pool and the workspace keeps what it held."""
    torch, kan = env
    from kolmogorov_arnold_network_amd import _lib as L, functional as F
    torch.manual_seed(2)
    for B, T, H, Dk, Dv in ((3, 65, 2, 31, 33), (1, 1500, 1, 24, 40), (2, 128, 2, 128, 128)):
        q, k = (torch.randn(B, T, H, Dk, device="cuda:0") for _ in range(2))
        v, dy = (torch.randn(B, T, H, Dv, device="cuda:0") for _ in range(2))
        g, beta = -torch.rand(B, T, H, device="cuda:0"), torch.rand(B, T, H, device="cuda:0")
        for p in (L.KAN_PASS_FORWARD, L.KAN_PASS_BACKWARD):
            n = F.kan_delta_workspace_size(F.delta_desc(q, k, v, None, True, q, k, v), p)
            buf = torch.full((n + 8192,), 171, dtype=torch.uint8, device="cuda:0")
            at = (-buf.data_ptr()) % 256 + 2048
            ws = (buf[at:at + n], n)
            rows = torch.full((B * T * H * Dv + 2048,), 9.0, device="cuda:0")
            y = rows[1024:-1024].view(B, T, H, Dv)
            if p == L.KAN_PASS_FORWARD:
                kan.kan_delta_forward(q, k, v, g, beta, unit=True, ws=ws, out=y)
            else:
                kan.kan_delta_backward(q, k, v, g, beta, dy, unit=True, ws=ws, dq=torch.empty_like(q),
                                       dk=torch.empty_like(k), dv=y)
            assert bool((buf[:at] == 171).all()) and bool((buf[at + n:] == 171).all())
            assert bool((rows[:1024] == 9).all()) and bool((rows[-1024:] == 9).all())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_join(env, dtype):
    torch, kan = env
    torch.manual_seed(3)
    h, r, gate, dy, dx = (torch.randn(9, 50, device="cuda:0").to(getattr(torch, dtype)) for _ in range(5))
    w, u = torch.rand(50, device="cuda:0"), torch.rand(50, device="cuda:0")
    args = [h, r, gate, w, u]
    want = kan.kan_join_forward(*args)
    for i in range(5):
        assert _same(torch, want, kan.kan_join_forward(*(_off(torch, t) if j == i else t for j, t in enumerate(args)))), i
    y, _, stats = want
    back = [h, y, stats, dy, dx, gate, w, u]
    grads = kan.kan_join_backward(*back)
    for i in range(8):
        assert _same(torch, grads, kan.kan_join_backward(*(_off(torch, t) if j == i else t for j, t in enumerate(back)))), i
    one = h[:1].expand(9, 50)                         # one row for all
    assert _same(torch, kan.kan_join_forward(one, one, one, w, u), kan.kan_join_forward(*(one.contiguous(),) * 3, w, u))


def test_gradients_that_autograd_hands_on(env):
    """dy as a part of a cat's gradient starts anywhere; a sum's is expanded."""
    torch, kan = env
    torch.manual_seed(4)
    rule, join = kan.KANDeltaRule(6, 1, 5, 7, device="cuda:0"), kan.KANJoin(7, device="cuda:0")
    x = torch.rand(2, 9, 6, device="cuda:0", requires_grad=True)
    pad, c = torch.zeros(1, 7, device="cuda:0"), torch.randn(1 + 4 * 18, 7, device="cuda:0")

    def run(cat):
        x.grad = None
        y, s = rule(x)
        z, rows = join(y)
        parts = [t.reshape(-1, 7) for t in (y, z, rows, rows)]
        if cat:
            (torch.cat([pad, *parts]) * c).sum().backward()
        else:
            sum((t * c[1 + 18 * i:19 + 18 * i]).sum() for i, t in enumerate(parts)).backward()
        return x.grad.clone()
    a, b = run(True), run(False)
    assert float((a - b).abs().max()) <= 1e-6 * float(a.abs().max())
    join(rule(x)[0])[1].sum().backward()
