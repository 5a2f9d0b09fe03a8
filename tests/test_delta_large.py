"""GPU: the gated delta rule at its larger sizes: arrays past 2^31 elements, rows 2^24
elements apart, many heads, long sequences, all columns; expanded inputs and
infinities.

A large call is held against small ones of its sequences, which the other tests hold
against the float64 oracle; tolerances are theirs, for each of the two.
"""

import pytest

from kan_testutil import ensure_built
from test_delta import _draw, _error, _np, _tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    yield torch, F
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def seeded(env):
    env[0].manual_seed(0)


def _last_rows(t, n=500):
    return _np(t[:, -n:])


def test_rows_past_32_bits(env):
    """v, y, dy and dv of 2^31 elements and more."""
    torch, F = env
    B, T, H, Dk, Dv = 2, 65600, 16, 8, 1024
    args = _draw(torch, B, T, H, H, Dk, Dv, "bf16", "apart", 1)
    dy = torch.randn(B, T, H, Dv, device="cuda:0", dtype=torch.bfloat16)
    assert dy.numel() > 2 ** 31
    y, hT = F.kan_delta_forward(*args)
    part = tuple(t[1:, :, -2:].contiguous() for t in args)             # the last two heads of the last sequence
    wy, wh = F.kan_delta_forward(*part)
    assert _error(_last_rows(y[1:, :, -2:]), _last_rows(wy)) <= 2 * _tol(T, "bf16")
    assert _error(_np(hT[1:, -2:]), _np(wh)) <= 2 * _tol(T)
    del y
    got = F.kan_delta_backward(*args, dy)
    want = F.kan_delta_backward(*part, dy[1:, :, -2:].contiguous())
    for i in range(5):
        assert _error(_last_rows(got[i][1:, :, -2:]), _last_rows(want[i])) <= 2 * _tol(T, "bf16" if i < 3 else None, True), i


def test_float32_rows_2_to_the_24_apart(env):
    """64 rows span 2^32 bytes."""
    torch, F = env
    B, T, D, row = 1, 70, 32, 2 ** 24
    base, grad = (torch.empty((T - 1) * row + 3 * D, device="cuda:0") for _ in range(2))

    def views(t):
        return [t.as_strided((B, T, 1, D), (T * row, row, D, 1), i * D) for i in range(3)]
    args = _draw(torch, B, T, 1, 1, D, D, "f32", "apart", 8)
    far = views(base)
    for a, b in zip(far, args):
        a.copy_(b)
    dy = torch.randn(B, T, 1, D, device="cuda:0")
    near = F.kan_delta_forward(*args), F.kan_delta_backward(*args, dy)
    assert all(torch.equal(a, b) for a, b in zip(near[0], F.kan_delta_forward(*far, *args[3:])))
    dq, dk, dv = views(grad)
    F.kan_delta_backward(*far, *args[3:], dy, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip(near[1][:3], (dq, dk, dv)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_heads(env, dtype):
    torch, F = env
    args = _draw(torch, 32000, 5, 4, 8, 7, 9, dtype, "packed", 2, unit=True)       # 256000 heads
    dy = torch.randn(32000, 5, 8, 9, device="cuda:0").to(args[0].dtype)
    y, hT = F.kan_delta_forward(*args, unit=True)
    got = F.kan_delta_backward(*args, dy, unit=True, need_dh0=True)
    for lo in (0, 15990, 31990):
        part = tuple(t[lo:lo + 10].contiguous() for t in args)
        wy, wh = F.kan_delta_forward(*part, unit=True)
        assert _error(_np(y[lo:lo + 10]), _np(wy)) <= 2 * _tol(5, dtype)
        assert _error(_np(hT[lo:lo + 10]), _np(wh)) <= 2 * _tol(5)
        want = F.kan_delta_backward(*part, dy[lo:lo + 10].contiguous(), unit=True, need_dh0=True)
        for i, (a, b) in enumerate(zip(got, want)):
            assert _error(_np(a[lo:lo + 10]), _np(b)) <= 2 * _tol(5, dtype if i < 3 else None, True), i
    pool = torch.randn(32000, 8, 7, 9, device="cuda:0")
    few = pool[-10:].clone()
    row = [t[:, 0] if t.dim() == 4 else t[:, 0].contiguous() for t in args]
    y = F.kan_delta_step(*row, pool, unit=True)
    assert torch.equal(y[-10:], F.kan_delta_step(*(t[-10:].contiguous() for t in row), few, unit=True))
    assert torch.equal(pool[-10:], few)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1e-5, 0.3])
def test_a_long_sequence_in_parts(env, decay, dtype):
    """Segments of one call against a call for each part with its state handed on, also where nothing is forgotten."""
    torch, F = env
    T, cut = 50001, 20000
    args = _draw(torch, 1, T, 1, 2, 32, 48, dtype, "apart", 3, decay=decay)
    y, hT = F.kan_delta_forward(*args)
    a = [tuple(t[:, s].contiguous() for t in args) for s in (slice(0, cut), slice(cut, T))]
    y0, h = F.kan_delta_forward(*a[0])
    y1, h1 = F.kan_delta_forward(*a[1], h)
    assert _error(_np(y[:, :cut]), _np(y0)) <= 2 * _tol(T, dtype) and _error(_np(y[:, cut:]), _np(y1)) <= 2 * _tol(T, dtype)
    assert _error(_np(hT), _np(h1)) <= 2 * _tol(T)
    dy, dhT = torch.randn(1, T, 2, 48, device="cuda:0").to(args[0].dtype), torch.randn(1, 2, 32, 48, device="cuda:0")
    got = F.kan_delta_backward(*args, dy, None, None, dhT)
    late = F.kan_delta_backward(*a[1], dy[:, cut:].contiguous(), h, None, dhT)
    early = F.kan_delta_backward(*a[0], dy[:, :cut].contiguous(), None, None, late[5])
    for i in range(5):
        for part, s in ((early, slice(0, cut)), (late, slice(cut, T))):
            assert _error(_np(got[i][:, s]), _np(part[i])) <= 2 * _tol(T, dtype if i < 3 else None, True), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_expanded_inputs(env, dtype):
    """q and k of one head and one sequence for all, by strides of 0."""
    torch, F = env
    q, k, v, g, beta = _draw(torch, 3, 150, 4, 4, 64, 72, dtype, "apart", 4)
    q, k, v = q[:1, :, :1].expand_as(q), k[:1, :, :1].expand_as(k), v[:, :, :1].expand_as(v)
    dy = torch.randn(3, 150, 4, 72, device="cuda:0").to(q.dtype)
    whole = [t.contiguous() for t in (q, k, v)]
    assert all(torch.equal(a, b) for a, b in zip(F.kan_delta_forward(q, k, v, g, beta), F.kan_delta_forward(*whole, g, beta)))
    assert all(torch.equal(a, b) for a, b in zip(F.kan_delta_backward(q, k, v, g, beta, dy)[:5],
                                                 F.kan_delta_backward(*whole, g, beta, dy)[:5]))


def test_one_row_of_a_far_view(env):
    """A dimension of one element may have any stride."""
    torch, F = env
    args = _draw(torch, 2, 1, 1, 1, 16, 16, "f32", "apart", 5)
    odd = [t.as_strided(t.shape, (t.stride(0), 2 ** 41, 2 ** 42, 1)) for t in args[:3]]
    assert all(torch.equal(a, b) for a, b in zip(F.kan_delta_forward(*args), F.kan_delta_forward(*odd, *args[3:])))
    row = [t[:, 0] for t in odd]
    state = torch.zeros(2, 1, 16, 16, device="cuda:0")
    y = F.kan_delta_step(*row, *(t[:, 0].contiguous() for t in args[3:]), state)
    assert _error(_np(y[:, None]), _np(F.kan_delta_forward(*args)[0])) <= 2 * _tol(1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [200, 3000])
def test_an_infinity_does_not_go_missing(env, T, dtype):
    """An infinite value stays infinite or becomes NaN, through whole and cut sequences, in its column and no other head."""
    torch, F = env
    args = _draw(torch, 1, T, 2, 2, 32, 48, dtype, "apart", 6)
    y0, h0 = F.kan_delta_forward(*args)
    args[2][0, 70, 1, 5] = float("inf")
    y, h = F.kan_delta_forward(*args)
    assert torch.equal(y[:, :, 0], y0[:, :, 0]) and torch.equal(h[:, 0], h0[:, 0])
    assert not y[0, 70:, 1, 5].isfinite().any() and not h[0, 1, :, 5].isfinite().any()
    assert torch.equal(y[0, :64], y0[0, :64])
