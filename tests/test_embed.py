"""GPU: the embedding lookup and its gradient against the float64 oracle.

Tolerances, with e = 2^-24 (half an ulp of float32, relative): the lookup is one
product, so e relative (plus 2^-8 where the row is rounded to bf16); a sum of
n terms in any fixed order is within (n + 1) e sum |terms|, and the scale is
one more product.
"""

import numpy as np
import pytest

from kan_testutil import ensure_built, to_dev
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


def _bf16(a):
    import torch
    return torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).float().numpy()


def _ids(rng, N, V, kind):
    if kind == "uniform":
        return rng.integers(0, V, N)
    if kind == "one":
        return np.full(N, V - 1)
    if kind == "none":
        return np.where(np.arange(N) % 2, -1, V)
    if kind == "sorted":
        return np.sort(rng.integers(0, V, N))
    ids = np.minimum(((V + 1.0) ** rng.random(N)).astype(np.int64) - 1, V - 1)
    ids[rng.random(N) < 0.2] = -1
    return ids


@pytest.mark.parametrize("N", [1, 3, 64, 1000])
@pytest.mark.parametrize("D", [1, 3, 4, 7, 8, 64, 770, 2049])
@pytest.mark.parametrize("table,row", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_lookup(env, N, D, table, row):
    torch, F = env
    rng = np.random.default_rng(N * 10 + D)
    V = 37
    E = rng.standard_normal((V, D)).astype(np.float32)
    E = _bf16(E) if table == "bf16" else E
    ids = rng.integers(-2, V + 2, N)
    idt = torch.from_numpy(ids).to("cuda:0", torch.int32 if N % 2 else torch.int64)
    dt = torch.bfloat16 if row == "bf16" else torch.float32
    y = F.kan_embed_forward(idt, to_dev(E, table), 1.7, row_dtype=dt)
    assert y.dtype == dt
    want = O.embed_forward(ids, E, np.float32(1.7).astype(np.float64))
    tol = np.abs(want) * ((2.0 ** -8 if row == "bf16" else 0) + 1.01 * EPS)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    assert (got[(ids < 0) | (ids >= V)] == 0).all()


@pytest.mark.parametrize("many", [False, True])
def test_lookup_of_many_rows(env, many):
    """Above and below the count at which a lane takes four rows."""
    torch, F = env
    N = 16500 if many else 4000
    ids = torch.randint(0, 501, (N,), device="cuda:0")
    E = torch.randn(501, 1030, device="cuda:0").to(torch.bfloat16)
    assert torch.equal(F.kan_embed_forward(ids, E), E[ids])


@pytest.mark.parametrize("N,V,D,kind", [
    (1, 1, 1, "one"), (1, 5, 3, "uniform"), (31, 7, 4, "uniform"), (32, 7, 5, "one"), (33, 7, 64, "one"),
    (64, 1000, 770, "uniform"), (65, 1000, 6, "zipf"), (1000, 1, 9, "one"), (1000, 513, 130, "zipf"),
    (4999, 3203, 33, "zipf"), (5000, 131, 257, "sorted"), (3000, 40, 16, "one"), (300, 50, 12, "none"),
    (2500, 200000, 8, "zipf"), (1100, 9, 1027, "zipf"),
])
@pytest.mark.parametrize("row", ["f32", "bf16"])
def test_gradient(env, N, V, D, kind, row):
    torch, F = env
    rng = np.random.default_rng(N + V + D)
    ids = _ids(rng, N, V, kind)
    dy = rng.standard_normal((N, D)).astype(np.float32)
    dy = _bf16(dy) if row == "bf16" else dy
    idt = torch.from_numpy(ids).to("cuda:0", torch.int32 if D % 2 else torch.int64)
    dE = torch.full((V, D), float("nan"), device="cuda:0")
    got = F.kan_embed_backward(idt, to_dev(dy, row), V, 0.6, out=dE)
    want = O.embed_backward(ids, dy, V, np.float32(0.6).astype(np.float64))
    n = np.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None]
    tol = (n + 2) * EPS * O.embed_backward(ids, np.abs(dy), V, 0.6)
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    assert torch.equal(got, F.kan_embed_backward(idt, to_dev(dy, row), V, 0.6))      # the same bits


def test_gradient_is_the_transpose_of_the_lookup_by_differences(env):
    """(L(E + h dE) - L(E - h dE)) / 2h with L = <y(E), dy>: linear in E, so exact
    up to the rounding of y and of the sums (1e-5 of the terms' sizes)."""
    torch, F = env
    torch.manual_seed(1)
    ids = torch.randint(-1, 50, (400,), device="cuda:0")
    E, way = torch.randn(50, 33, device="cuda:0"), torch.randn(50, 33, device="cuda:0")
    dy = torch.randn(400, 33, device="cuda:0")

    def loss(t):
        return (F.kan_embed_forward(ids, t, 1.5).double() * dy.double()).sum()

    got = (F.kan_embed_backward(ids, dy, 50, 1.5).double() * way.double()).sum()
    want = (loss(E + 0.5 * way) - loss(E - 0.5 * way))
    assert abs(float(got - want)) < 1e-5 * float(dy.abs().sum())


def test_ids_past_32_bits_are_outside_the_table(env):
    torch, F = env
    ids = torch.tensor([2, (1 << 32) + 2, -(1 << 32) + 2, 1 << 62, -1], device="cuda:0")
    E = torch.randn(4, 8, device="cuda:0")
    y = F.kan_embed_forward(ids, E)
    assert torch.equal(y[0], E[2]) and not y[1:].any()
    dE = F.kan_embed_backward(ids, torch.ones(5, 8, device="cuda:0"), 4)
    assert torch.equal(dE[2], torch.ones(8, device="cuda:0")) and float(dE.sum()) == 8


def test_rows_of_absent_tokens_do_not_count(env):
    """NaN and infinity in the gradient of a padding row reach nothing."""
    torch, F = env
    ids = torch.tensor([0, -1, 1, -1] * 20, device="cuda:0")
    dy = torch.ones(80, 12, device="cuda:0")
    dy[1::4], dy[3::4] = float("nan"), float("inf")
    dE = F.kan_embed_backward(ids, dy, 3)
    assert (dE[:2] == 20).all() and not dE[2].any()


def test_empty(env):
    torch, F = env
    ids = torch.empty(0, dtype=torch.int64, device="cuda:0")
    E = torch.randn(5, 7, device="cuda:0")
    assert F.kan_embed_forward(ids, E).shape == (0, 7)
    dE = F.kan_embed_backward(ids, torch.empty(0, 7, device="cuda:0"), 5, out=torch.ones(5, 7, device="cuda:0"))
    assert not dE.any()


def test_refusals(env):
    torch, F = env
    from kolmogorov_arnold_network_amd import _lib as L
    dev = "cuda:0"
    ids, E = torch.zeros(6, dtype=torch.int64, device=dev), torch.zeros(5, 8, device=dev)
    for bad in (dict(ids=ids.float()), dict(ids=ids.cpu()), dict(table=E.half()), dict(table=E[:, :4]),
                dict(table=E[0]), dict(row_dtype=torch.float16), dict(out=torch.empty(5, 8, device=dev)),
                dict(ids=ids[::2])):
        with pytest.raises(ValueError):
            F.kan_embed_forward(**dict(dict(ids=ids, table=E), **bad))
    for bad in (dict(dy=torch.zeros(5, 8, device=dev)), dict(dy=torch.zeros(6, 8, device=dev).half()),
                dict(out=torch.empty(5, 7, device=dev)), dict(out=torch.empty(5, 8, device=dev).bfloat16())):
        with pytest.raises(ValueError):
            F.kan_embed_backward(**dict(dict(ids=ids, dy=torch.zeros(6, 8, device=dev), num_rows=5), **bad))
    with pytest.raises(L.KanError) as e:
        F.kan_embed_forward(ids, E, scale=float("nan"))
    assert e.value.status == L.KAN_ERR_UNSUPPORTED
    with pytest.raises(L.KanError) as e:
        F.kan_embed_backward(ids, torch.zeros(6, 8, device=dev), 5, ws=(torch.empty(64, dtype=torch.uint8,
                                                                                   device=dev), 64))
    assert e.value.status == L.KAN_ERR_WORKSPACE
