"""Pins of the float64 oracles of the delta rule and the join: closed forms and differences."""

import numpy as np
import pytest

from oracle import delta as O


def _draw(seed, B=2, T=5, Hk=1, Hv=2, Dk=3, Dv=4):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, T, Hk, Dk)), r.standard_normal((B, T, Hk, Dk)), r.standard_normal((B, T, Hv, Dv)),
            -r.random((B, T, Hv)), r.random((B, T, Hv)), r.standard_normal((B, Hv, Dk, Dv)))


def test_a_stored_pair_is_recalled():
    """beta = 1 and a unit key: the state answers the key with its value exactly."""
    q, k, v, g, beta, h0 = _draw(0)
    k = k / np.linalg.norm(k, axis=-1, keepdims=True)
    y, _ = O.delta_forward(k, k, v, g, np.ones_like(beta), h0, scale=1.0)
    np.testing.assert_allclose(y, v, atol=1e-12)


def test_beta_zero_decays_alone():
    q, k, v, g, beta, h0 = _draw(1)
    _, hT = O.delta_forward(q, k, v, g, 0 * beta, h0)
    np.testing.assert_allclose(hT, h0 * np.exp(g.sum(1))[..., None, None], rtol=1e-12)


def test_lengths_and_unit():
    q, k, v, g, beta, h0 = _draw(2)
    y, hT = O.delta_forward(q, k, v, g, beta, h0, lengths=[3, 0])
    short = O.delta_forward(q[:1, :3], k[:1, :3], v[:1, :3], g[:1, :3], beta[:1, :3], h0[:1])
    np.testing.assert_array_equal(y[:1, :3], short[0])
    assert not y[0, 3:].any() and not y[1].any()
    np.testing.assert_array_equal(hT[1], h0[1])
    big = O.delta_forward(q * 1e4, k * 3e4, v, g, beta, h0, unit=True)[0]
    np.testing.assert_allclose(big, O.delta_forward(q * 1e5, k * 1e5, v, g, beta, h0, unit=True)[0], rtol=1e-9)


@pytest.mark.parametrize("unit", [False, True])
def test_delta_gradients_by_differences(unit):
    a = list(_draw(3))
    r = np.random.default_rng(4)
    dy, dhT = r.standard_normal(a[2].shape), r.standard_normal(a[5].shape)
    lengths = [5, 3]

    def loss(*b):
        y, hT = O.delta_forward(*b, lengths=lengths, unit=unit)
        return (y * dy).sum() + (hT * dhT).sum()

    grads = O.delta_backward(*a[:5], dy, a[5], lengths=lengths, dhT=dhT, unit=unit)
    for i, grad in enumerate(grads):
        for at in [tuple(r.integers(0, n) for n in a[i].shape) for _ in range(6)]:
            e, d = 1e-6, []
            for s in (e, -e):
                b = [x.copy() for x in a]
                b[i][at] += s
                d.append(loss(*b))
            assert abs((d[0] - d[1]) / (2 * e) - grad[at]) <= 1e-7 * (1 + abs(grad[at])), (i, at)


@pytest.mark.parametrize("post,pre,gate,activation", [(True, True, True, "silu"), (True, False, True, "sigmoid"),
                                                      (False, True, False, "silu"), (True, True, False, "silu")])
def test_join_gradients_by_differences(post, pre, gate, activation):
    r = np.random.default_rng(5)
    N, D = 3, 7
    a = {"h": r.standard_normal((N, D)), "r": r.standard_normal((N, D)), "w_post": r.standard_normal(D)}
    if gate:
        a["gate"] = r.standard_normal((N, D))
    if pre:
        a["w_pre"] = r.standard_normal(D)
    kw = dict(post=post, activation=activation, scale=0.7)
    dy, dx = r.standard_normal((N, D)), r.standard_normal((N, D)) if pre else None

    def loss(b):
        y, x, _, _ = O.join_forward(**b, pre=pre, **kw)
        return (y * dy).sum() + (0 if x is None else (x * dx).sum())

    y, _, n1, n2 = O.join_forward(**a, pre=pre, **kw)
    got = O.join_backward(a["h"], y, n1, n2, dy, dx, a.get("gate"), a["w_post"], a.get("w_pre"), **kw)
    for name, grad in zip(("h", "r", "gate", "w_post", "w_pre"), got):
        if name not in a:
            continue
        for at in np.ndindex(*a[name].shape):
            e, d = 1e-6, []
            for s in (e, -e):
                b = {n: x.copy() for n, x in a.items()}
                b[name][at] += s
                d.append(loss(b))
            assert abs((d[0] - d[1]) / (2 * e) - grad[at]) <= 1e-7 * (1 + abs(grad[at])), (name, at)
