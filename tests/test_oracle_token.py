"""CPU: the float64 oracles of the token-side operators against closed forms
and their gradients against central differences."""

import numpy as np
import pytest

from oracle import token as O


def _diff(f, a, eps=1e-6):
    """Central differences of the scalar ``f`` at every element of ``a`` (float64).
    Their error: eps^2 / 6 times the third derivative, and 2^-53 |f| / eps."""
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + eps
        hi = f()
        a[i] = keep - eps
        lo = f()
        a[i] = keep
        out[i] = (hi - lo) / (2 * eps)
    return out


TOL = 1e-7          # differences: 1e-12 + 2^-53 * 100 / 1e-6 ~ 1e-8, ten times that


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    rng = np.random.default_rng(1)
    ids = np.array([3, 0, 3, -1, 7, 5, 3])
    E, dy = rng.standard_normal((6, 4)), rng.standard_normal((7, 4))
    got = O.embed_backward(ids, dy, 6, 1.5)
    want = _diff(lambda: float((O.embed_forward(ids, E, 1.5) * dy).sum()), E)
    assert np.abs(got - want).max() < TOL
    assert (O.embed_forward(ids, E, 1.5)[[3, 4]] == 0).all()


def test_recurrence_with_a_constant_gate_is_a_geometric_sum():
    T, g = 40, 1.3
    x = np.random.default_rng(2).standard_normal((1, T, 3))
    f = 1 / (1 + np.exp(-g))
    y, hT = O.recur_forward(x, np.full_like(x, g))
    w = np.array([[f ** (t - s) * (1 - f) if s <= t else 0.0 for s in range(T)] for t in range(T)])
    assert np.abs(y[0] - w @ x[0]).max() < 1e-13 and (hT == y[:, -1]).all()


@pytest.mark.parametrize("lengths", [None, [4, 0, 2]])
def test_recurrence_gradients_match_differences(lengths):
    rng = np.random.default_rng(3)
    B, T, D = 3, 4, 2
    x, g, dy = (rng.standard_normal((B, T, D)) for _ in range(3))
    h0, dhT = rng.standard_normal((B, D)), rng.standard_normal((B, D))

    def loss():
        y, hT = O.recur_forward(x, g, h0, lengths)
        return float((y * dy).sum() + (hT * dhT).sum())

    dx, dg, dh0 = O.recur_backward(x, g, dy, h0, lengths, dhT)
    for got, a in ((dx, x), (dg, g), (dh0, h0)):
        assert np.abs(got - _diff(loss, a)).max() < TOL


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distillation_gradient_matches_differences(tau):
    rng = np.random.default_rng(4)
    z, t = rng.standard_normal((4, 9)), rng.standard_normal((4, 3))
    ids = np.array([[0, 4, 8], [2, 2, 5], [-1, 3, 9], [-1, 9, 100]])      # repeated, absent
    w, dl = np.array([1.0, 0.5, 2.0, 1.0]), np.array([0.3, 1.0, 2.0, 1.0])

    def loss():
        return float((O.distill(z, ids, t, tau, w)[0] * dl).sum())

    dz = O.distill(z, ids, t, tau, w, dl)[2]
    assert np.abs(dz - _diff(loss, z)).max() < TOL
    assert (dz[3] == 0).all() and np.abs(dz[:3].sum(1)).max() < 1e-14


def test_distillation_of_a_student_equal_to_its_teacher_is_zero():
    z = np.random.default_rng(5).standard_normal((3, 6))
    ids = np.tile(np.arange(6), (3, 1))
    loss, lse, dz = O.distill(z, ids, z, 2.0)
    assert np.abs(loss).max() < 1e-14 and np.abs(dz).max() < 1e-15
    assert np.abs(lse - np.log(np.exp(z / 2).sum(1))).max() < 1e-14


def test_distillation_rows_without_a_distribution():
    z = np.zeros((3, 4))
    z[1] = -np.inf
    ids = np.array([[0, 1], [0, 1], [-1, 4]])
    loss, lse, dz = O.distill(z, ids, np.zeros((3, 2)), 1.0, np.array([0.0, 1.0, 1.0]))
    assert (loss == 0).all() and (dz == 0).all()
    assert abs(lse[0] - np.log(4)) < 1e-15 and lse[1] == -np.inf and abs(lse[2] - np.log(4)) < 1e-15
