"""GPU: digits of the gated delta rule's bfloat16 answers where their terms cancel.

Two rows write nearly the same values, u_0 and u_1, under different keys, and every
later row asks for the difference of the two: y = D_0 u_0 - D_1 u_1 with D the
decays since, 2^-12 of its terms t = |D_1 u_1|.  Keys have one entry, so that every
sum has two terms.  With e = 2^-24 an answer is off by, of t,

  a decay: its argument, below 1, rounds to e and the hardware's 2^x to 2 e; a row's
      factor is one decay and the chunks' are two more, 9 e a term;
  u: a product, e; times a decay, 2 e a term; the state's entry, e a chunk (three);
  products on planes of bfloat16: what three planes leave, e for each of two floats,
      and the products left out, 2 e; the six added, e of at most 2 t each: 16 e,
      once in the state's entry and once in the answer,

44 e a term and 88 e for both, and by the rounding to bfloat16, 2^-8 of |y|.
Floats held in two planes would be off by up to 2^-15 t = 512 e.
"""

import numpy as np
import pytest

from kan_testutil import ensure_built
from oracle import delta as O

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import functional as F
    return torch, F


# (B, Hv, Dk, Dv): every padded width of keys, few heads and many, whole pieces of eight and odd ones
SHAPES = [(1, 2, 32, 64), (2, 1, 64, 128), (1, 2, 128, 128), (3, 2, 33, 31), (2, 1, 127, 65),
          (130, 2, 32, 64), (128, 2, 64, 64), (64, 2, 128, 128), (130, 1, 65, 129)]


@pytest.mark.parametrize("B,Hv,Dk,Dv", SHAPES)
def test_answers_that_cancel(env, B, Hv, Dk, Dv):
    torch, F = env
    T = 150
    r = np.random.default_rng(B + Dk + Dv)
    q, k = np.zeros((B, T, 1, Dk), np.float32), np.zeros((B, T, 1, Dk), np.float32)
    q[:, :, 0, 0], q[:, :, 0, Dk - 1] = 1, -1
    k[:, 0, 0, 0], k[:, 1, 0, Dk - 1], k[:, 2:, 0, Dk // 2] = 1, 1, 1
    v = r.standard_normal((B, T, Hv, Dv)).astype(np.float32)
    v[:, 1] = v[:, 0]
    g = (-0.005 * r.random((B, T, Hv))).astype(np.float32)
    beta = np.zeros((B, T, Hv), np.float32)
    beta[:, 0] = 0.5 + 0.5 * r.random((B, Hv))
    beta[:, 1] = beta[:, 0] * np.exp(g[:, 1].astype(np.float64)) * (1 + 2.0 ** -12)
    args = [torch.from_numpy(t).cuda() for t in (q, k, v, g, beta)]
    args[:3] = [t.to(torch.bfloat16) for t in args[:3]]
    y, _ = F.kan_delta_forward(*args, scale=1.0)
    some = sorted({0, B // 2, B - 1})
    host = [t[some].double().cpu().numpy() for t in args]
    want = O.delta_forward(*host, scale=1.0)[0][:, 2:]
    # the answer of row t to the second key alone, the terms' size
    c = np.cumsum(host[3], 1)
    term = np.abs(np.exp(c[:, 2:] - c[:, 1:2]) * host[4][:, 1:2])[..., None] * np.abs(host[2][:, 1:2])
    off = np.abs(y[some, 2:].double().cpu().numpy() - want)
    assert (np.abs(want) < 2.0 ** -11.9 * term).all()
    assert (off <= 88 * E * term + 2.0 ** -8 * np.abs(want)).all(), (off / term).max() / E
