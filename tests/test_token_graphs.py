"""GPU: the token-side entry points under HIP graph capture and on two streams.

Each operator's calls are captured once with their workspaces allocated
beforehand and replayed several times, with eager work and synchronisations
between the replays; every replay equals the eager result bitwise.  On two
streams at once the results equal the eager ones too.
"""

import pytest

from kan_testutil import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from kolmogorov_arnold_network_amd import _lib as L
    from kolmogorov_arnold_network_amd import functional as F
    return torch, L, F


def _ws(torch, n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda:0"), n


def _embed(torch, L, F, seed):
    torch.manual_seed(seed)
    ids = torch.randint(-1, 700, (3000,), device="cuda:0")
    E, dy = torch.randn(700, 96, device="cuda:0"), torch.randn(3000, 96, device="cuda:0")
    y, dE = torch.empty(3000, 96, device="cuda:0"), torch.empty(700, 96, device="cuda:0")
    ws = _ws(torch, F.kan_embed_workspace_size(F.embed_desc(3000, 700, 96, torch.float32, torch.float32, torch.int64, 1.0)))

    def step():
        F.kan_embed_forward(ids, E, 2.0, out=y)
        F.kan_embed_backward(ids, dy, 700, 2.0, ws=ws, out=dE)
    return step, (y, dE)


def _recur(torch, L, F, seed, T=5000):
    """Few channels and a long sequence: cut into segments, with a workspace."""
    torch.manual_seed(seed)
    x, g, dy = (torch.randn(1, T, 40, device="cuda:0") for _ in range(3))
    y, dx, dg = (torch.empty_like(x) for _ in range(3))
    desc = F.recur_desc(x, g, dx, dg)
    wf, wb = (_ws(torch, F.kan_recur_workspace_size(desc, p)) for p in (L.KAN_PASS_FORWARD, L.KAN_PASS_BACKWARD))

    def step():
        F.kan_recur_forward(x, g, out=y, ws=wf)
        F.kan_recur_backward(x, g, y, dy, dx=dx, dg=dg, ws=wb)
    return step, (y, dx, dg)


def _step(torch, L, F, seed):
    torch.manual_seed(seed)
    x, g = torch.randn(9, 40, device="cuda:0"), torch.randn(9, 40, device="cuda:0")
    first, state, y = torch.randn(9, 40, device="cuda:0"), torch.empty(9, 40, device="cuda:0"), torch.empty(
        9, 40, device="cuda:0")

    def step():
        state.copy_(first)
        F.kan_recur_step(x, g, state, out=y)
    return step, (y, state)


def _distill(torch, L, F, seed):
    torch.manual_seed(seed)
    z, t = torch.randn(40, 5001, device="cuda:0"), torch.randn(40, 12, device="cuda:0")
    ids = torch.randint(0, 5001, (40, 12), device="cuda:0")
    dl, dz, dz2 = torch.rand(40, device="cuda:0"), torch.empty_like(z), torch.empty_like(z)
    ws = _ws(torch, F.kan_distill_workspace_size(F.distill_desc(z, ids, t, 2.0)))

    def step():
        _, lse = F.kan_distill_forward(z, ids, t, 2.0, ws=ws)
        F.kan_distill_backward(z, ids, t, lse, dl, 2.0, out=dz)
        F.kan_distill_step(z, ids, t, 2.0, out=dz2, ws=ws)
    return step, (dz, dz2)


CASES = [_embed, _recur, _step, _distill]


@pytest.mark.parametrize("make", CASES, ids=[f.__name__ for f in CASES])
def test_replays_equal_eager(env, make):
    torch, L, F = env
    step, outs = make(torch, L, F, 1)
    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other, _ = make(torch, L, F, 2)
    for _ in range(4):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        other()                                   # eager work between the replays
        torch.cuda.synchronize()


def test_two_streams(env):
    """The same operators on two streams, other inputs on each, interleaved."""
    torch, L, F = env
    made = [(make(torch, L, F, 10 + k), make(torch, L, F, 20 + k)) for k, make in enumerate(CASES)]
    want = []
    for pair in made:
        for step, outs in pair:
            step()
            torch.cuda.synchronize()
            want.append([o.clone() for o in outs])
            for o in outs:
                o.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for pair in made:
            for s, (step, _) in zip(streams, pair):
                with torch.cuda.stream(s):
                    step()
    torch.cuda.synchronize()
    got = [outs for pair in made for _, outs in pair]
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
