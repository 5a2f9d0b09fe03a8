"""GPU: the gated delta rule and the join under HIP graph capture, on two streams, and
with workspaces that captured graphs share.

Calls are captured with their workspaces allocated beforehand and replayed several
times, with eager work and synchronisations between the replays; every replay
equals the eager result bitwise.
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


def _delta(torch, L, F, seed, B, T, Hk, Hv, Dk, Dv, dtype, ws=None):
    torch.manual_seed(seed)
    q, k = (torch.randn(B, T, Hk, Dk, device="cuda:0").to(dtype) for _ in range(2))
    v, dy = (torch.randn(B, T, Hv, Dv, device="cuda:0").to(dtype) for _ in range(2))
    g, beta = -torch.rand(B, T, Hv, device="cuda:0"), torch.rand(B, T, Hv, device="cuda:0")
    lengths = torch.randint(T // 2, T + 1, (B,), dtype=torch.int32, device="cuda:0")
    y, (dq, dk, dv) = torch.empty_like(v), (torch.empty_like(t) for t in (q, k, v))
    dh = torch.randn(B, Hv, Dk, Dv, device="cuda:0")
    desc = F.delta_desc(q, k, v, None, True, dq, dk, dv)
    if ws is None:
        ws = _ws(torch, F.kan_delta_workspace_size(desc, L.KAN_PASS_BACKWARD))
        assert ws[1] >= F.kan_delta_workspace_size(desc, L.KAN_PASS_FORWARD)
    last = [torch.empty_like(dh), torch.empty_like(g), torch.empty_like(g)]

    def step():
        last[0].copy_(F.kan_delta_forward(q, k, v, g, beta, dh, lengths, unit=True, out=y, ws=ws)[1])
        got = F.kan_delta_backward(q, k, v, g, beta, dy, None, lengths, dh, unit=True, dq=dq, dk=dk, dv=dv, ws=ws)
        last[1].copy_(got[3])
        last[2].copy_(got[4])
    return step, [y, dq, dk, dv, *last], ws


def _whole(torch, L, F, seed, ws=None):
    return _delta(torch, L, F, seed, 3, 200, 2, 4, 64, 64, torch.bfloat16, ws)


def _cut(torch, L, F, seed, ws=None):
    """Few heads and a long sequence: cut into segments."""
    made = _delta(torch, L, F, seed, 1, 3000, 1, 2, 40, 48, torch.float32, ws)
    return made


def _step(torch, L, F, seed, ws=None):
    torch.manual_seed(seed)
    q, k, v = torch.randn(9, 2, 64, device="cuda:0"), torch.randn(9, 2, 64, device="cuda:0"), torch.randn(
        9, 2, 40, device="cuda:0")
    g, beta = -torch.rand(9, 2, device="cuda:0"), torch.rand(9, 2, device="cuda:0")
    first, y = torch.randn(9, 2, 64, 40, device="cuda:0"), torch.empty(9, 2, 40, device="cuda:0")
    state = torch.empty_like(first)

    def step():
        state.copy_(first)
        for _ in range(3):
            F.kan_delta_step(q, k, v, g, beta, state, unit=True, out=y)
    return step, [y, state], None


def _join(torch, L, F, seed, ws=None):
    torch.manual_seed(seed)
    h, r, gate, dy, dx = (torch.randn(3000, 130, device="cuda:0") for _ in range(5))
    w = torch.rand(130, device="cuda:0")
    ws = ws or _ws(torch, F.kan_join_workspace_size(F.join_desc(h, r, gate)))
    outs = [torch.empty_like(t) for t in (h, h, h, h, h, w, w)]

    def step():
        y, x, stats = F.kan_join_forward(h, r, gate, w, w)
        got = F.kan_join_backward(h, y, stats, dy, dx, gate, w, w, ws=ws)
        for to, t in zip(outs, (y, x, *got)):
            to.copy_(t)
    return step, outs, ws


CASES = [_whole, _cut, _step, _join]


def _eager(torch, step, outs):
    step()
    torch.cuda.synchronize()
    return [o.clone() for o in outs]


def _capture(torch, step):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


@pytest.mark.parametrize("make", CASES, ids=[f.__name__ for f in CASES])
def test_replays_equal_eager(env, make):
    torch, L, F = env
    step, outs, _ = make(torch, L, F, 1)
    want = _eager(torch, step, outs)
    graph = _capture(torch, step)
    other = make(torch, L, F, 2)[0]
    for _ in range(4):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        other()                                   # eager work between the replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("make", [_whole, _cut, _join], ids=["whole", "cut", "join"])
def test_graphs_that_share_a_workspace(env, make):
    """Two captured calls with one workspace, replayed in turn on one stream: nothing is kept in it between calls."""
    torch, L, F = env
    one, outs1, ws = make(torch, L, F, 3)
    two, outs2, _ = make(torch, L, F, 4, ws)
    want1, want2 = _eager(torch, one, outs1), _eager(torch, two, outs2)
    graphs = _capture(torch, one), _capture(torch, two)
    for _ in range(3):
        for o in (*outs1, *outs2):
            o.fill_(float("nan"))
        ws[0].fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs1 + outs2, want1 + want2))


def test_two_streams(env):
    """The same operators on two streams, other inputs on each, interleaved."""
    torch, L, F = env
    made = [(make(torch, L, F, 10 + k), make(torch, L, F, 20 + k)) for k, make in enumerate(CASES)]
    want = [_eager(torch, step, outs) for pair in made for step, outs, _ in pair]
    for pair in made:
        for _, outs, _ in pair:
            for o in outs:
                o.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for pair in made:
            for s, (step, _, _) in zip(streams, pair):
                with torch.cuda.stream(s):
                    step()
    torch.cuda.synchronize()
    got = [outs for pair in made for _, outs, _ in pair]
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_threads(env):
    """Two host threads, each with its own stream, calling at once."""
    import threading
    torch, L, F = env
    made = [_whole(torch, L, F, 30), _whole(torch, L, F, 31)]
    want = [_eager(torch, step, outs) for step, outs, _ in made]

    def work(step):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                step()
    threads = [threading.Thread(target=work, args=(m[0],)) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for m, w in zip(made, want) for a, b in zip(m[1], w))
