"""GPU: the calls of two and three launches that hand results on through their
workspace - the distillation step of few long rows, the recurrence in segments
with a state that is not finite - under HIP graph capture and on two streams.

Replays with a poisoned workspace and eager work between them equal the eager
result bitwise, and so do the calls on two streams at once.
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
    assert n > 0
    return torch.empty(n, dtype=torch.uint8, device="cuda:0"), n


def _distill(torch, L, F, seed):
    torch.manual_seed(seed)
    z, t = torch.randn(5, 131077, device="cuda:0"), torch.randn(5, 12, device="cuda:0")
    ids = torch.randint(0, 131077, (5, 12), device="cuda:0")
    dz, loss = torch.empty_like(z), torch.empty(5, device="cuda:0")
    ws = _ws(torch, F.kan_distill_workspace_size(F.distill_desc(z, ids, t, 2.0)))

    def step():
        loss.copy_(F.kan_distill_step(z, ids, t, 2.0, out=dz, ws=ws)[0])
    return step, (dz, loss), (ws[0],)


def _recur(torch, L, F, seed):
    torch.manual_seed(seed)
    x, g, dy = (torch.randn(1, 70000, 24, device="cuda:0") for _ in range(3))
    x[0, 9, 3] = float("inf")
    dy[0, -9, 5] = float("inf")
    y, dx, dg = (torch.empty_like(x) for _ in range(3))
    desc = F.recur_desc(x, g, dx, dg)
    wf, wb = (_ws(torch, F.kan_recur_workspace_size(desc, p)) for p in (L.KAN_PASS_FORWARD, L.KAN_PASS_BACKWARD))

    def step():
        F.kan_recur_forward(x, g, out=y, ws=wf)
        F.kan_recur_backward(x, g, y, dy, dx=dx, dg=dg, ws=wb)
    return step, (y, dx, dg), (wf[0], wb[0])


CASES = [_distill, _recur]


def _equal(torch, a, b):
    return torch.equal(torch.isfinite(a), torch.isfinite(b)) and torch.equal(a.nan_to_num(0, 0, 0), b.nan_to_num(0, 0, 0))


@pytest.mark.parametrize("make", CASES, ids=[f.__name__ for f in CASES])
def test_replays_equal_eager(env, make):
    torch, L, F = env
    step, outs, spaces = make(torch, L, F, 1)
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
    other = make(torch, L, F, 2)[0]
    for k in range(4):
        for o in outs:
            o.fill_(float("nan"))
        for w in spaces:
            w.fill_(0xff if k % 2 else 0x3f)
        graph.replay()
        torch.cuda.synchronize()
        assert all(_equal(torch, a, b) for a, b in zip(outs, want))
        other()
        torch.cuda.synchronize()


def test_two_streams(env):
    torch, L, F = env
    made = [(make(torch, L, F, 10 + k), make(torch, L, F, 20 + k)) for k, make in enumerate(CASES)]
    want = []
    for pair in made:
        for step, outs, _ in pair:
            step()
            torch.cuda.synchronize()
            want.append([o.clone() for o in outs])
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
    assert all(_equal(torch, a, b) for g, w in zip(got, want) for a, b in zip(g, w))
