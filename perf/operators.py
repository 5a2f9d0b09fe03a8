"""Cases and plain forms of the token-side operators: embedding, gated recurrence, distillation.

The operators surround the spline layers in a model over tokens: ``embed`` turns
token ids into rows and sums the rows' gradients by token, ``recur`` mixes the
rows of a sequence, ``distill`` is the loss of the last layer's logits against a
teacher's top logits, with its gradient.  ``run`` computes one pass in elementary
float32 torch operations (``own`` false) or with the package's kernels (``own``
true); ``exact`` computes the same from the definitions in 64 bits.
"""

import math

import torch

own = False

_DEV = "cuda:0"
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token for each of 64 sequences being served: latency
        dict(name="embed_fwd_64x2048_bf16", op="embed_fwd", N=64, V=65536, D=2048, dtype="bf16", ids="zipf", pad=0.0),
        # a training batch of 8 sequences of 4096 tokens
        dict(name="embed_fwd_32768x2048_bf16", op="embed_fwd", N=32768, V=65536, D=2048, dtype="bf16", ids="zipf",
             pad=0.0),
        # its gradient, float32 dy as the layers' backward passes write it
        dict(name="embed_bwd_32768x2048_f32", op="embed_bwd", N=32768, V=65536, D=2048, dtype="f32", ids="zipf",
             pad=0.0),
        # a small ragged batch: odd table, odd width, a tenth of the rows padding
        dict(name="embed_bwd_4999x770_bf16", op="embed_bwd", N=4999, V=32003, D=770, dtype="bf16", ids="zipf",
             pad=0.1),
        # one new token for 64 of 256 served sequences, x and g as a float32 layer wrote them
        dict(name="recur_step_64x2048_f32", op="recur_step", B=64, S=256, D=2048, dtype="f32", packed=True),
        # a training batch of 8 sequences of 4096 tokens, bf16 inputs
        dict(name="recur_fwd_8x4096x2048_bf16", op="recur_fwd", B=8, T=4096, D=2048, dtype="bf16", packed=False,
             h0=False, ragged=False),
        # one long document, continued from a state, x and g the halves of one projection
        dict(name="recur_fwd_1x65536x1024_f32", op="recur_fwd", B=1, T=65536, D=1024, dtype="f32", packed=True,
             h0=True, ragged=False),
        # the training batch's backward pass on a float32 layer's output
        dict(name="recur_bwd_8x4096x2048_f32", op="recur_bwd", B=8, T=4096, D=2048, dtype="f32", packed=True,
             h0=False, ragged=False, grad="f32"),
        # a few sequences of unequal lengths (one of them empty), odd sizes
        dict(name="recur_bwd_7x1531x770_bf16", op="recur_bwd", B=7, T=1531, D=770, dtype="bf16", packed=False,
             h0=True, ragged=True, grad="f32"),
        # the last rows of a short sequence: few rows, an odd vocabulary
        dict(name="distill_step_16x32003_f32", op="distill_step", N=16, V=32003, K=16, dtype="f32", grad="f32",
             tau=2.0, masked=0.0),
        # a training batch of 8192 rows, loss and gradient in one pass
        dict(name="distill_step_8192x65536_f32", op="distill_step", N=8192, V=65536, K=64, dtype="f32", grad="f32",
             tau=2.0, masked=0.1),
        # the backward pass alone, as autograd calls it, bf16 logits, odd vocabulary
        dict(name="distill_bwd_4096x50021_bf16", op="distill_bwd", N=4096, V=50021, K=128, dtype="bf16", grad="bf16",
             tau=1.0, masked=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "recur_fwd", "recur_bwd", "recur_step", "distill_fwd", "distill_bwd",
                     "distill_step"])
    dtype = rng.choice(["f32", "bf16"])
    if op.startswith("embed"):
        V, D = _log_int(rng, 1000, 131072), _log_int(rng, 64, 4096)
        while V * D > 1 << 28:
            V, D = _log_int(rng, 1000, 131072), _log_int(rng, 64, 4096)
        N = _log_int(rng, 1, min(131072, (1 << 27) // D))
        return dict(op=op, N=N, V=V, D=D, dtype=dtype, ids=rng.choice(["zipf", "uniform"]),
                    pad=rng.choice([0.0, 0.1, 0.5]))
    if op == "recur_step":
        B = _log_int(rng, 1, 1024)
        return dict(op=op, B=B, S=B + _log_int(rng, 1, 1024), D=_log_int(rng, 64, 4096), dtype=dtype,
                    packed=rng.random() < 0.5)
    if op.startswith("recur"):
        while True:
            B, T, D = _log_int(rng, 1, 64), _log_int(rng, 1, 65536), _log_int(rng, 64, 4096)
            if B * T * D <= 1 << 26:
                break
        c = dict(op=op, B=B, T=T, D=D, dtype=dtype, packed=rng.random() < 0.5, h0=rng.random() < 0.5,
                 ragged=rng.random() < 0.5)
        if op == "recur_bwd":
            c["grad"] = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
        return c
    V = _log_int(rng, 1000, 131072)
    c = dict(op=op, N=_log_int(rng, 1, min(16384, (1 << 29) // V)), V=V, K=_log_int(rng, 1, 256), dtype=dtype,
             tau=rng.choice([1.0, 2.0, 4.0]), masked=rng.choice([0.0, 0.1, 0.5]))
    if op != "distill_fwd":
        c["grad"] = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
    return c


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(int(seed))
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, device=_DEV, generator=gen)

    def uniform(*shape):
        return torch.rand(shape, device=_DEV, generator=gen)

    dt = _DT[case["dtype"]]
    if case["op"].startswith("embed"):
        N, V, D = case["N"], case["V"], case["D"]
        u = uniform(N).double()
        if case["ids"] == "zipf":       # frequency about 1 / rank, ranks in the order of the ids
            ids = ((V + 1.0) ** u).long() - 1
        else:
            ids = (u * V).long()
        ids = ids.clamp_(0, V - 1)
        pad = uniform(N) < case["pad"]
        pad[0] = False
        s["ids"] = torch.where(pad, torch.full_like(ids, -1), ids)
        s["scale"] = math.sqrt(D)
        if case["op"] == "embed_fwd":
            s["table"] = (normal(V, D) * 0.02).to(dt)
        else:
            s["dy"] = normal(N, D).mul_(1e-3).to(dt)
        return s
    if case["op"] == "recur_step":
        B, S, D = case["B"], case["S"], case["D"]
        _inputs(s, normal, (B, D), dt, case["packed"])
        s["state"] = normal(S, D)
        s["slots"] = torch.randperm(S, device=_DEV, generator=gen)[:B].to(torch.int32)
        return s
    if case["op"].startswith("recur"):
        B, T, D = case["B"], case["T"], case["D"]
        _inputs(s, normal, (B, T, D), dt, case["packed"])
        s["h0"] = normal(B, D) if case["h0"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = (uniform(B) * (T + 1)).int().clamp_(max=T)
            n[0] = T
            if B > 2:
                n[B // 2] = 0
            s["lengths"] = n
        if case["op"] == "recur_bwd":
            s["y"] = _recur_forward(s["x"], s["g"], s["h0"], s["lengths"])[0]
            s["dy"] = normal(B, T, D)
            s["dhT"] = normal(B, D) if case["h0"] else None
        return s
    N, V, K = case["N"], case["V"], case["K"]
    z = normal(N, V).mul_(2.5)
    t, ids = torch.topk(z + 0.0 if N * V > 1 << 24 else z + normal(N, V), min(K, V), dim=1)
    s["t"] = t + normal(N, t.shape[1])
    s["ids"] = ids
    s["z"] = z.to(dt)
    s["weight"] = (uniform(N) >= case["masked"]).float() / N
    s["weight"][0] = 1.0 / N
    if case["op"] == "distill_bwd":
        s["lse"] = _log_sum_exp(s["z"].float() / case["tau"])
        s["dloss"] = uniform(N) + 0.5
    return s


def _inputs(s, normal, shape, dt, packed):
    """x and g: two arrays, or the halves of one array as a layer of twice the width writes it."""
    D = shape[-1]
    p = normal(*shape[:-1], 2 * D)
    p[..., D:].mul_(1.5).add_(2.0)       # gates: most of the state kept, memories from a few steps to hundreds
    p = p.to(dt)
    if packed:
        s["x"], s["g"] = p[..., :D], p[..., D:]
    else:
        s["x"], s["g"] = p[..., :D].contiguous(), p[..., D:].contiguous()


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


# ---- the package's kernels ---------------------------------------------------

def _run_own(s):
    import kolmogorov_arnold_network_amd as kan

    op = s["op"]
    if op == "embed_fwd":
        return kan.kan_embed_forward(s["ids"], s["table"], s["scale"])
    if op == "embed_bwd":
        return kan.kan_embed_backward(s["ids"], s["dy"], s["V"], s["scale"])
    if op == "recur_step":
        return [kan.kan_recur_step(s["x"], s["g"], s["state"], slots=s["slots"]), s["state"]]
    if op == "recur_fwd":
        return list(kan.kan_recur_forward(s["x"], s["g"], h0=s["h0"], lengths=s["lengths"]))
    if op == "recur_bwd":
        B, T, D = s["x"].shape
        dt = _DT[s["grad"]]
        if s["packed"]:
            dp = torch.empty((B, T, 2 * D), dtype=dt, device=_DEV)
            dx, dg = dp[..., :D], dp[..., D:]
        else:
            dx, dg = torch.empty((2, B, T, D), dtype=dt, device=_DEV)
        dh0 = kan.kan_recur_backward(s["x"], s["g"], s["y"], s["dy"], h0=s["h0"], lengths=s["lengths"],
                                     dhT=s["dhT"], dx=dx, dg=dg)[2]
        return [dx, dg, dh0]
    if op == "distill_fwd":
        return list(kan.kan_distill_forward(s["z"], s["ids"], s["t"], s["tau"], weight=s["weight"]))
    if op == "distill_bwd":
        return kan.kan_distill_backward(s["z"], s["ids"], s["t"], s["lse"], s["dloss"], s["tau"], weight=s["weight"],
                                        grad_dtype=_DT[s["grad"]])
    return list(kan.kan_distill_step(s["z"], s["ids"], s["t"], s["tau"], weight=s["weight"],
                                     grad_dtype=_DT[s["grad"]]))


# ---- plain forms: elementary float32 operations ---------------------------------

def _embed_fwd(s):
    ids, table = s["ids"], s["table"]
    rows = table[ids.clamp(min=0)].float() * s["scale"]
    return torch.where((ids >= 0)[:, None], rows, torch.zeros_like(rows)).to(table.dtype)


def _embed_bwd(s):
    ids = s["ids"]
    rows = torch.where((ids >= 0)[:, None], s["dy"].float() * s["scale"], 0.0)
    return torch.zeros(s["V"], s["D"], device=_DEV).index_add_(0, ids.clamp(min=0), rows)


def _gates(g):
    g = g.float()
    return 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))       # f, 1 - f


def _scan(a, b):
    """b[:, t] + a[:, t] * (the same at t - 1) along dim 1: runs of 1, 2, 4, ... steps joined to their neighbours."""
    k, T = 1, b.shape[1]
    while k < T:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _inside(lengths, T):
    return None if lengths is None else (torch.arange(T, device=_DEV)[None, :] < lengths[:, None])[..., None]


def _recur_forward(x, g, h0, lengths):
    f, u = _gates(g)
    b = u * x.float()
    if h0 is not None:
        b[:, 0] += f[:, 0] * h0
    y = _scan(f, b)
    if lengths is None:
        return y, y[:, -1].clone()
    rows = torch.arange(x.shape[0], device=_DEV)
    last = y[rows, (lengths.long() - 1).clamp(min=0)]
    start = torch.zeros_like(last) if h0 is None else h0
    return torch.where(_inside(lengths, x.shape[1]), y, 0.0), torch.where((lengths > 0)[:, None], last, start)


def _recur_fwd(s):
    return list(_recur_forward(s["x"], s["g"], s["h0"], s["lengths"]))


def _recur_bwd(s):
    B, T, D = s["x"].shape
    f, u = _gates(s["g"])
    inside = _inside(s["lengths"], T)
    e = s["dy"] if inside is None else torch.where(inside, s["dy"], 0.0)
    if s["dhT"] is not None:
        n = torch.full((B,), T, device=_DEV) if s["lengths"] is None else s["lengths"].long()
        last = torch.where((n > 0)[:, None], s["dhT"], 0.0)
        e = e.index_put((torch.arange(B, device=_DEV), (n - 1).clamp(min=0)), last, accumulate=True)
    a = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1)
    d = _scan(a.flip(1), e.flip(1)).flip(1)
    start = torch.zeros((B, 1, D), device=_DEV) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([start, s["y"][:, :-1]], 1)
    dx, dg = u * d, f * u * (before - s["x"].float()) * d
    if inside is not None:
        dx, dg = torch.where(inside, dx, 0.0), torch.where(inside, dg, 0.0)
    dh0 = f[:, 0] * d[:, 0]
    if s["lengths"] is not None:
        through = torch.zeros_like(dh0) if s["dhT"] is None else s["dhT"]
        dh0 = torch.where((s["lengths"] > 0)[:, None], dh0, through)
    dt = _DT[s["grad"]]
    return [dx.to(dt), dg.to(dt), dh0 if s["h0"] is not None else None]


def _recur_step(s):
    f, u = _gates(s["g"])
    slots = s["slots"].long()
    h = f * s["state"][slots] + u * s["x"].float()
    s["state"][slots] = h
    return [h, s["state"]]


def _log_sum_exp(v):
    m = v.amax(1, keepdim=True)
    return (m + torch.exp(v - m).sum(1, keepdim=True).log())[:, 0]


def _teacher(s):
    t = s["t"].float() / s["tau"]
    log_p = t - _log_sum_exp(t)[:, None]
    return log_p, torch.exp(log_p)


def _distill_loss(s, v, lse):
    log_p, p = _teacher(s)
    return s["weight"] * s["tau"] ** 2 * (p * (log_p - v.gather(1, s["ids"]) + lse[:, None])).sum(1)


def _distill_grad(s, v, lse, scale):
    d = torch.exp(v - lse[:, None]).scatter_add_(1, s["ids"], -_teacher(s)[1])
    return (d * (s["weight"] * s["tau"] * scale)[:, None]).to(_DT[s["grad"]])


def _distill_fwd(s):
    v = s["z"].float() / s["tau"]
    lse = _log_sum_exp(v)
    return [_distill_loss(s, v, lse), lse]


def _distill_bwd(s):
    return _distill_grad(s, s["z"].float() / s["tau"], s["lse"], s["dloss"])


def _distill_step(s):
    v = s["z"].float() / s["tau"]
    lse = _log_sum_exp(v)
    return [_distill_loss(s, v, lse), _distill_grad(s, v, lse, 1.0)]


_PLAIN = dict(embed_fwd=_embed_fwd, embed_bwd=_embed_bwd, recur_fwd=_recur_fwd, recur_bwd=_recur_bwd,
              recur_step=_recur_step, distill_fwd=_distill_fwd, distill_bwd=_distill_bwd, distill_step=_distill_step)


# ---- what a pass cannot do without -----------------------------------------------

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op.startswith("embed"):
        N, V, D = case["N"], case["V"], case["D"]
        kept = N * (1.0 - case["pad"])
        if op == "embed_bwd":
            return {"bytes": 8 * N + kept * D * e + 4 * V * D, "flops": 2 * kept * D}
        if case["ids"] == "zipf":
            rows = sum(1.0 - math.exp(kept * math.log1p(-math.log((r + 2) / (r + 1)) / math.log(V + 1)))
                       for r in range(V))
        else:
            rows = V * -math.expm1(kept * math.log1p(-1.0 / V))
        return {"bytes": 8 * N + (rows + N) * D * e, "flops": kept * D}
    if op == "recur_step":
        n = case["B"] * case["D"]
        return {"bytes": n * (2 * e + 12) + 4 * case["B"], "flops": 10 * n}
    if op.startswith("recur"):
        B, T, D = case["B"], case["T"], case["D"]
        n, share = B * T * D, 0.5 if case["ragged"] else 1.0     # lengths are uniform: half of the rows on average
        state = 4 * B * D * (2 if case["h0"] else 1)
        if op == "recur_fwd":
            return {"bytes": n * (2 * e * share + 4) + state, "flops": 12 * n * share}
        return {"bytes": n * ((2 * e + 8) * share + 2 * _size(case["grad"])) + 1.5 * state, "flops": 20 * n * share}
    N, V, K = case["N"], case["V"], case["K"]
    kept = N * (1.0 - case["masked"])
    small = 12 * N + kept * 12 * K
    read = kept * V * e
    write = 0 if op == "distill_fwd" else N * V * _size(case["grad"])
    return {"bytes": read + write + small, "flops": kept * V * (4 if op == "distill_fwd" else 6)}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        keep = s["ids"] >= 0
        y = torch.zeros(case["N"], case["D"], dtype=torch.float64, device=_DEV)
        y[keep] = s["table"].index_select(0, s["ids"][keep]).double() * s["scale"]
        return y
    if op == "embed_bwd":
        # rows in the order of their tokens, running sums, differences at the tokens' ends
        keep = s["ids"] >= 0
        ids, order = torch.sort(s["ids"][keep])
        run_sum = torch.cumsum(s["dy"][keep].double()[order], 0)
        token, count = torch.unique_consecutive(ids, return_counts=True)
        at = run_sum[torch.cumsum(count, 0) - 1]
        dE = torch.zeros(case["V"], case["D"], dtype=torch.float64, device=_DEV)
        dE[token] = s["scale"] * torch.cat([at[:1], at[1:] - at[:-1]])
        return dE
    if op == "recur_step":
        slots = s["slots"].long()
        h = s["state"].double()
        u = torch.sigmoid(-s["g"].double())
        new = h[slots] + u * (s["x"].double() - h[slots])
        h[slots] = new
        return [new, h]
    if op.startswith("recur"):
        return _exact_recur(s, case)
    z, tau = s["z"].double() / case["tau"], case["tau"]
    t = s["t"].double() / tau
    p = torch.softmax(t, 1)
    log_q = torch.log_softmax(z, 1)
    if op in ("distill_fwd", "distill_step"):
        loss = s["weight"].double() * tau * tau * (p * (torch.log_softmax(t, 1) - log_q.gather(1, s["ids"]))).sum(1)
    if op == "distill_fwd":
        return [loss, torch.logsumexp(z, 1)]
    scale = s["weight"].double() * tau * (s["dloss"].double() if op == "distill_bwd" else 1.0)
    rows = torch.arange(case["N"], device=_DEV)[:, None]
    d = log_q.exp_()
    d[rows, s["ids"]] -= p                # a teacher's ids are distinct
    d *= scale[:, None]
    return d if op == "distill_bwd" else [loss, d]


def _exact_recur(s, case):
    """Step by step along the sequences."""
    B, T, D = case["B"], case["T"], case["D"]
    n = torch.full((B,), T, device=_DEV) if s["lengths"] is None else s["lengths"].long()
    h = torch.zeros(B, D, dtype=torch.float64, device=_DEV) if s["h0"] is None else s["h0"].double()
    hs = torch.zeros(B, T + 1, D, dtype=torch.float64, device=_DEV)
    hs[:, 0] = h
    on = (torch.arange(T, device=_DEV)[:, None] < n[None, :])[..., None]
    full = s["lengths"] is None
    for t in range(T):
        new = torch.lerp(h, s["x"][:, t].double(), torch.sigmoid(-s["g"][:, t].double()))
        h = new if full else torch.where(on[t], new, h)
        hs[:, t + 1] = h
    if case["op"] == "recur_fwd":
        return [hs[:, 1:] * on.transpose(0, 1), h]
    d = torch.zeros(B, D, dtype=torch.float64, device=_DEV) if s["dhT"] is None else s["dhT"].double()
    dx = torch.zeros(B, T, D, dtype=torch.float64, device=_DEV)
    dg = torch.zeros_like(dx)
    for t in reversed(range(T)):
        f = torch.sigmoid(s["g"][:, t].double())
        u = torch.sigmoid(-s["g"][:, t].double())
        here = d + s["dy"][:, t].double()
        here = here if full else here * on[t]
        dx[:, t] = u * here
        dg[:, t] = f * u * (hs[:, t] - s["x"][:, t].double()) * here
        d = f * here if full else torch.where(on[t], f * here, d)
    return [dx, dg, d if s["h0"] is not None else None]
