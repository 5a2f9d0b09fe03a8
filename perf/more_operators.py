"""Cases and plain forms of the gated delta rule and of the join between blocks.

``delta`` mixes the rows of a sequence through a matrix of states a head; ``join``
puts a block's output through its norm and gate onto the residual rows and
normalises those for the next block.  ``run`` computes one pass in elementary
float32 torch operations (``own`` false) or with the package's kernels (``own``
true); ``exact`` computes the same from the definitions in 64 bits: the delta
rule row by row, where the plain form goes by chunks.
"""

import math

import torch

own = False

_DEV = "cuda:0"
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_CHUNK = 64
_UNIT_EPS = 1e-6
_EPS = 1e-6


def listed():
    return [
        # one new token for one sequence of a small model: latency
        dict(name="delta_step_1x4x64_f32", op="delta_step", B=1, S=16, Hk=4, Hv=4, Dk=64, Dv=64, dtype="f32", unit=True,
             packed=True),
        # one new token for 64 of 96 served sequences
        dict(name="delta_step_64x16x128_bf16", op="delta_step", B=64, S=96, Hk=16, Hv=16, Dk=128, Dv=128, dtype="bf16",
             unit=True, packed=False),
        # a training batch of 8 sequences of 4096 tokens, 16 heads
        dict(name="delta_fwd_8x4096x16x128_bf16", op="delta_fwd", B=8, T=4096, Hk=16, Hv=16, Dk=128, Dv=128,
             dtype="bf16", unit=True, packed=False, h0=False, ragged=False),
        # one long document, continued from a state, heads sharing keys, slices of one projection
        dict(name="delta_fwd_1x32768x8x128_f32", op="delta_fwd", B=1, T=32768, Hk=4, Hv=8, Dk=128, Dv=128, dtype="f32",
             unit=True, packed=True, h0=True, ragged=False),
        # a padded batch of unequal sequences (one of them empty), odd heads
        dict(name="delta_fwd_7x1531x6x72x104_bf16", op="delta_fwd", B=7, T=1531, Hk=3, Hv=6, Dk=72, Dv=104,
             dtype="bf16", unit=False, packed=False, h0=True, ragged=True),
        # the training batch's backward pass
        dict(name="delta_bwd_4x4096x16x128_bf16", op="delta_bwd", B=4, T=4096, Hk=16, Hv=16, Dk=128, Dv=128,
             dtype="bf16", unit=True, packed=False, h0=False, ragged=False),
        # gradients of a small float32 model on unequal sequences, odd heads, slices of one projection
        dict(name="delta_bwd_5x777x4x48x80_f32", op="delta_bwd", B=5, T=777, Hk=2, Hv=4, Dk=48, Dv=80, dtype="f32",
             unit=True, packed=True, h0=True, ragged=True),
        # the rows of 64 sequences being served, with everything a join has: latency
        dict(name="join_fwd_64x2048_f32", op="join_fwd", N=64, D=2048, dtype="f32", res="f32", row="f32", post=True,
             gate="silu", r=True, pre=True, weights=True),
        # a training batch of 8 sequences of 4096 tokens: bf16 blocks on float32 residual rows
        dict(name="join_fwd_32768x2048_bf16", op="join_fwd", N=32768, D=2048, dtype="bf16", res="f32", row="bf16",
             post=True, gate="none", r=True, pre=True, weights=True),
        # heads on their way out of the delta rule: a norm and a gate for each head of the batch
        dict(name="join_fwd_524288x128_bf16", op="join_fwd", N=524288, D=128, dtype="bf16", res="bf16", row="bf16",
             post=True, gate="silu", r=False, pre=False, weights=True),
        # the training batch's backward pass, float32 layers
        dict(name="join_bwd_32768x2048_f32", op="join_bwd", N=32768, D=2048, dtype="f32", res="f32", row="f32",
             post=True, gate="silu", r=True, pre=True, weights=True),
        # a ragged batch's rows of odd width
        dict(name="join_bwd_4999x770_bf16", op="join_bwd", N=4999, D=770, dtype="bf16", res="bf16", row="bf16",
             post=True, gate="sigmoid", r=True, pre=True, weights=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step", "join_fwd", "join_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op.startswith("join"):
        D = _log_int(rng, 16, 8192)
        N = _log_int(rng, 1, min(1 << 20, (1 << 26) // D))
        c = dict(op=op, N=N, D=D, dtype=dtype, res=rng.choice(["f32", dtype]), row=dtype,
                 gate=rng.choice(["none", "sigmoid", "silu"]), r=rng.random() < 0.7, weights=rng.random() < 0.8)
        c["post"], c["pre"] = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return c
    while True:
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hk * rng.choice([1, 1, 2, 4])
        Dk, Dv = _log_int(rng, 16, 128), _log_int(rng, 16, 256)
        if op == "delta_step":
            B = _log_int(rng, 1, 256)
            c = dict(op=op, B=B, S=B + _log_int(rng, 1, 64), Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype)
            if c["S"] * Hv * Dk * Dv > 1 << 26:
                continue
        else:
            B, T = _log_int(rng, 1, 16), _log_int(rng, 1, 16384)
            if B * T * Hv * max(Dk, Dv) > (1 << 25 if op == "delta_fwd" else 1 << 24):
                continue
            c = dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, h0=rng.random() < 0.5,
                     ragged=rng.random() < 0.5)
        c["unit"], c["packed"] = rng.random() < 0.7, rng.random() < 0.5
        return c


# ---- inputs ----------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(int(seed))
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, device=_DEV, generator=gen)

    dt = _DT[case["dtype"]]
    if case["op"].startswith("join"):
        N, D = case["N"], case["D"]
        s["h"] = (normal(N, D) * (0.5 + torch.rand((N, 1), device=_DEV, generator=gen))).to(dt)
        s["gate_rows"] = normal(N, D).to(dt) if case["gate"] != "none" else None
        s["r"] = (normal(N, D) * 2.0).to(_DT[case["res"]]) if case["r"] else None
        s["w_post"] = 1.0 + 0.2 * normal(D) if case["weights"] else None
        s["w_pre"] = 1.0 + 0.2 * normal(D) if case["weights"] and case["pre"] else None
        s["factor"] = 0.5 if case["r"] else 1.0
        if case["op"] == "join_bwd":
            y, _, s["stats"] = _join_rows(s)
            s["y"] = y.to(_DT[case["res"]])
            s["dy"] = (normal(N, D) * 1e-2).to(_DT[case["res"]]) if case["r"] or not case["pre"] else None
            s["dx"] = (normal(N, D) * 1e-2).to(_DT[case["row"]]) if case["pre"] else None
        return s
    B, T = case["B"], case.get("T", 1)
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    q, k, v = normal(B, T, Hk, Dk), normal(B, T, Hk, Dk), normal(B, T, Hv, Dv)
    if not case["unit"]:                    # made unit by the caller
        q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    if case["packed"]:                      # slices of one projection's rows
        p = torch.cat([q.reshape(B, T, Hk * Dk), k.reshape(B, T, Hk * Dk), v.reshape(B, T, Hv * Dv)], -1).to(dt)
        s["q"], s["k"], s["v"] = _slices(p, s)
    else:
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), v.to(dt)
    # decays: memories from a few rows to some hundred, a level of its own for each head
    level = 4.0 + 1.5 * normal(Hv)
    s["g"] = torch.nn.functional.logsigmoid(level + normal(B, T, Hv))
    s["beta"] = torch.sigmoid(normal(B, T, Hv))
    if case["op"] == "delta_step":
        for name in ("q", "k", "v", "g", "beta"):
            s[name] = s[name][:, 0]
        s["state"] = normal(case["S"], Hv, Dk, Dv) * 0.3
        s["slots"] = torch.randperm(case["S"], device=_DEV, generator=gen)[:B].to(torch.int32)
        return s
    s["start"] = normal(B, Hv, Dk, Dv) * 0.3 if case["h0"] else None
    s["lengths"] = None
    if case["ragged"]:
        n = (torch.rand(B, device=_DEV, generator=gen) * (T + 1)).int().clamp_(max=T)
        n[0] = T
        if B > 2:
            n[B // 2] = 0
        s["lengths"] = n
    if case["op"] == "delta_bwd":
        s["dy"] = normal(B, T, Hv, Dv).to(dt)
        s["dhT"] = normal(B, Hv, Dk, Dv) * 0.3 if case["h0"] else None
    return s


def _slices(p, s):
    """q, k and v as slices of the rows p [B, T, 2 Hk Dk + Hv Dv]."""
    n = s["Hk"] * s["Dk"]
    lead = p.shape[:2]
    return (p[..., :n].unflatten(-1, (s["Hk"], s["Dk"])), p[..., n:2 * n].unflatten(-1, (s["Hk"], s["Dk"])),
            p[..., 2 * n:].view(*lead, s["Hv"], s["Dv"]))


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


# ---- the package's kernels ---------------------------------------------------------

def _run_own(s):
    import kolmogorov_arnold_network_amd as kan

    op = s["op"]
    if op == "delta_step":
        y = kan.kan_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], unit=s["unit"])
        return [y, s["state"]]
    if op == "delta_fwd":
        return list(kan.kan_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["start"],
                                          lengths=s["lengths"], unit=s["unit"]))
    if op == "delta_bwd":
        dq = dk = dv = None
        if s["packed"]:
            dp = torch.empty((*s["v"].shape[:2], 2 * s["Hk"] * s["Dk"] + s["Hv"] * s["Dv"]), dtype=s["q"].dtype,
                             device=_DEV)
            dq, dk, dv = _slices(dp, s)
        return list(kan.kan_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], h0=s["start"],
                                           lengths=s["lengths"], dhT=s["dhT"], unit=s["unit"], dq=dq, dk=dk, dv=dv))
    if op == "join_fwd":
        return list(kan.kan_join_forward(s["h"], s["r"], s["gate_rows"], s["w_post"], s["w_pre"], post=s["post"],
                                         pre=s["pre"], activation=_activation(s), scale=s["factor"], eps=_EPS,
                                         res_dtype=_DT[s["res"]], row_dtype=_DT[s["row"]]))
    return list(kan.kan_join_backward(s["h"], s["y"], s["stats"], s["dy"], s["dx"], s["gate_rows"], s["w_post"],
                                      s["w_pre"], post=s["post"], activation=_activation(s), scale=s["factor"],
                                      need_dr=s["r"] is not None))


def _activation(s):
    return "silu" if s["gate"] == "none" else s["gate"]


# ---- plain forms: elementary float32 operations -------------------------------------

def _unit(x):
    return 1.0 / (x.square().sum(-1, keepdim=True) + _UNIT_EPS).sqrt()


def _delta_step(s):
    q, k = s["q"].float(), s["k"].float()
    if s["unit"]:
        q, k = q * _unit(q), k * _unit(k)
    share = s["Hv"] // s["Hk"]
    q, k = (x.repeat_interleave(share, 1)[..., None] for x in (q, k))
    slots = s["slots"].long()
    state = s["state"][slots] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (state * k).sum(-2))
    state = state + k * u[..., None, :]
    s["state"][slots] = state
    return [((state * q).sum(-2) / math.sqrt(s["Dk"])).to(s["q"].dtype), s["state"]]


def _in_chunks(x, inside, heads):
    """[B, T, H, D] as float32 [B, heads, chunks, 64, D], zero past the sequences' ends."""
    B, T, H, D = x.shape
    x = x.float() if inside is None else torch.where(inside[:, :, None, None], x.float(), 0.0)
    x = torch.cat([x, x.new_zeros(B, -T % _CHUNK, H, D)], 1)
    return x.transpose(1, 2).reshape(B, H, -1, _CHUNK, D).repeat_interleave(heads // H, 1)


def _from_chunks(x, T):
    B, H, D = x.shape[0], x.shape[1], x.shape[-1]
    return x.reshape(B, H, -1, D)[:, :, :T].transpose(1, 2)


def _delta_parts(s):
    """What a chunk's rows have among themselves."""
    T, Hv = s["T"], s["Hv"]
    inside = None
    if s["lengths"] is not None:
        inside = torch.arange(T, device=_DEV)[None, :] < s["lengths"][:, None]
    p = {"q": _in_chunks(s["q"], inside, Hv), "k": _in_chunks(s["k"], inside, Hv), "v": _in_chunks(s["v"], inside, Hv)}
    for x in "qk":
        p["n" + x] = _unit(p[x]) if s["unit"] else 1.0
        p[x] = p[x] * p["n" + x]
    p["beta"] = _in_chunks(s["beta"][..., None], inside, Hv)
    c = torch.cumsum(_in_chunks(s["g"][..., None], inside, Hv)[..., 0].double(), -1)   # 64 bits: differences of long sums
    lower = torch.ones(_CHUNK, _CHUNK, device=_DEV, dtype=torch.bool).tril()
    D = torch.where(lower, c[..., :, None] - c[..., None, :], -math.inf).exp().float()
    p["from_start"] = c.exp().float()[..., None]
    p["to_end"] = (c[..., -1:] - c).exp().float()[..., None]
    p["whole"] = c[..., -1].exp().float()[..., None, None]
    p["D"], p["strict"] = D, lower.tril(-1)
    p["scale"] = 1.0 / math.sqrt(s["Dk"])
    kt = p["k"].transpose(-1, -2)
    p["P"] = p["scale"] * (p["q"] @ kt) * D
    p["A"] = torch.where(p["strict"], (p["k"] @ kt) * D, 0.0)
    G, A, beta = torch.zeros_like(D), p["A"], p["beta"]
    for r in range(1, _CHUNK):              # G = A - A diag(beta) G, row after row
        G[..., r:r + 1, :] = A[..., r:r + 1, :] - A[..., r:r + 1, :r] @ (beta[..., :r, :] * G[..., :r, :])
    p["G"] = G
    return p


def _delta_chunks(s, p):
    """Rows, corrections w, the chunks' first states and the last one."""
    B, Hv, n = p["q"].shape[:3]
    S = torch.zeros(B, Hv, s["Dk"], s["Dv"], device=_DEV) if s["start"] is None else s["start"]
    y, w, states = [], [], []
    for i in range(n):
        states.append(S)
        f, beta = p["from_start"][:, :, i], p["beta"][:, :, i]
        e = p["v"][:, :, i] - f * (p["k"][:, :, i] @ S)
        w.append(e - p["G"][:, :, i] @ (beta * e))
        u = beta * w[-1]
        y.append(p["scale"] * f * (p["q"][:, :, i] @ S) + p["P"][:, :, i] @ u)
        S = p["whole"][:, :, i] * S + (p["to_end"][:, :, i] * p["k"][:, :, i]).transpose(-1, -2) @ u
    return torch.stack(y, 2), torch.stack(w, 2), torch.stack(states, 2), S


def _delta_fwd(s):
    y, _, _, S = _delta_chunks(s, _delta_parts(s))
    return [_from_chunks(y, s["T"]).to(s["q"].dtype), S]


def _delta_bwd(s):
    T, Hk, Hv = s["T"], s["Hk"], s["Hv"]
    inside = None
    if s["lengths"] is not None:
        inside = torch.arange(T, device=_DEV)[None, :] < s["lengths"][:, None]
    p = _delta_parts(s)
    q, k, scale = p["q"], p["k"], p["scale"]
    _, w, S0, _ = _delta_chunks(s, p)
    dy = _in_chunks(s["dy"], inside, Hv)
    n = q.shape[2]
    dS = torch.zeros_like(S0[:, :, 0]) if s["dhT"] is None else s["dhT"]
    r, dS1 = [None] * n, [None] * n
    for i in reversed(range(n)):
        dS1[i] = dS
        f, beta = p["from_start"][:, :, i], p["beta"][:, :, i]
        du = p["P"][:, :, i].transpose(-1, -2) @ dy[:, :, i] + p["to_end"][:, :, i] * (k[:, :, i] @ dS)
        r[i] = du - p["G"][:, :, i].transpose(-1, -2) @ (beta * du)
        dS = (p["whole"][:, :, i] * dS + scale * (f * q[:, :, i]).transpose(-1, -2) @ dy[:, :, i]
              - (f * k[:, :, i]).transpose(-1, -2) @ (beta * r[i]))
    r, dS1 = torch.stack(r, 2), torch.stack(dS1, 2)
    u, dv = p["beta"] * w, p["beta"] * r
    dP = dy @ u.transpose(-1, -2)
    X = torch.where(p["strict"], dv @ u.transpose(-1, -2), 0.0)
    q_start = scale * p["from_start"] * (dy @ S0.transpose(-1, -2))
    k_start = -p["from_start"] * (dv @ S0.transpose(-1, -2))
    k_end = p["to_end"] * (u @ dS1.transpose(-1, -2))
    PD, XD = scale * dP * p["D"], X * p["D"]
    dq = q_start + PD @ k
    dk = PD.transpose(-1, -2) @ q + k_start + k_end - XD @ k - XD.transpose(-1, -2) @ k
    # the decay of a row: all pairs of rows that it stands between
    E = dP * p["P"] - X * p["A"]
    before = torch.cumsum(E, -1) - E
    dg = before.tril().sum(-2)
    x = (q * q_start + k * k_start).sum(-1)
    z = (k * k_end).sum(-1)
    dg = dg + x.flip(-1).cumsum(-1).flip(-1) + z.cumsum(-1) - z
    dg = dg + (p["whole"] * dS1 * S0).sum((-1, -2))[..., None]
    dbeta = (r * w).sum(-1)
    dq, dk = (d.unflatten(1, (Hk, Hv // Hk)).sum(2) for d in (dq, dk))
    if s["unit"]:
        first = slice(None, None, Hv // Hk)
        dq, dk = (p["n" + m][:, first] * (d - h[:, first] * (h[:, first] * d).sum(-1, keepdim=True))
                  for m, h, d in (("q", q, dq), ("k", k, dk)))
    dt = s["q"].dtype
    dq, dk, dv = (_from_chunks(d, T) for d in (dq, dk, dv))
    dg, dbeta = (_from_chunks(d[..., None], T)[..., 0] for d in (dg, dbeta))
    if inside is not None:
        dg, dbeta = (torch.where(inside[..., None], d, 0.0) for d in (dg, dbeta))
    return [dq.to(dt), dk.to(dt), dv.to(dt), dg, dbeta, dS if s["start"] is not None else None]


def _rstd(x):
    return 1.0 / (x.square().mean(-1, keepdim=True) + _EPS).sqrt()


def _act(s, g):
    sig = 1.0 / (1.0 + torch.exp(-g))
    return sig if s["gate"] == "sigmoid" else g * sig


def _join_rows(s):
    """float32 y, x and the norms' factors [2, N] (1 where there is no norm)."""
    h = s["h"].float()
    n1 = _rstd(h) if s["post"] else torch.ones_like(h[:, :1])
    p = h * n1
    if s["w_post"] is not None:
        p = p * s["w_post"]
    if s["gate_rows"] is not None:
        p = p * _act(s, s["gate_rows"].float())
    y = s["factor"] * p
    if s["r"] is not None:
        y = y + s["r"].float()
    n2 = _rstd(y) if s["pre"] else torch.ones_like(h[:, :1])
    x = y * n2 if s["pre"] else None
    if s["w_pre"] is not None:
        x = x * s["w_pre"]
    return y, x, torch.cat([n1, n2], 1).t().contiguous()


def _join_fwd(s):
    y, x, stats = _join_rows(s)
    return [y.to(_DT[s["res"]]), None if x is None else x.to(_DT[s["row"]]), stats]


def _join_bwd(s):
    n1, n2 = s["stats"][0][:, None], s["stats"][1][:, None]
    d = 0.0 if s["dy"] is None else s["dy"].float()
    dw_pre = None
    if s["dx"] is not None:
        z = s["y"].float() * n2
        c = s["dx"].float()
        if s["w_pre"] is not None:
            dw_pre = (c * z).sum(0)
            c = c * s["w_pre"]
        d = d + n2 * (c - z * (c * z).mean(-1, keepdim=True))
    t = s["h"].float() * n1
    p = t if s["w_post"] is None else t * s["w_post"]
    dp, dgate = s["factor"] * d, None
    if s["gate_rows"] is not None:
        g = s["gate_rows"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        slope = sig * (1.0 - sig) if s["gate"] == "sigmoid" else sig * (1.0 + g * (1.0 - sig))
        dgate = (dp * p * slope).to(s["h"].dtype)
        dp = dp * _act(s, g)
    dw_post = None if s["w_post"] is None else (dp * t).sum(0)
    dt = dp if s["w_post"] is None else dp * s["w_post"]
    dh = n1 * (dt - t * (dt * t).mean(-1, keepdim=True)) if s["post"] else dt
    dr = d.to(s["y"].dtype) if s["r"] is not None else None
    return [dh.to(s["h"].dtype), dr, dgate, dw_post, dw_pre]


_PLAIN = dict(delta_fwd=_delta_fwd, delta_bwd=_delta_bwd, delta_step=_delta_step, join_fwd=_join_fwd,
              join_bwd=_join_bwd)


# ---- what a pass cannot do without -----------------------------------------------------

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op.startswith("join"):
        n, res, row = case["N"] * case["D"], _size(case["res"]), _size(case["row"])
        inputs = e * (2 if case["gate"] != "none" else 1)
        weights = 4 * case["D"] * (1 + case["pre"]) * case["weights"]
        if op == "join_fwd":
            each = inputs + res * (2 if case["r"] else 1) + (row if case["pre"] else 0)
            return {"bytes": n * each + 8 * case["N"] + weights, "flops": 12 * n}
        given = res * (case["r"] or not case["pre"]) + (row + res if case["pre"] else 0)
        each = 2 * inputs + given + (res if case["r"] else 0)
        return {"bytes": n * each + 8 * case["N"] + 2 * weights, "flops": 30 * n}
    B, T, Hk, Hv, Dk, Dv = case["B"], case.get("T", 1), case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    rows, state = B * T * (0.5 if case.get("ragged") else 1.0), 4 * B * Hv * Dk * Dv     # ragged: half on average
    row_in = e * (2 * Hk * Dk + Hv * Dv) + 8 * Hv
    if op == "delta_step":
        return {"bytes": rows * (row_in + e * Hv * Dv) + 2 * state, "flops": 8 * rows * Hv * Dk * Dv}
    if op == "delta_fwd":
        return {"bytes": rows * row_in + B * T * e * Hv * Dv + state * (1 + case["h0"]),
                "flops": 6 * rows * Hv * Dk * Dv}
    return {"bytes": rows * (row_in + e * Hv * Dv) + B * T * row_in + 3 * state * case["h0"],
            "flops": 18 * rows * Hv * Dk * Dv}


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "join_fwd":
        return _exact_join_fwd(s)
    if op == "join_bwd":
        return _exact_join_bwd(s)
    if op == "delta_step":
        state = s["state"].double()
        slots = s["slots"].long()
        q, k, _, _ = _exact_heads(s)
        y, state[slots] = _exact_row(state[slots], q, k, s["v"].double(), s["g"].double(), s["beta"].double(),
                                     s["Dk"])[:2]
        return [y, state]
    return _exact_delta_fwd(s) if op == "delta_fwd" else _exact_delta_bwd(s)


def _exact_heads(s):
    """q and k [..., Hv, Dk] in 64 bits, and the factors that made them unit."""
    got, share = [], s["Hv"] // s["Hk"]
    for x in (s["q"].double(), s["k"].double()):
        n = (x.pow(2).sum(-1, keepdim=True) + _UNIT_EPS).pow(-0.5) if s["unit"] else torch.ones_like(x[..., :1])
        got.append(((x * n).repeat_interleave(share, -2), n))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def _exact_row(S, q, k, v, g, beta, Dk):
    """One row of all sequences and heads: y, the new state, the decayed one, w."""
    decayed = S * torch.exp(g)[..., None, None]
    w = v - torch.matmul(k[..., None, :], decayed)[..., 0, :]
    new = decayed + k[..., :, None] * (beta[..., None] * w)[..., None, :]
    return torch.matmul(q[..., None, :], new)[..., 0, :] * Dk ** -0.5, new, decayed, w


def _exact_rows(s):
    """Rows first, in 64 bits; past a sequence's end: no decay, no correction."""
    q, k, nq, nk = _exact_heads(s)
    v, g, beta = s["v"].double(), s["g"].double(), s["beta"].double()
    if s["lengths"] is not None:
        past = (torch.arange(s["T"], device=_DEV)[None, :] >= s["lengths"][:, None])[..., None]
        g, beta = g.masked_fill(past, 0.0), beta.masked_fill(past, 0.0)
    rows = [x.transpose(0, 1).contiguous() for x in (q, k, v, g, beta)]
    return rows, nq, nk


def _exact_first(s):
    if s["start"] is not None:
        return s["start"].double()
    return torch.zeros(s["B"], s["Hv"], s["Dk"], s["Dv"], dtype=torch.float64, device=_DEV)


def _exact_delta_fwd(s):
    rows, _, _ = _exact_rows(s)
    S = _exact_first(s)
    y = torch.empty(rows[2].shape, dtype=torch.float64, device=_DEV)
    for t in range(s["T"]):
        y[t], S = _exact_row(S, *(x[t] for x in rows), s["Dk"])[:2]
    y = y.transpose(0, 1)
    if s["lengths"] is not None:
        y = y.masked_fill((torch.arange(s["T"], device=_DEV)[None, :] >= s["lengths"][:, None])[..., None, None], 0.0)
    return [y, S]


def _exact_delta_bwd(s):
    rows, nq, nk = _exact_rows(s)
    q, k, v, g, beta = rows
    T, step = s["T"], 64
    past = None
    dy = s["dy"].double()
    if s["lengths"] is not None:
        past = torch.arange(T, device=_DEV)[None, :] >= s["lengths"][:, None]
        dy = dy.masked_fill(past[..., None, None], 0.0)
    dy = dy.transpose(0, 1).contiguous() * s["Dk"] ** -0.5
    S, kept = _exact_first(s), []
    for t in range(T):
        if t % step == 0:
            kept.append(S)
        S = _exact_row(S, *(x[t] for x in rows), s["Dk"])[1]
    dS = torch.zeros_like(S) if s["dhT"] is None else s["dhT"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    for first in reversed(range(0, T, step)):
        S, seen = kept.pop(), []
        for t in range(first, min(first + step, T)):
            _, S, decayed, w = _exact_row(S, *(x[t] for x in rows), s["Dk"])
            seen.append((S, decayed, w))
        for t in reversed(range(first, min(first + step, T))):
            new, decayed, w = seen.pop()
            dq[t] = torch.matmul(new, dy[t][..., None])[..., 0]
            dS = dS + q[t][..., :, None] * dy[t][..., None, :]
            du = torch.matmul(k[t][..., None, :], dS)[..., 0, :]
            dbeta[t] = (du * w).sum(-1)
            dv[t] = beta[t][..., None] * du
            dk[t] = torch.matmul(dS, (beta[t][..., None] * w)[..., None])[..., 0]
            dk[t] -= torch.matmul(decayed, dv[t][..., None])[..., 0]
            dS = dS - k[t][..., :, None] * dv[t][..., None, :]
            dg[t] = (dS * decayed).sum((-1, -2))
            dS = dS * torch.exp(g[t])[..., None, None]
    dq, dk, dv, dg, dbeta = (x.transpose(0, 1) for x in (dq, dk, dv, dg, dbeta))
    share = s["Hv"] // s["Hk"]
    dq, dk = (x.unflatten(2, (s["Hk"], share)).sum(3) for x in (dq, dk))
    if s["unit"]:
        hats = (s["q"].double() * nq, nq, dq), (s["k"].double() * nk, nk, dk)
        dq, dk = (n * (d - hat * (hat * d).sum(-1, keepdim=True)) for hat, n, d in hats)
    if past is not None:
        dq, dk, dv = (x.masked_fill(past[..., None, None], 0.0) for x in (dq, dk, dv))
        dg, dbeta = (x.masked_fill(past[..., None], 0.0) for x in (dg, dbeta))
    return [dq, dk, dv, dg, dbeta, dS if s["start"] is not None else None]


def _exact_branch(s, h, n1):
    """The block's output through norm, weight and gate, before the residual scale; and its gate's value and slope."""
    t = h * n1
    w = 1.0 if s["w_post"] is None else s["w_post"].double()
    a, slope = 1.0, None
    if s["gate_rows"] is not None:
        g = s["gate_rows"].double()
        sig = torch.sigmoid(g)
        a, slope = (sig, sig * torch.sigmoid(-g)) if s["gate"] == "sigmoid" else \
            (g * sig, sig + g * sig * torch.sigmoid(-g))
    return t, w, a, slope


def _exact_join_fwd(s):
    h = s["h"].double()
    D = s["D"]
    n1 = (h.pow(2).sum(-1, keepdim=True) / D + _EPS).pow(-0.5) if s["post"] else torch.ones_like(h[:, :1])
    t, w, a, _ = _exact_branch(s, h, n1)
    y = s["factor"] * (t * w * a) + (0.0 if s["r"] is None else s["r"].double())
    n2, x = torch.ones_like(n1), None
    if s["pre"]:
        n2 = (y.pow(2).sum(-1, keepdim=True) / D + _EPS).pow(-0.5)
        x = y * n2 * (1.0 if s["w_pre"] is None else s["w_pre"].double())
    return [y, x, torch.stack([n1[:, 0], n2[:, 0]])]


def _exact_join_bwd(s):
    h, D = s["h"].double(), s["D"]
    n1, n2 = s["stats"].double()[:, :, None]
    t, w, a, slope = _exact_branch(s, h, n1)
    d = torch.zeros_like(h) if s["dy"] is None else s["dy"].double()
    dw_pre = None
    if s["dx"] is not None:
        z, c = s["y"].double() * n2, s["dx"].double()
        if s["w_pre"] is not None:
            dw_pre = torch.matmul(torch.ones(1, s["N"], dtype=torch.float64, device=_DEV), c * z)[0]
            c = c * s["w_pre"].double()
        d = d + n2 * c - n2 * z * ((c * z).sum(-1, keepdim=True) / D)
    dgate = None if slope is None else s["factor"] * d * t * w * slope
    to_t = s["factor"] * d * a
    dw_post = None
    if s["w_post"] is not None:
        dw_post = torch.matmul(torch.ones(1, s["N"], dtype=torch.float64, device=_DEV), to_t * t)[0]
    to_t = to_t * w
    dh = n1 * to_t - n1 * t * ((to_t * t).sum(-1, keepdim=True) / D) if s["post"] else to_t
    return [dh, d if s["r"] is not None else None, dgate, dw_post, dw_pre]
