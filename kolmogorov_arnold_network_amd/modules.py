"""``KANLayer`` / ``KANNetwork`` / ``KANGroupedActivation`` / ``KANSurfaceLayer``, and
for models over tokens ``KANEmbedding`` / ``KANRecurrence`` / ``KANDistillLoss``:
torch modules over the HIP library.

"KANLayer(in, out) replaces nn.Linear(in, out). Same interface, same
optimizer, same training loop" (InKAN project page, "Why InKAN?"): the layer
takes ``[..., in_features]`` and returns ``[..., out_features]``, and its
parameters are plain tensors that any torch optimizer updates.  Autograd
calls ``kan_backward``; torch only accumulates the returned gradients.
"""

import math

import torch
from torch.autograd.function import once_differentiable

from . import functional as F


class KANFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, C, W, lo, hi, G, variant):
        ctx.grid = (lo, hi, G)
        ctx.variant = variant
        ctx.has_base = W is not None
        ctx.save_for_backward(x, C, W)
        return F.kan_forward(x, C, W, (lo, hi, G), variant)

    @staticmethod
    def backward(ctx, dy):
        x, C, W = ctx.saved_tensors
        need_x, need_C, need_W = ctx.needs_input_grad[:3]
        dx, dC, dW = F.kan_backward(x, C, W, dy.contiguous().float(), ctx.grid, need_dx=need_x,
                                    need_dC=need_C, need_dW=need_W and ctx.has_base,
                                    variant=ctx.variant)
        if dx is not None and dx.dtype != x.dtype:
            dx = dx.to(x.dtype)
        if dC is not None and dC.dtype != C.dtype:
            dC = dC.to(C.dtype)
        if dW is not None and dW.dtype != W.dtype:
            dW = dW.to(W.dtype)
        return dx, dC, dW, None, None, None, None


class CastBF16(torch.autograd.Function):
    """float32 -> bfloat16 on the device; the gradient passes through as float32."""

    @staticmethod
    def forward(ctx, t):
        return F.kan_cast_f32_to_bf16(t.contiguous())

    @staticmethod
    def backward(ctx, g):
        return g.float()


class KANLayer(torch.nn.Module):
    """One KAN layer: ``y_j = sum_i phi_ji(x_i)`` with cubic B-spline ``phi_ji``.

    Parameters: ``coef [out, in, grid_size + degree]`` and, with ``base=True``,
    ``base_weight [out, in]`` for the ``W_base * silu(x)`` branch.  ``dtype``
    (float32 or bfloat16) is the storage of inputs and parameters; outputs
    and gradients are computed in float32.  ``degree`` (1 .. 5) is the spline
    degree, 3 (cubic) by default.
    """

    def __init__(self, in_features, out_features, grid_size=8, grid_range=(-1.0, 1.0), base=True,
                 dtype=torch.float32, device=None, variant="auto", coef_std=0.1, degree=3):
        super().__init__()
        self.in_features = int(in_features)
        self.out_features = int(out_features)
        self.grid_size = int(grid_size)
        self.grid_range = (float(grid_range[0]), float(grid_range[1]))
        self.variant = variant
        self.degree = int(degree)
        fk = dict(dtype=dtype, device=device)
        self.coef = torch.nn.Parameter(
            torch.randn(out_features, in_features, grid_size + self.degree, **fk) * coef_std)
        if base:
            self.base_weight = torch.nn.Parameter(
                torch.randn(out_features, in_features, **fk) / math.sqrt(in_features))
        else:
            self.register_parameter("base_weight", None)

    @property
    def grid(self):
        return (self.grid_range[0], self.grid_range[1], self.grid_size)

    def forward(self, x):
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features)
        if x2.dtype != self.coef.dtype:
            x2 = CastBF16.apply(x2) if self.coef.dtype == torch.bfloat16 else x2.to(self.coef.dtype)
        x2 = x2.contiguous()
        y = KANFunction.apply(x2, self.coef, self.base_weight, self.grid_range[0],
                              self.grid_range[1], self.grid_size, self.variant)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        return "in=%d, out=%d, grid_size=%d, degree=%d, range=%s, base=%s, dtype=%s" % (
            self.in_features, self.out_features, self.grid_size, self.degree, self.grid_range,
            self.base_weight is not None, self.coef.dtype)


class KANNetwork(torch.nn.Module):
    """A chain of ``KANLayer`` with nothing in between (InKAN "Quick Start")."""

    def __init__(self, widths, **kw):
        super().__init__()
        self.layers = torch.nn.ModuleList(
            KANLayer(widths[l], widths[l + 1], **kw) for l in range(len(widths) - 1))

    def forward(self, x):
        for layer in self.layers:
            x = layer(x)
        return x


def _to_storage(x, dtype):
    if x.dtype == dtype:
        return x
    return CastBF16.apply(x) if dtype == torch.bfloat16 else x.to(dtype)


class GroupedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, C, lo, hi, G):
        ctx.grid = (lo, hi, G)
        ctx.save_for_backward(x, C)
        return F.kan_group_forward(x, C, (lo, hi, G))

    @staticmethod
    def backward(ctx, dy):
        x, C = ctx.saved_tensors
        need_x, need_C = ctx.needs_input_grad[:2]
        dx, dC = F.kan_group_backward(x, C, dy.contiguous().float(), ctx.grid, need_dx=need_x,
                                      need_dC=need_C)
        if dx is not None and dx.dtype != x.dtype:
            dx = dx.to(x.dtype)
        if dC is not None and dC.dtype != C.dtype:
            dC = dC.to(C.dtype)
        return dx, dC, None, None, None


class KANGroupedActivation(torch.nn.Module):
    """Element-wise spline activation: channel ``i`` of ``[..., channels]``
    passes through cubic B-spline ``phi_{g(i)}``, shared by the consecutive
    channels of group ``g(i) = i * groups // channels``; ``groups ==
    channels`` gives one spline per channel.  Parameter ``coef [groups,
    grid_size + 3]``; output and gradients in float32."""

    def __init__(self, channels, groups=1, grid_size=8, grid_range=(-1.0, 1.0), dtype=torch.float32,
                 device=None, coef_std=0.1):
        super().__init__()
        if not 1 <= groups <= channels:
            raise ValueError("need 1 <= groups <= channels")
        self.channels = int(channels)
        self.groups = int(groups)
        self.grid_size = int(grid_size)
        self.grid_range = (float(grid_range[0]), float(grid_range[1]))
        self.coef = torch.nn.Parameter(torch.randn(groups, grid_size + 3, dtype=dtype, device=device) * coef_std)

    def forward(self, x):
        lead = x.shape[:-1]
        x2 = _to_storage(x.reshape(-1, self.channels), self.coef.dtype).contiguous()
        y = GroupedFunction.apply(x2, self.coef, self.grid_range[0], self.grid_range[1], self.grid_size)
        return y.reshape(*lead, self.channels)

    def extra_repr(self):
        return "channels=%d, groups=%d, grid_size=%d, range=%s, dtype=%s" % (
            self.channels, self.groups, self.grid_size, self.grid_range, self.coef.dtype)


class SurfaceFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, C, lo, hi, G):
        ctx.grid = (lo, hi, G)
        ctx.save_for_backward(x, C)
        return F.kan_surface_forward(x, C, (lo, hi, G))

    @staticmethod
    def backward(ctx, dy):
        x, C = ctx.saved_tensors
        need_x, need_C = ctx.needs_input_grad[:2]
        dx, dC = F.kan_surface_backward(x, C, dy.contiguous().float(), ctx.grid, need_dx=need_x,
                                        need_dC=need_C)
        if dx is not None and dx.dtype != x.dtype:
            dx = dx.to(x.dtype)
        if dC is not None and dC.dtype != C.dtype:
            dC = dC.to(C.dtype)
        return dx, dC, None, None, None


class KANSurfaceLayer(torch.nn.Module):
    """2-D tensor-product spline layer: the inputs are taken in consecutive
    pairs ``(x[..., 2p], x[..., 2p+1])`` and output ``j`` sums a bicubic
    surface per pair, ``sum_{m,n} C[j, p, m, n] B_m(x1) B_n(x2)``.
    Parameter ``coef [out, in/2, grid_size + 3, grid_size + 3]``
    (``grid_size <= 13``); output and gradients in float32."""

    def __init__(self, in_features, out_features, grid_size=5, grid_range=(-1.0, 1.0), dtype=torch.float32,
                 device=None, coef_std=0.02):
        super().__init__()
        if in_features % 2:
            raise ValueError("the 2-D layer takes an even number of inputs")
        self.in_features = int(in_features)
        self.out_features = int(out_features)
        self.grid_size = int(grid_size)
        self.grid_range = (float(grid_range[0]), float(grid_range[1]))
        K = grid_size + 3
        self.coef = torch.nn.Parameter(
            torch.randn(out_features, in_features // 2, K, K, dtype=dtype, device=device) * coef_std)

    def forward(self, x):
        lead = x.shape[:-1]
        x2 = _to_storage(x.reshape(-1, self.in_features), self.coef.dtype).contiguous()
        y = SurfaceFunction.apply(x2, self.coef, self.grid_range[0], self.grid_range[1], self.grid_size)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        return "in=%d (pairs=%d), out=%d, grid_size=%d, range=%s, dtype=%s" % (
            self.in_features, self.in_features // 2, self.out_features, self.grid_size, self.grid_range,
            self.coef.dtype)


class EmbedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, row_dtype):
        ctx.scale = scale
        ctx.rows = table.shape[0]
        ctx.table_dtype = table.dtype
        ctx.save_for_backward(ids)
        return F.kan_embed_forward(ids, table, scale, row_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        dE = F.kan_embed_backward(ids, dy.contiguous(), ctx.rows, ctx.scale)
        return None, dE if ctx.table_dtype == torch.float32 else dE.to(ctx.table_dtype), None, None


class KANEmbedding(torch.nn.Module):
    """Token rows: ``scale * table[ids]`` (default scale ``sqrt(features)``, for a
    table of standard deviation ``1 / sqrt(features)``); ids outside the table
    (padding) give zero rows.  The gradient is summed by token without atomics.
    Parameter ``table [num_tokens, features]`` in ``dtype``; rows in
    ``row_dtype`` (default ``dtype``)."""

    def __init__(self, num_tokens, features, scale=None, dtype=torch.float32, row_dtype=None, device=None):
        super().__init__()
        self.num_tokens = int(num_tokens)
        self.features = int(features)
        self.scale = math.sqrt(features) if scale is None else float(scale)
        self.row_dtype = row_dtype or dtype
        self.table = torch.nn.Parameter(
            torch.randn(num_tokens, features, dtype=dtype, device=device) / math.sqrt(features))

    def forward(self, ids):
        return EmbedFunction.apply(ids.contiguous(), self.table, self.scale, self.row_dtype)

    def extra_repr(self):
        return "tokens=%d, features=%d, scale=%g, dtype=%s, rows=%s" % (
            self.num_tokens, self.features, self.scale, self.table.dtype, self.row_dtype)


class RecurFunction(torch.autograd.Function):
    """The recurrence over ``p [B, T, 2 D]``, whose halves are x and g."""

    @staticmethod
    def forward(ctx, p, h0, lengths):
        D = p.shape[2] // 2
        y, hT = F.kan_recur_forward(p[..., :D], p[..., D:], h0, lengths)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(p, h0, lengths, y)
        return y, hT

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dhT):
        p, h0, lengths, y = ctx.saved_tensors
        D = p.shape[2] // 2
        dy = torch.zeros_like(y) if dy is None else dy.contiguous()
        dp = torch.empty(p.shape, dtype=p.dtype, device=p.device)
        dhT = None if dhT is None else dhT.contiguous()
        dh0 = F.kan_recur_backward(p[..., :D], p[..., D:], y, dy, h0, lengths, dhT,
                                   need_dh0=ctx.needs_input_grad[1], dx=dp[..., :D], dg=dp[..., D:])[2]
        return dp, dh0, None


class KANRecurrence(torch.nn.Module):
    """Mixes the rows of a sequence: a ``KANLayer`` of twice the width makes a
    value x and a gate g of every row, and each channel follows
    ``h_t = sigmoid(g_t) h_{t-1} + sigmoid(-g_t) x_t``.

    ``forward(x [B, T, in], h0 [B, out], lengths [B])`` returns the rows ``y [B, T,
    out]`` and the last states ``[B, out]``, float32; ``step(x [B, in], state [S,
    out], slots [B])`` takes one row of each of B sequences and replaces their
    states in the pool."""

    def __init__(self, in_features, out_features, **kw):
        super().__init__()
        self.in_features = int(in_features)
        self.out_features = int(out_features)
        self.layer = KANLayer(in_features, 2 * out_features, **kw)

    def forward(self, x, h0=None, lengths=None):
        # one initial state for all sequences comes expanded
        return RecurFunction.apply(self.layer(x), None if h0 is None else h0.contiguous(),
                                   None if lengths is None else lengths.contiguous())

    @torch.no_grad()
    def step(self, x, state, slots=None):
        p = self.layer(x)
        return F.kan_recur_step(p[:, :self.out_features], p[:, self.out_features:], state,
                                None if slots is None else slots.contiguous())

    def extra_repr(self):
        return "in=%d, out=%d" % (self.in_features, self.out_features)


_NO_GRADIENT = "the loss has no gradient of the teacher's logits or of the weights: detach them"


class DistillFunction(torch.autograd.Function):
    """The rows' losses; their gradient is that of the student's logits alone."""

    @staticmethod
    def forward(ctx, z, ids, t, temperature, weight):
        loss, lse = F.kan_distill_forward(z, ids, t, temperature, weight)
        ctx.temperature = temperature
        ctx.save_for_backward(z, ids, t, lse, weight)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        if ctx.needs_input_grad[2] or ctx.needs_input_grad[4]:
            raise ValueError(_NO_GRADIENT)
        z, ids, t, lse, weight = ctx.saved_tensors
        dz = F.kan_distill_backward(z, ids, t, lse, dloss.contiguous().float(), ctx.temperature, weight,
                                    grad_dtype=z.dtype)
        return dz, None, None, None, None


class KANDistillLoss(torch.nn.Module):
    """``tau^2`` times the divergence of a student's logits ``z [..., V]`` from a
    teacher's top logits ``t [..., K]`` of the tokens ``ids [..., K]``, both
    softened by the temperature ``tau``.  ``weight [...]`` (float32) scales rows;
    rows of weight 0 (padding) reach neither loss nor gradient.  The gradient is
    that of ``z``; ``t`` and ``weight`` must not require one.  ``reduction``: ``mean`` over all
    rows, ``sum`` or ``none``."""

    def __init__(self, temperature=1.0, reduction="mean"):
        super().__init__()
        if reduction not in ("mean", "sum", "none"):
            raise ValueError("reduction must be mean, sum or none")
        self.temperature = float(temperature)
        self.reduction = reduction

    def forward(self, z, ids, t, weight=None):
        lead = z.shape[:-1]
        if ids.shape[:-1] != lead or t.shape != ids.shape or (weight is not None and weight.shape != lead):
            raise ValueError("z, ids, t and weight must share their leading dimensions")
        if torch.is_grad_enabled() and (t.requires_grad or (weight is not None and weight.requires_grad)):
            raise ValueError(_NO_GRADIENT)
        K = ids.shape[-1]
        z = z.reshape(-1, z.shape[-1])
        if z.stride(1) != 1 or z.stride(0) < z.shape[1]:        # rows that are columns, or one for all
            z = z.contiguous()
        loss = DistillFunction.apply(z, ids.reshape(-1, K).contiguous(),
                                     t.reshape(-1, K).contiguous(), self.temperature,
                                     None if weight is None else weight.reshape(-1).contiguous())
        if self.reduction == "none":
            return loss.reshape(lead)
        return loss.mean() if self.reduction == "mean" else loss.sum()

    def extra_repr(self):
        return "temperature=%g, reduction=%s" % (self.temperature, self.reduction)


class DeltaFunction(torch.autograd.Function):
    """The gated delta rule over ``p [B, T, 2 Hk Dk + Hv Dv]``, whose slices are q, k and v."""

    @staticmethod
    def _slices(p, Hk, Dk, Hv, Dv):
        n = Hk * Dk
        return (p[..., :n].unflatten(-1, (Hk, Dk)), p[..., n:2 * n].unflatten(-1, (Hk, Dk)),
                p[..., 2 * n:].unflatten(-1, (Hv, Dv)))

    @staticmethod
    def forward(ctx, p, g, beta, h0, lengths, heads):
        y, hT = F.kan_delta_forward(*DeltaFunction._slices(p, *heads), g, beta, h0, lengths, unit=True)
        ctx.heads = heads
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(p, g, beta, h0, lengths)
        return y, hT

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dhT):
        p, g, beta, h0, lengths = ctx.saved_tensors
        Hk, Dk, Hv, Dv = ctx.heads
        dy = p.new_zeros((*p.shape[:2], Hv, Dv)) if dy is None else dy.contiguous()
        dp = torch.empty(p.shape, dtype=p.dtype, device=p.device)
        dq, dk, dv = DeltaFunction._slices(dp, *ctx.heads)
        _, _, _, dg, dbeta, dh0 = F.kan_delta_backward(
            *DeltaFunction._slices(p, *ctx.heads), g, beta, dy, h0, lengths, None if dhT is None else dhT.contiguous(),
            unit=True, need_dh0=ctx.needs_input_grad[3], dq=dq, dk=dk, dv=dv)
        return dp, dg, dbeta, dh0, None, None


class KANDeltaRule(torch.nn.Module):
    """Mixes the rows of a sequence by the gated delta rule: a ``KANLayer`` makes
    queries and keys of ``key_heads`` heads and values of ``heads`` heads of every row, a
    second one a decay and a rate for each of ``heads`` heads, both through a sigmoid.
    Each head keeps a state ``[key_features, value_features]`` that answers keys with
    values; queries and keys are unit vectors.

    ``forward(x [B, T, in], h0 [B, heads, key_features, value_features], lengths [B])`` returns
    the rows ``[B, T, heads * value_features]`` and the last states, float32;
    ``step(x [B, in], state [S, heads, key_features, value_features], slots [B])`` takes one row
    of each of B sequences and replaces their states in the pool.  The decays start
    near ``sigmoid(gate_offset)``."""

    def __init__(self, in_features, heads, key_features, value_features, key_heads=None, gate_offset=4.0, **kw):
        super().__init__()
        self.in_features = int(in_features)
        self.heads = int(heads)
        self.key_heads = int(heads if key_heads is None else key_heads)
        self.key_features, self.value_features = int(key_features), int(value_features)
        if self.heads % self.key_heads:
            raise ValueError("heads must be a multiple of key_heads")
        self.gate_offset = float(gate_offset)
        self.layer = KANLayer(in_features, 2 * self.key_heads * self.key_features + self.heads * self.value_features, **kw)
        self.gates = KANLayer(in_features, 2 * self.heads, **kw)

    def _shape(self):
        return self.key_heads, self.key_features, self.heads, self.value_features

    def _gates(self, x):
        a, b = self.gates(x).split(self.heads, -1)
        return torch.nn.functional.logsigmoid(a + self.gate_offset), torch.sigmoid(b)

    def forward(self, x, h0=None, lengths=None):
        g, beta = self._gates(x)
        y, hT = DeltaFunction.apply(self.layer(x), g, beta, None if h0 is None else h0.contiguous(),
                                    None if lengths is None else lengths.contiguous(), self._shape())
        return y.flatten(2), hT

    @torch.no_grad()
    def step(self, x, state, slots=None):
        g, beta = self._gates(x)
        q, k, v = DeltaFunction._slices(self.layer(x), *self._shape())
        return F.kan_delta_step(q, k, v, g, beta, state, None if slots is None else slots.contiguous(),
                                unit=True).flatten(1)

    def extra_repr(self):
        return "in=%d, heads=%d (keys %d), key_features=%d, value_features=%d" % (
            self.in_features, self.heads, self.key_heads, self.key_features, self.value_features)


class JoinFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, r, gate, w_post, w_pre, post, pre, activation, scale, eps, row_dtype):
        y, x, stats = F.kan_join_forward(h, r, gate, w_post, w_pre, post, pre, activation, scale, eps, None, row_dtype)
        ctx.kw = dict(post=post, activation=activation, scale=scale)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, gate, w_post, w_pre, y, stats)
        return y, x

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dx):
        h, gate, w_post, w_pre, y, stats = ctx.saved_tensors
        dh, dr, dgate, dw_post, dw_pre = F.kan_join_backward(
            h, y, stats, None if dy is None else dy.contiguous(), None if dx is None else dx.contiguous(), gate, w_post,
            None if dx is None else w_pre, need_dr=ctx.needs_input_grad[1], **ctx.kw)
        return (dh, dr, dgate, dw_post, dw_pre) + (None,) * 6


class KANJoin(torch.nn.Module):
    """What stands between two blocks: the norm of the block's output (``post``), its
    gate, its scale, the residual sum, and the norm of the sum for the next block
    (``pre``), in one pass over the rows:

        y = residual + scale * act(gate) * w_post * norm(h),   x = w_pre * norm(y)

    ``forward(h [..., D], residual, gate)`` returns ``(y, x)``, or y alone without
    ``pre``; residual and gate may be None.  ``y`` has the residual's dtype (or h's), x
    ``row_dtype`` (default h's).  With ``pre=False`` and neither residual nor gate it is a
    norm.  Parameters ``w_post`` and ``w_pre [D]`` float32, ones at the start."""

    def __init__(self, features, post=True, pre=True, activation="silu", scale=1.0, eps=1e-6, row_dtype=None,
                 device=None):
        super().__init__()
        if activation not in ("silu", "sigmoid"):
            raise ValueError("activation must be silu or sigmoid")
        self.features, self.post, self.pre = int(features), bool(post), bool(pre)
        self.activation, self.scale, self.eps, self.row_dtype = activation, float(scale), float(eps), row_dtype
        self.w_post = torch.nn.Parameter(torch.ones(features, device=device))
        self.w_pre = torch.nn.Parameter(torch.ones(features, device=device)) if pre else None

    def forward(self, h, residual=None, gate=None):
        if h.dim() < 1 or h.shape[-1] != self.features:
            raise ValueError("h must have rows of %d features, got %s" % (self.features, tuple(h.shape)))
        for name, t in (("residual", residual), ("gate", gate)):
            if t is not None and t.shape != h.shape:
                raise ValueError("%s must be %s, got %s" % (name, tuple(h.shape), tuple(t.shape)))

        def rows(t):
            if t is None:
                return None
            t = t.reshape(-1, self.features)
            return t if t.shape[1] == 1 or t.stride(1) == 1 else t.contiguous()

        y, x = JoinFunction.apply(rows(h), rows(residual), rows(gate), self.w_post, self.w_pre, self.post, self.pre,
                                  self.activation, self.scale, self.eps, self.row_dtype)
        y = y.reshape(h.shape)
        return (y, x.reshape(h.shape)) if self.pre else y

    def extra_repr(self):
        return "features=%d, post=%s, pre=%s, activation=%s, scale=%g" % (
            self.features, self.post, self.pre, self.activation, self.scale)
