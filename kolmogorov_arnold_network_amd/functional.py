"""Torch-facing wrappers of the C entry points, under the same names.

Each wrapper checks dtype / device / contiguity, allocates the outputs and the
workspace with torch (device memory only), and passes raw pointers plus the
current HIP stream to the library.  No arithmetic of the layer happens here.
"""

import ctypes

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.KAN_F32, torch.bfloat16: L.KAN_BF16}
_VARIANTS = {"auto": L.KAN_VARIANT_AUTO, "mfma": L.KAN_VARIANT_MFMA, "gather": L.KAN_VARIANT_GATHER}


def _variant(v):
    return _VARIANTS[v] if isinstance(v, str) else int(v)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_current = torch._C._cuda_getDevice                     # the current device's number
_raw_stream = torch._C._cuda_getCurrentRawStream        # of a device number


def _launch(what, dev, fn, *args):
    """Calls entry point ``fn`` for tensors on device number ``dev``, on that
    device's current stream and with it as the current device: a launch on the
    null stream goes to the current one, whatever device its tensors are on."""
    if _current() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    L.check(status, what)


def _check_tensor(t, name, dtypes, device=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _check_out(t, name, shape, device):
    """A caller's output tensor: float32, contiguous, on ``device``, of ``shape``."""
    _check_tensor(t, name, (torch.float32,), device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _check_ws(ws, device):
    """A caller's ``(buffer, bytes)`` workspace: the buffer must hold the bytes
    it declares (the library trusts the declared size)."""
    buf, n = ws
    n = int(n)
    if n < 0:
        raise ValueError("workspace size must be >= 0")
    if n > 0:
        if buf is None or not buf.is_cuda or buf.device != device or not buf.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor on %s" % device)
        if buf.numel() * buf.element_size() < n:
            raise ValueError("workspace holds %d bytes, %d declared"
                             % (buf.numel() * buf.element_size(), n))
    return buf, n


def layer_desc(x, C, W, grid, variant="auto", flags=0):
    """``kan_desc_t`` for ``x [N, I]``, ``C [O, I, G+D]``, ``W [O, I]`` or None;
    the spline degree D (1 .. 5, 3 for the pages' cubic layer) is read off C."""
    lo, hi, G = grid
    N, I = x.shape
    O, I2, K = C.shape
    if I2 != I or not 1 <= K - G <= 5:
        raise ValueError("C must be [O, I, G+D] = [%d, %d, %d+D], D in 1..5, got %s"
                         % (O, I, G, tuple(C.shape)))
    if W is not None and tuple(W.shape) != (O, I):
        raise ValueError("W_base must be [O, I]")
    if x.dtype != C.dtype or (W is not None and W.dtype != C.dtype):
        raise ValueError("x, C and W_base must share one dtype")
    return L.make_desc(N, I, O, lo, hi, G, _DTYPES[x.dtype], W is not None, _variant(variant), flags,
                       degree=K - G)


def kan_workspace_size(desc, pass_):
    n = L.lib().kan_workspace_size(ctypes.byref(desc), int(pass_))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid layer description")
    return int(n)


def workspace(desc, pass_, device):
    """A fresh device workspace for one pass (torch allocator; 512-byte aligned)."""
    n = kan_workspace_size(desc, pass_)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n


def _fwd_flags(dense_forward, tp_forward):
    return (L.KAN_FLAG_DENSE_FORWARD if dense_forward else 0) | (L.KAN_FLAG_TP_FORWARD if tp_forward else 0)


def kan_prepare(x, C, W, grid, pass_, dy=None, variant="auto", ws=None, dense_forward=False, tp_forward=False):
    """Packs the pass's operands into a workspace; returns ``(ws, ws_bytes)``."""
    _check_tensor(C, "C", _DTYPES)
    _check_tensor(W, "W_base", _DTYPES, C.device)
    _check_tensor(dy, "dy", (torch.float32,), C.device)
    desc = layer_desc(x, C, W, grid, variant, _fwd_flags(dense_forward, tp_forward))
    if dy is not None and tuple(dy.shape) != (x.shape[0], C.shape[0]):
        raise ValueError("dy must be [N, O]")
    if ws is None:
        ws = workspace(desc, pass_, C.device)
    buf, n = _check_ws(ws, C.device)
    _launch("kan_prepare", C.get_device(), L.lib().kan_prepare, ctypes.byref(desc), int(pass_), _ptr(C), _ptr(W),
            _ptr(dy), _ptr(buf), n)
    return ws


def kan_forward(x, C, W, grid, variant="auto", ws=None, prepared=False, out=None,
                dense_forward=False, tp_forward=False):
    """``y [N, O]`` float32 of one KAN layer.  ``dense_forward`` turns off the
    structured-sparse forward of bf16 layers (``KAN_FLAG_DENSE_FORWARD``);
    ``tp_forward`` generates the dense bf16 basis tile by the truncated-power
    form (``KAN_FLAG_TP_FORWARD``)."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    _check_tensor(W, "W_base", _DTYPES, x.device)
    flags = (L.KAN_FLAG_PREPARED if prepared else 0) | _fwd_flags(dense_forward, tp_forward)
    desc = layer_desc(x, C, W, grid, variant, flags)
    if ws is None:
        ws = workspace(desc, L.KAN_PASS_FORWARD, x.device)
    buf, n = _check_ws(ws, x.device)
    y = out if out is not None else torch.empty((x.shape[0], C.shape[0]), dtype=torch.float32,
                                                device=x.device)
    _check_out(y, "y", (x.shape[0], C.shape[0]), x.device)
    _launch("kan_forward", x.get_device(), L.lib().kan_forward, ctypes.byref(desc), _ptr(x), _ptr(C), _ptr(W),
            _ptr(y), _ptr(buf), n)
    return y


def kan_forward_static(x, C, W, grid, variant="auto", out=None, dense_forward=False):
    """``y [N, O]`` float32 of one KAN layer with the library's own static
    device workspace (no workspace argument, nothing allocated but ``y``
    when ``out`` is not given)."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    _check_tensor(W, "W_base", _DTYPES, x.device)
    desc = layer_desc(x, C, W, grid, variant, L.KAN_FLAG_DENSE_FORWARD if dense_forward else 0)
    y = out if out is not None else torch.empty((x.shape[0], C.shape[0]), dtype=torch.float32,
                                                device=x.device)
    _check_out(y, "y", (x.shape[0], C.shape[0]), x.device)
    _launch("kan_forward_static", x.get_device(), L.lib().kan_forward_static, ctypes.byref(desc), _ptr(x), _ptr(C),
            _ptr(W), _ptr(y))
    return y


def kan_backward(x, C, W, dy, grid, need_dx=True, need_dC=True, need_dW=True, variant="auto",
                 ws=None, prepared=False):
    """``(dx [N, I], dC [O, I, G+3], dW_base [O, I])`` float32; unrequested ones are None."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    _check_tensor(W, "W_base", _DTYPES, x.device)
    _check_tensor(dy, "dy", (torch.float32,), x.device)
    desc = layer_desc(x, C, W, grid, variant, L.KAN_FLAG_PREPARED if prepared else 0)
    if tuple(dy.shape) != (x.shape[0], C.shape[0]):
        raise ValueError("dy must be [N, O]")
    if ws is None:
        ws = workspace(desc, L.KAN_PASS_BACKWARD, x.device)
    buf, n = _check_ws(ws, x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    dx = torch.empty(x.shape, **f32) if need_dx else None
    dC = torch.empty(C.shape, **f32) if need_dC else None
    dW = torch.empty(W.shape, **f32) if (need_dW and W is not None) else None
    _launch("kan_backward", x.get_device(), L.lib().kan_backward, ctypes.byref(desc), _ptr(x), _ptr(C), _ptr(W),
            _ptr(dy), _ptr(dx), _ptr(dC), _ptr(dW), _ptr(buf), n)
    return dx, dC, dW


def _basis(fn, name, x, grid, need_B, need_dB, degree):
    _check_tensor(x, "x", _DTYPES)
    lo, hi, G = grid
    g = L.kan_grid_t(float(lo), float(hi), int(G), int(degree))
    n = x.numel()
    B = torch.empty((n, G + degree), dtype=torch.float32, device=x.device) if need_B else None
    dB = torch.empty((n, G + degree), dtype=torch.float32, device=x.device) if need_dB else None
    _launch(name, x.get_device(), fn, ctypes.byref(g), n, _DTYPES[x.dtype], _ptr(x), _ptr(B), _ptr(dB))
    return B, dB


def kan_basis_eval(x, grid, need_B=True, need_dB=True, degree=3):
    """Dense ``B [n, G+degree]`` and ``dB`` of a 1-D tensor of inputs (local span form)."""
    return _basis(L.lib().kan_basis_eval, "kan_basis_eval", x, grid, need_B, need_dB, degree)


def kan_basis_eval_tp(x, grid, need_B=True, need_dB=True, degree=3):
    """The same, from the truncated-power form (every basis function on its own)."""
    return _basis(L.lib().kan_basis_eval_tp, "kan_basis_eval_tp", x, grid, need_B, need_dB, degree)


def group_desc(x, C, grid):
    """``kan_group_desc_t`` for ``x [N, I]`` and ``C [groups, G+3]``."""
    lo, hi, G = grid
    if x.dim() != 2 or C.dim() != 2 or C.shape[1] != G + 3:
        raise ValueError("x must be [N, I] and C [groups, G+3]")
    if x.dtype != C.dtype:
        raise ValueError("x and C must share one dtype")
    return L.make_group_desc(x.shape[0], x.shape[1], C.shape[0], lo, hi, G, _DTYPES[x.dtype])


def kan_group_workspace_size(desc):
    n = L.lib().kan_group_workspace_size(ctypes.byref(desc))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid grouped activation description")
    return int(n)


def kan_group_forward(x, C, grid, out=None):
    """``y [N, I]`` float32 of the grouped spline activation
    ``y[b, i] = sum_m C[g(i), m] B_m(x[b, i])``, ``g(i) = i * groups // I``."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    desc = group_desc(x, C, grid)
    y = out if out is not None else torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _check_out(y, "y", x.shape, x.device)
    _launch("kan_group_forward", x.get_device(), L.lib().kan_group_forward, ctypes.byref(desc), _ptr(x), _ptr(C),
            _ptr(y))
    return y


def kan_group_backward(x, C, dy, grid, need_dx=True, need_dC=True, ws=None):
    """``(dx [N, I], dC [groups, G+3])`` float32; unrequested ones are None."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    _check_tensor(dy, "dy", (torch.float32,), x.device)
    desc = group_desc(x, C, grid)
    if tuple(dy.shape) != tuple(x.shape):
        raise ValueError("dy must be [N, I]")
    if ws is None:
        n = kan_group_workspace_size(desc) if need_dC else 0
        ws = (torch.empty(max(n, 1), dtype=torch.uint8, device=x.device), n)
    buf, n = _check_ws(ws, x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    dx = torch.empty(x.shape, **f32) if need_dx else None
    dC = torch.empty(C.shape, **f32) if need_dC else None
    _launch("kan_group_backward", x.get_device(), L.lib().kan_group_backward, ctypes.byref(desc), _ptr(x), _ptr(C),
            _ptr(dy), _ptr(dx), _ptr(dC), _ptr(buf), n)
    return dx, dC


def surface_desc(x, C, grid):
    """``kan_surface_desc_t`` for ``x [N, 2P]`` and ``C [O, P, G+3, G+3]``."""
    lo, hi, G = grid
    if x.dim() != 2 or x.shape[1] % 2 or C.dim() != 4:
        raise ValueError("x must be [N, 2P] and C [O, P, G+3, G+3]")
    O, P, K1, K2 = C.shape
    if 2 * P != x.shape[1] or K1 != G + 3 or K2 != G + 3:
        raise ValueError("C must be [O, %d, %d, %d], got %s" % (x.shape[1] // 2, G + 3, G + 3, tuple(C.shape)))
    if x.dtype != C.dtype:
        raise ValueError("x and C must share one dtype")
    return L.make_surface_desc(x.shape[0], P, O, lo, hi, G, _DTYPES[x.dtype])


def kan_surface_workspace_size(desc, pass_):
    n = L.lib().kan_surface_workspace_size(ctypes.byref(desc), int(pass_))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid 2-D layer description")
    return int(n)


def _surface_ws(desc, pass_, device):
    n = kan_surface_workspace_size(desc, pass_)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n


def kan_surface_forward(x, C, grid, ws=None, out=None, dense_forward=False):
    """``y [N, O]`` float32 of the 2-D tensor-product layer
    ``y[b, j] = sum_p sum_{m,n} C[j, p, m, n] B_m(x[b, 2p]) B_n(x[b, 2p+1])``;
    ``dense_forward`` turns off the structured-sparse forward (bf16, G = 5)."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    desc = surface_desc(x, C, grid)
    if dense_forward:
        desc.flags = L.KAN_FLAG_DENSE_FORWARD
    buf, n = _check_ws(ws if ws is not None else _surface_ws(desc, L.KAN_PASS_FORWARD, x.device), x.device)
    y = out if out is not None else torch.empty((x.shape[0], C.shape[0]), dtype=torch.float32,
                                                device=x.device)
    _check_out(y, "y", (x.shape[0], C.shape[0]), x.device)
    _launch("kan_surface_forward", x.get_device(), L.lib().kan_surface_forward, ctypes.byref(desc), _ptr(x),
            _ptr(C), _ptr(y), _ptr(buf), n)
    return y


def kan_surface_backward(x, C, dy, grid, need_dx=True, need_dC=True, ws=None):
    """``(dx [N, 2P], dC [O, P, G+3, G+3])`` float32; unrequested ones are None."""
    _check_tensor(x, "x", _DTYPES)
    _check_tensor(C, "C", _DTYPES, x.device)
    _check_tensor(dy, "dy", (torch.float32,), x.device)
    desc = surface_desc(x, C, grid)
    if tuple(dy.shape) != (x.shape[0], C.shape[0]):
        raise ValueError("dy must be [N, O]")
    buf, n = _check_ws(ws if ws is not None else _surface_ws(desc, L.KAN_PASS_BACKWARD, x.device), x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    dx = torch.empty(x.shape, **f32) if need_dx else None
    dC = torch.empty(C.shape, **f32) if need_dC else None
    _launch("kan_surface_backward", x.get_device(), L.lib().kan_surface_backward, ctypes.byref(desc), _ptr(x),
            _ptr(C), _ptr(dy), _ptr(dx), _ptr(dC), _ptr(buf), n)
    return dx, dC


def kan_cast_f32_to_bf16(t, out=None):
    """Round-to-nearest-even float32 -> bfloat16 on the device."""
    _check_tensor(t, "input", (torch.float32,))
    o = out if out is not None else torch.empty(t.shape, dtype=torch.bfloat16, device=t.device)
    _launch("kan_cast_f32_to_bf16", t.get_device(), L.lib().kan_cast_f32_to_bf16, _ptr(t), _ptr(o), t.numel())
    return o


# ---- token rows, sequence mixing and distillation -------------------------------
#
# These are called once a token when serving, so their host side is kept short:
# tensors are checked through their device number, addresses and the stream go
# to the library as plain integers, and a call whose tensors lie on another
# device than the current one, or start off the 16 bytes that the entry points
# ask for, is made again on that device with copies of the latter.  (Both tests
# are one expression in each wrapper: a function for them takes 0.4 us a call.)

_INDEX = {torch.int32: L.KAN_I32, torch.int64: L.KAN_I64}
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_NO_WS = ctypes.c_size_t(-1).value


def _dev(t, name):
    """The device number of a call's first tensor."""
    k = t.get_device()
    if k < 0:
        raise ValueError("%s must be a device tensor" % name)
    return k


def _rows(t, name, dtypes, dev, shape=None):
    """Checks a tensor whose last dimension alone must be contiguous."""
    if (t.get_device() == dev and t.dtype in dtypes and (t.is_contiguous() or t.stride(-1) == 1)
            and (shape is None or t.shape == shape)):
        return
    if t.get_device() != dev:
        raise ValueError("%s must be on device %d, is on %s" % (name, dev, t.device))
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected one of %s" % (name, t.dtype, tuple(dtypes)))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)


def _whole(t, name, dtypes, dev, shape=None):
    """Checks a contiguous tensor."""
    if (t.get_device() == dev and t.dtype in dtypes and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    _rows(t, name, dtypes, dev, shape)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _placed(t):
    """An input whose data starts on 16 bytes: a copy of a view that starts
    elsewhere (``ids[1:]``, the gradient of a part of ``torch.cat``), the tensor
    itself otherwise."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _sized_ws(ws, n, t):
    """The caller's workspace, or a fresh one of ``n`` bytes on ``t``'s device
    (none for an invalid description, which the entry point itself refuses)."""
    if ws is not None:
        return _check_ws(ws, t.device)
    if n == 0 or n == _NO_WS:
        return None, 0
    return torch.empty(n, dtype=torch.uint8, device=t.device), n


def _valid_size(n, what):
    if n == _NO_WS:
        raise ValueError("invalid %s description" % what)
    return int(n)


def embed_desc(n, V, D, table_dtype, row_dtype, id_dtype, scale):
    """``kan_embed_desc_t`` of ``n`` tokens over a table ``[V, D]``."""
    return L.kan_embed_desc_t(n, V, D, _DTYPES[table_dtype], _DTYPES[row_dtype], _INDEX[id_dtype], scale)


def kan_embed_workspace_size(desc):
    return _valid_size(L.lib().kan_embed_workspace_size(desc), "embedding")


def kan_embed_forward(ids, table, scale=1.0, row_dtype=None, out=None):
    """``y [*ids.shape, D] = scale * table[ids]``, rounded once to ``row_dtype``
    (default: the table's); the rows of ids outside the table are zero."""
    dev = _dev(ids, "ids")
    _whole(ids, "ids", _INDEX, dev)
    _whole(table, "table", _DTYPES, dev)
    if table.dim() != 2:
        raise ValueError("table must be [V, D]")
    ids_at, table_at = ids.data_ptr(), table.data_ptr()
    if (ids_at | table_at) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_embed_forward(_placed(ids), _placed(table), scale, row_dtype, out)
    V, D = table.shape
    row_dtype = row_dtype or (table.dtype if out is None else out.dtype)
    if row_dtype not in _DTYPES:
        raise ValueError("row_dtype must be one of %s" % (tuple(_DTYPES),))
    if out is None:
        y = table.new_empty((*ids.shape, D), dtype=row_dtype)
    else:
        y = out
        _whole(y, "y", (row_dtype,), dev, (*ids.shape, D))
    desc = embed_desc(ids.numel(), V, D, table.dtype, row_dtype, ids.dtype, scale)
    L.check(L.lib().kan_embed_forward(desc, ids_at, table_at, y.data_ptr(), _raw_stream(dev)), "kan_embed_forward")
    return y


def kan_embed_backward(ids, dy, num_rows, scale=1.0, ws=None, out=None):
    """``dE [num_rows, D]`` float32 of the lookup, from ``dy [*ids.shape, D]``."""
    dev = _dev(ids, "ids")
    _whole(ids, "ids", _INDEX, dev)
    _whole(dy, "dy", _DTYPES, dev)
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        raise ValueError("dy must be [*ids.shape, D], got %s" % (tuple(dy.shape),))
    ids_at, dy_at = ids.data_ptr(), dy.data_ptr()
    if (ids_at | dy_at) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_embed_backward(_placed(ids), _placed(dy), num_rows, scale, ws, out)
    D = dy.shape[-1]
    if out is None:
        dE = dy.new_empty((num_rows, D), dtype=torch.float32)
    else:
        dE = out
        _whole(dE, "dE", _F32, dev, (num_rows, D))
    desc = embed_desc(ids.numel(), num_rows, D, torch.float32, dy.dtype, ids.dtype, scale)
    lib = L.lib()
    buf, n = _sized_ws(ws, lib.kan_embed_workspace_size(desc), dy)
    L.check(lib.kan_embed_backward(desc, ids_at, dy_at, dE.data_ptr(), _addr(buf), n, _raw_stream(dev)),
            "kan_embed_backward")
    return dE


def recur_desc(x, g, dx=None, dg=None):
    """``kan_recur_desc_t`` of ``x``, ``g`` and, for the backward pass, ``dx`` and
    ``dg``, all ``[B, T, D]`` with any strides between rows and sequences."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D], got %s" % (tuple(x.shape),))
    if g.shape != x.shape:
        raise ValueError("g must be %s, got %s" % (tuple(x.shape), tuple(g.shape)))
    if x.dtype != g.dtype:
        raise ValueError("x and g must share one dtype")
    xs, gs = x.stride(), g.stride()
    if dx is None:
        return L.kan_recur_desc_t(*x.shape, xs[1], xs[0], gs[1], gs[0], 0, 0, 0, 0, _DTYPES[x.dtype], L.KAN_F32)
    ds, es = dx.stride(), dg.stride()
    return L.kan_recur_desc_t(*x.shape, xs[1], xs[0], gs[1], gs[0], ds[1], ds[0], es[1], es[0], _DTYPES[x.dtype],
                              _DTYPES[dx.dtype])


def kan_recur_workspace_size(desc, pass_):
    return _valid_size(L.lib().kan_recur_workspace_size(desc, int(pass_)), "recurrence")


def _recur_inputs(x, g, h0, lengths):
    dev = _dev(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D], got %s" % (tuple(x.shape),))
    _rows(x, "x", _DTYPES, dev)
    _rows(g, "g", _DTYPES, dev)
    if h0 is not None:
        _whole(h0, "h0", _F32, dev, (x.shape[0], x.shape[2]))
    if lengths is not None:
        _whole(lengths, "lengths", _I32, dev, x.shape[:1])
    return dev


def kan_recur_forward(x, g, h0=None, lengths=None, ws=None, out=None):
    """``(y [B, T, D], hT [B, D])`` float32 of the gated recurrence
    ``h_t = sigmoid(g_t) h_{t-1} + sigmoid(-g_t) x_t``.  ``h0 [B, D]`` float32
    (default 0), ``lengths [B]`` int32 (default T); ``y`` is 0 past a length."""
    dev = _recur_inputs(x, g, h0, lengths)
    h0_at, lengths_at = _addr(h0), _addr(lengths)
    if ((h0_at or 0) | (lengths_at or 0)) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_recur_forward(x, g, _placed(h0), _placed(lengths), ws, out)
    desc = recur_desc(x, g)
    B, T, D = x.shape
    if out is None:
        y = x.new_empty((B, T, D), dtype=torch.float32)
    else:
        y = out
        _whole(y, "y", _F32, dev, x.shape)
    hT = y.new_empty((B, D))
    lib = L.lib()
    buf, n = _sized_ws(ws, lib.kan_recur_workspace_size(desc, L.KAN_PASS_FORWARD), x)
    L.check(lib.kan_recur_forward(desc, x.data_ptr(), g.data_ptr(), h0_at, lengths_at, y.data_ptr(), hT.data_ptr(),
                                  _addr(buf), n, _raw_stream(dev)), "kan_recur_forward")
    return y, hT


def kan_recur_backward(x, g, y, dy, h0=None, lengths=None, dhT=None, need_dh0=None, grad_dtype=torch.float32,
                       dx=None, dg=None, ws=None):
    """``(dx, dg, dh0)`` from the forward's ``y`` and ``dy [B, T, D]`` (and
    ``dhT [B, D]``).  ``dx`` and ``dg`` are written into the given tensors (any
    row and sequence strides, for instance the halves of one array) or into
    new ones of ``grad_dtype``; ``dh0 [B, D]`` float32 (default: with ``h0``)."""
    dev = _recur_inputs(x, g, h0, lengths)
    shape = x.shape
    _whole(y, "y", _F32, dev, shape)
    _whole(dy, "dy", _F32, dev, shape)
    if dhT is not None:
        _whole(dhT, "dhT", _F32, dev, (shape[0], shape[2]))
    if (dx is None) != (dg is None):
        raise ValueError("give both dx and dg or neither")
    h0_at, lengths_at, y_at, dy_at, dhT_at = _addr(h0), _addr(lengths), y.data_ptr(), dy.data_ptr(), _addr(dhT)
    if ((h0_at or 0) | (lengths_at or 0) | y_at | dy_at | (dhT_at or 0)) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_recur_backward(x, g, _placed(y), _placed(dy), _placed(h0), _placed(lengths), _placed(dhT),
                                      need_dh0, grad_dtype, dx, dg, ws)
    if dx is None:
        dx, dg = x.new_empty((2, *shape), dtype=grad_dtype).unbind(0)
    _rows(dx, "dx", _DTYPES, dev, shape)
    _rows(dg, "dg", (dx.dtype,), dev, shape)
    desc = recur_desc(x, g, dx, dg)
    need_dh0 = h0 is not None if need_dh0 is None else need_dh0
    dh0 = y.new_empty((shape[0], shape[2])) if need_dh0 else None
    lib = L.lib()
    buf, n = _sized_ws(ws, lib.kan_recur_workspace_size(desc, L.KAN_PASS_BACKWARD), x)
    L.check(lib.kan_recur_backward(desc, x.data_ptr(), g.data_ptr(), h0_at, lengths_at, y_at, dy_at, dhT_at,
                                   dx.data_ptr(), dg.data_ptr(), _addr(dh0), _addr(buf), n, _raw_stream(dev)),
            "kan_recur_backward")
    return dx, dg, dh0


def kan_recur_step(x, g, state, slots=None, out=None):
    """One row of each sequence: ``state [S, D]`` float32 is read and replaced in
    rows ``slots [B]`` (int32, all different; default ``0 .. B-1``) and the new
    rows are returned as ``y [B, D]``; a slot outside the pool is skipped."""
    dev = _dev(x, "x")
    if x.dim() != 2 or state.dim() != 2 or state.shape[1] != x.shape[1]:
        raise ValueError("x must be [B, D] and state [S, D]")
    shape = x.shape
    _rows(x, "x", _DTYPES, dev)
    _rows(g, "g", (x.dtype,), dev, shape)
    _whole(state, "state", _F32, dev)
    if slots is not None:
        _whole(slots, "slots", _I32, dev, shape[:1])
    slots_at = _addr(slots)
    if (slots_at or 0) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_recur_step(x, g, state, _placed(slots), out)
    B, D = shape
    xs, gs = x.stride(0), g.stride(0)
    desc = L.kan_recur_desc_t(B, 1, D, xs, xs, gs, gs, 0, 0, 0, 0, _DTYPES[x.dtype], L.KAN_F32)
    if out is None:
        y = state.new_empty((B, D))
    else:
        y = out
        _whole(y, "y", _F32, dev, shape)
    L.check(L.lib().kan_recur_step(desc, state.shape[0], x.data_ptr(), g.data_ptr(), state.data_ptr(), slots_at,
                                   y.data_ptr(), _raw_stream(dev)), "kan_recur_step")
    return y


def _row_stride(t):
    """The stride between the rows of ``[N, V]`` (a single row's stride is free)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def distill_desc(z, ids, t, tau, dz=None, grad_dtype=torch.float32):
    """``kan_distill_desc_t`` of ``z [N, V]`` (a row stride of V or more) and ``ids``, ``t [N, K]``."""
    if z.dim() != 2 or ids.dim() != 2 or ids.shape[0] != z.shape[0]:
        raise ValueError("z must be [N, V] and ids [N, K]")
    if t.shape != ids.shape:
        raise ValueError("t must be %s, got %s" % (tuple(ids.shape), tuple(t.shape)))
    N, V = z.shape
    return L.kan_distill_desc_t(N, V, ids.shape[1], _row_stride(z), V if dz is None else _row_stride(dz),
                                _DTYPES[z.dtype], _DTYPES[t.dtype], _INDEX[ids.dtype],
                                _DTYPES[grad_dtype if dz is None else dz.dtype], tau)


def kan_distill_workspace_size(desc):
    return _valid_size(L.lib().kan_distill_workspace_size(desc), "distillation")


def _distill_inputs(z, ids, t, weight):
    dev = _dev(z, "z")
    if z.dim() != 2:
        raise ValueError("z must be [N, V], got %s" % (tuple(z.shape),))
    _rows(z, "z", _DTYPES, dev)
    _whole(ids, "ids", _INDEX, dev)
    _whole(t, "t", _DTYPES, dev)
    if weight is not None:
        _whole(weight, "weight", _F32, dev, z.shape[:1])
    return dev


def _distill_grad(z, out, grad_dtype, dev):
    if out is None:
        return z.new_empty(z.shape, dtype=grad_dtype)
    _rows(out, "dz", _DTYPES, dev, z.shape)
    return out


def kan_distill_forward(z, ids, t, temperature=1.0, weight=None, ws=None):
    """``(loss [N], lse [N])`` float32: row ``b``'s ``weight_b tau^2`` times the
    divergence of the student's distribution ``softmax(z_b / tau)`` from the
    teacher's, the softmax of its top logits ``t [N, K] / tau`` over the tokens
    ``ids [N, K]`` (int32 or int64; ids outside ``[0, V)`` are absent)."""
    dev = _distill_inputs(z, ids, t, weight)
    ids_at, t_at, weight_at = ids.data_ptr(), t.data_ptr(), _addr(weight)
    if (ids_at | t_at | (weight_at or 0)) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_distill_forward(z, _placed(ids), _placed(t), temperature, _placed(weight), ws)
    desc = distill_desc(z, ids, t, temperature)
    loss = z.new_empty(z.shape[:1], dtype=torch.float32)
    lse = torch.empty_like(loss)
    buf, n = (None, 0) if ws is None else _check_ws(ws, z.device)
    L.check(L.lib().kan_distill_forward(desc, z.data_ptr(), ids_at, t_at, weight_at, loss.data_ptr(), lse.data_ptr(),
                                        _addr(buf), n, _raw_stream(dev)), "kan_distill_forward")
    return loss, lse


def kan_distill_backward(z, ids, t, lse, dloss, temperature=1.0, weight=None, grad_dtype=torch.float32, out=None):
    """``dz [N, V]`` in ``grad_dtype`` of the loss, from the forward's ``lse`` and
    the gradients ``dloss [N]`` of the rows' losses."""
    dev = _distill_inputs(z, ids, t, weight)
    _whole(lse, "lse", _F32, dev, z.shape[:1])
    _whole(dloss, "dloss", _F32, dev, z.shape[:1])
    ids_at, t_at, weight_at, lse_at, dloss_at = (ids.data_ptr(), t.data_ptr(), _addr(weight), lse.data_ptr(),
                                                 dloss.data_ptr())
    if (ids_at | t_at | (weight_at or 0) | lse_at | dloss_at) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_distill_backward(z, _placed(ids), _placed(t), _placed(lse), _placed(dloss), temperature,
                                        _placed(weight), grad_dtype, out)
    dz = _distill_grad(z, out, grad_dtype, dev)
    desc = distill_desc(z, ids, t, temperature, dz)
    L.check(L.lib().kan_distill_backward(desc, z.data_ptr(), ids_at, t_at, weight_at, lse_at, dloss_at, dz.data_ptr(),
                                         _raw_stream(dev)), "kan_distill_backward")
    return dz


def kan_distill_step(z, ids, t, temperature=1.0, weight=None, grad_dtype=torch.float32, out=None, ws=None):
    """``(loss [N], dz [N, V])`` in one call: the rows' losses and the gradient of
    their sum (put the mean's 1/N into ``weight``)."""
    dev = _distill_inputs(z, ids, t, weight)
    ids_at, t_at, weight_at = ids.data_ptr(), t.data_ptr(), _addr(weight)
    if (ids_at | t_at | (weight_at or 0)) & 15 or dev != _current():
        with torch.cuda.device(dev):
            return kan_distill_step(z, _placed(ids), _placed(t), temperature, _placed(weight), grad_dtype, out, ws)
    dz = _distill_grad(z, out, grad_dtype, dev)
    desc = distill_desc(z, ids, t, temperature, dz)
    loss = z.new_empty(z.shape[:1], dtype=torch.float32)
    lib = L.lib()
    buf, n = _sized_ws(ws, lib.kan_distill_workspace_size(desc), z)
    L.check(lib.kan_distill_step(desc, z.data_ptr(), ids_at, t_at, weight_at, loss.data_ptr(), dz.data_ptr(),
                                 _addr(buf), n, _raw_stream(dev)), "kan_distill_step")
    return loss, dz
