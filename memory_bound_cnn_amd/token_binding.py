"""ctypes binding of libwtconv's token operators (include/wtconv_tokens.h):
argument marshalling only.

Every entry point here has the name of the C function it calls and runs on the
current stream.  Tensors are PyTorch device tensors; the last axis is
contiguous, other strides are passed on.  Outputs are new tensors unless given.
"""

import ctypes

import torch

from . import binding
from .binding import WTC_BF16, WTC_FP32, WTC_OK, WTCError, _workspace

__all__ = [
    "wtc_rms_desc", "wtc_rotary_desc", "wtc_attn_strides", "wtc_attn_desc",
    "wtconv_rms_norm_forward", "wtconv_rms_norm_backward", "wtconv_rotary", "wtconv_dropout",
    "wtconv_attention_forward", "wtconv_attention_backward", "RMS_MAX_C", "ATTN_MAX_D",
    "wtc_layer_desc", "wtc_scan_desc", "wtc_rows_desc", "wtc_expert_desc",
    "wtconv_layer_norm_forward", "wtconv_layer_norm_backward", "wtconv_gated_scan_forward", "wtconv_gated_scan_backward",
    "wtconv_gated_scan_step", "wtconv_expert_order", "wtconv_expert_gather", "wtconv_expert_combine",
    "wtconv_expert_combine_backward", "wtconv_expert_linear_forward", "wtconv_expert_linear_input_grad",
    "wtconv_expert_linear_weight_grad", "EXPERTS_MAX",
]

RMS_MAX_C, ROTARY_MAX_AXES, ATTN_MAX_D, EXPERTS_MAX = 16384, 4, 128, 512   # limits in include/wtconv_tokens.h
_DTYPE = {torch.float32: WTC_FP32, torch.bfloat16: WTC_BF16}
_I, _LL, _P, _SZ = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t


class wtc_rms_desc(ctypes.Structure):
    _fields_ = [("rows", _LL), ("x_stride", _LL), ("r_stride", _LL), ("g_stride", _LL), ("C", _I), ("dtype", _I),
                ("fp8", _I), ("eps", ctypes.c_float)]


class wtc_rotary_desc(ctypes.Structure):
    _fields_ = [("T", _LL), ("x_token", _LL), ("x_head", _LL), ("y_token", _LL), ("y_head", _LL), ("heads", _I),
                ("D", _I), ("dtype", _I), ("axes", _I), ("pairs", _I * ROTARY_MAX_AXES), ("interleaved", _I),
                ("inverse", _I)]


class wtc_attn_strides(ctypes.Structure):
    _fields_ = [("token", _LL), ("head", _LL)]


class wtc_attn_desc(ctypes.Structure):
    _fields_ = ([("T", _LL), ("n_seq", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("dtype", _I), ("causal", _I),
                 ("scale", ctypes.c_float)]
                + [(name, wtc_attn_strides) for name in ("q", "k", "v", "o", "g", "dq", "dk", "dv")])


class wtc_layer_desc(ctypes.Structure):
    _fields_ = [("rows", _LL), ("x_stride", _LL), ("r_stride", _LL), ("g_stride", _LL), ("C", _I), ("dtype", _I),
                ("eps", ctypes.c_float)]


class wtc_scan_desc(ctypes.Structure):
    _fields_ = [("T", _LL), ("x_stride", _LL), ("f_stride", _LL), ("g_stride", _LL), ("n_seq", _I), ("C", _I),
                ("dtype", _I), ("reverse", _I)]


class wtc_rows_desc(ctypes.Structure):
    _fields_ = [("T", _LL), ("x_stride", _LL), ("r_stride", _LL), ("k", _I), ("E", _I), ("C", _I), ("dtype", _I)]


class wtc_expert_desc(ctypes.Structure):
    _fields_ = [("R", _LL), ("x_stride", _LL), ("g_stride", _LL), ("E", _I), ("K", _I), ("N", _I), ("dtype", _I)]


_lib = None


def _load():
    """libwtconv with the token operators' signatures."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        for name, args in (
                ("wtconv_rms_norm_forward", [_P] * 9),
                ("wtconv_rms_norm_backward", [_P] * 9 + [_SZ, _P]),
                ("wtconv_rotary", [_P] * 6),
                ("wtconv_dropout", [_LL, _I, ctypes.c_double] + [_P] * 5),
                ("wtconv_attention_forward", [_P] * 9 + [_SZ, _P]),
                ("wtconv_attention_backward", [_P] * 13 + [_SZ, _P]),
                ("wtconv_layer_norm_forward", [_P] * 9),
                ("wtconv_layer_norm_backward", [_P] * 10 + [_SZ, _P]),
                ("wtconv_gated_scan_forward", [_P] * 9 + [_SZ, _P]),
                ("wtconv_gated_scan_backward", [_P] * 12 + [_SZ, _P]),
                ("wtconv_gated_scan_step", [_P] * 7),
                ("wtconv_expert_order", [_LL, _I] + [_P] * 5 + [_SZ, _P]),
                ("wtconv_expert_gather", [_P] * 6),
                ("wtconv_expert_combine", [_P] * 6),
                ("wtconv_expert_combine_backward", [_P] * 9),
                ("wtconv_expert_linear_forward", [_P] * 7),
                ("wtconv_expert_linear_input_grad", [_P] * 6),
                ("wtconv_expert_linear_weight_grad", [_P] * 7 + [_SZ, _P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = _I, args
        for name in ("wtconv_rms_norm_backward_workspace", "wtconv_attention_forward_workspace",
                     "wtconv_attention_backward_workspace", "wtconv_layer_norm_backward_workspace",
                     "wtconv_gated_scan_kept", "wtconv_gated_scan_workspace", "wtconv_expert_linear_weight_grad_workspace"):
            f = getattr(lib, name)
            f.restype, f.argtypes = _SZ, [_P]
        lib.wtconv_expert_order_workspace.restype, lib.wtconv_expert_order_workspace.argtypes = _SZ, [_LL, _I]
        _lib = lib
    return _lib


def _call(name, device, *args):
    """Calls a C function on `device`'s current stream (its last argument)."""
    f = getattr(_lib or _load(), name)
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        st = f(*args, stream)
    else:
        with torch.cuda.device(index):
            st = f(*args, stream)
    if st != WTC_OK:
        raise WTCError(st, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _narrow(name, *sizes):
    """Sizes that the library takes as int: ctypes would take them modulo 2^32."""
    if any(n >= 1 << 31 for n in sizes):
        raise ValueError(f"{name}: a size of {max(sizes)} does not fit 32 bits")


def _check(t, name, dtype, device, shape, contiguous=False):
    """A device tensor of this type and shape whose last axis is contiguous
    (all of it, if asked)."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")


def _activation(t, name, dims=None):
    """An activation: its storage type, checked; any shape unless dims is given."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name} has dtype {t.dtype}, expected float32 or bfloat16")
    if dims is not None:
        if t.dim() != dims:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {dims} axes")
        _narrow(name, *t.shape[1:])
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return _DTYPE[t.dtype]


def wtconv_rms_norm_forward(x, weight, residual=None, eps=1e-6, fp8=False, want_rstd=False):
    """(y, h, rstd, scale) for x [rows, C]: h is None without a residual, rstd
    unless wanted, scale unless fp8 (y is then float8_e4m3fn)."""
    dtype = _activation(x, "x", 2)
    rows, C = x.shape
    dev = x.device
    _check(weight, "weight", torch.float32, dev, (C,), True)
    if residual is not None:
        _check(residual, "residual", x.dtype, dev, x.shape)
    y = torch.empty((rows, C), dtype=torch.float8_e4m3fn if fp8 else x.dtype, device=dev)
    h = None if residual is None else torch.empty((rows, C), dtype=x.dtype, device=dev)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if want_rstd else None
    scale = torch.empty(rows, dtype=torch.float32, device=dev) if fp8 else None
    d = wtc_rms_desc(rows, x.stride(0), 0 if residual is None else residual.stride(0), 0, C, dtype, fp8, eps)
    _call("wtconv_rms_norm_forward", dev, ctypes.addressof(d), x.data_ptr(), _ptr(residual), weight.data_ptr(),
          y.data_ptr(), _ptr(h), _ptr(rstd), _ptr(scale))
    return y, h, rstd, scale


def wtconv_rms_norm_backward(dy, dh, h, weight, rstd, eps=1e-6, workspace=None):
    """(dx, dw): dx is the gradient of x and of the residual.  h: the norm's
    input (x where there was no residual); dh: the gradient reaching h by its
    other use, or None."""
    dtype = _activation(h, "h", 2)
    rows, C = h.shape
    dev = h.device
    _check(dy, "dy", h.dtype, dev, h.shape)
    if dh is not None:
        _check(dh, "dh", h.dtype, dev, h.shape, True)
    _check(weight, "weight", torch.float32, dev, (C,), True)
    _check(rstd, "rstd", torch.float32, dev, (rows,), True)
    dx = torch.empty((rows, C), dtype=h.dtype, device=dev)
    dw = torch.empty(C, dtype=torch.float32, device=dev)
    d = wtc_rms_desc(rows, h.stride(0), 0, dy.stride(0), C, dtype, 0, eps)
    ws, size = _workspace(_load().wtconv_rms_norm_backward_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_rms_norm_backward", dev, ctypes.addressof(d), dy.data_ptr(), _ptr(dh), h.data_ptr(),
          weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), _ptr(ws), size)
    return dx, dw


def wtconv_rotary(x, positions, inv_freq, sections, interleaved=False, inverse=False, out=None):
    """x [T, heads, D] with its pairs turned.  positions [T, axes] int32,
    sections: pairs of each axis, inv_freq [sum(sections)] float32.  out may be
    x itself."""
    dtype = _activation(x, "x", 3)
    T, heads, D = x.shape
    dev = x.device
    axes, P = len(sections), sum(sections)
    if not 1 <= axes <= ROTARY_MAX_AXES:
        raise ValueError(f"{axes} sections: 1 to {ROTARY_MAX_AXES} axes are supported")
    _check(positions, "positions", torch.int32, dev, (T, axes), True)
    _check(inv_freq, "inv_freq", torch.float32, dev, (P,), True)
    if out is None:
        out = torch.empty((T, heads, D), dtype=x.dtype, device=dev)
    else:
        _check(out, "out", x.dtype, dev, x.shape)
        if out.data_ptr() == x.data_ptr() and out.stride() != x.stride():
            raise ValueError("out shares x's memory with other strides")
    d = wtc_rotary_desc(T, x.stride(0), x.stride(1), out.stride(0), out.stride(1), heads, D, dtype, axes,
                        tuple(sections), interleaved, inverse)
    _call("wtconv_rotary", dev, ctypes.addressof(d), x.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(),
          out.data_ptr())
    return out


def wtconv_dropout(x, p, rng, residual=None, out=None):
    """residual + x kept with probability 1 - p and divided by it.  rng: int64
    [2] on the device, seed and offset; x, residual, out contiguous."""
    dtype = _activation(x, "x")
    dev = x.device
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if residual is not None:
        _check(residual, "residual", x.dtype, dev, x.shape, True)
    _check(rng, "rng", torch.int64, dev, (2,), True)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", x.dtype, dev, x.shape, True)
    _call("wtconv_dropout", dev, x.numel(), dtype, p, x.data_ptr(), _ptr(residual), rng.data_ptr(), out.data_ptr())
    return out


def _attn_desc(q, k, v, cu_seqlens, causal, scale):
    dtype = _activation(q, "q", 3)
    T, Hq, D = q.shape
    dev = q.device
    Hk = k.shape[1] if k.dim() == 3 else 0
    _check(k, "k", q.dtype, dev, (T, Hk, D))
    _check(v, "v", q.dtype, dev, (T, Hk, D))
    if Hk < 1 or Hq % Hk:
        raise ValueError(f"{Hq} heads of q do not divide into {Hk} of k and v")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [n + 1]")
    _narrow("cu_seqlens", *cu_seqlens.shape)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, cu_seqlens.shape, True)
    d = wtc_attn_desc(T, cu_seqlens.shape[0] - 1, Hq, Hk, D, dtype, causal, D ** -0.5 if scale is None else scale)
    d.q, d.k, d.v = q.stride()[:2], k.stride()[:2], v.stride()[:2]
    return d


def wtconv_attention_forward(q, k, v, cu_seqlens, causal=False, scale=None, want_lse=False, out=None, out_low=None,
                             workspace=None):
    """(out, lse) for q [T, Hq, D], k and v [T, Hk, D]; lse [Hq, T] float32 or
    None.  scale: 1 / sqrt(D) unless given.  out_low: a contiguous bfloat16
    tensor of q's shape for what is rounded off out, or None."""
    d = _attn_desc(q, k, v, cu_seqlens, causal, scale)
    dev = q.device
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _check(out, "out", q.dtype, dev, q.shape)
    if out_low is not None:
        _check(out_low, "out_low", torch.bfloat16, dev, q.shape, True)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=dev) if want_lse else None
    d.o = out.stride()[:2]
    ws, size = _workspace(_load().wtconv_attention_forward_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_attention_forward", dev, ctypes.addressof(d), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          cu_seqlens.data_ptr(), out.data_ptr(), _ptr(lse), _ptr(out_low), _ptr(ws), size)
    return out, lse


def wtconv_attention_backward(q, k, v, out, lse, dout, cu_seqlens, causal=False, scale=None, grads=None,
                              workspace=None, out_low=None):
    """(dq, dk, dv).  out_low: as the forward pass left it, or None.  grads: the
    tensors to write them to (q's, k's and v's shapes, any strides that the
    library takes), or None."""
    d = _attn_desc(q, k, v, cu_seqlens, causal, scale)
    dev = q.device
    _check(out, "out", q.dtype, dev, q.shape)
    _check(dout, "dout", q.dtype, dev, q.shape)
    if out_low is not None:
        _check(out_low, "out_low", torch.bfloat16, dev, q.shape, True)
    _check(lse, "lse", torch.float32, dev, (q.shape[1], q.shape[0]), True)
    if grads is None:
        grads = tuple(torch.empty(t.shape, dtype=q.dtype, device=dev) for t in (q, k, v))
    for g, t, name in zip(grads, (q, k, v), ("dq", "dk", "dv")):
        _check(g, name, q.dtype, dev, t.shape)
    dq, dk, dv = grads
    d.o, d.g, d.dq, d.dk, d.dv = (t.stride()[:2] for t in (out, dout, dq, dk, dv))
    ws, size = _workspace(_load().wtconv_attention_backward_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_attention_backward", dev, ctypes.addressof(d), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), lse.data_ptr(), _ptr(out_low), dout.data_ptr(), cu_seqlens.data_ptr(), dq.data_ptr(), dk.data_ptr(),
          dv.data_ptr(), _ptr(ws), size)
    return dq, dk, dv


def wtconv_layer_norm_forward(x, weight, bias=None, residual=None, eps=1e-6, want_stats=False):
    """(y, h, stats) for x [rows, C]: h is None without a residual, stats [rows,
    2] (mean and reciprocal deviation) unless wanted."""
    dtype = _activation(x, "x", 2)
    rows, C = x.shape
    dev = x.device
    _check(weight, "weight", torch.float32, dev, (C,), True)
    if bias is not None:
        _check(bias, "bias", torch.float32, dev, (C,), True)
    if residual is not None:
        _check(residual, "residual", x.dtype, dev, x.shape)
    y = torch.empty((rows, C), dtype=x.dtype, device=dev)
    h = None if residual is None else torch.empty((rows, C), dtype=x.dtype, device=dev)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=dev) if want_stats else None
    d = wtc_layer_desc(rows, x.stride(0), 0 if residual is None else residual.stride(0), 0, C, dtype, eps)
    _call("wtconv_layer_norm_forward", dev, ctypes.addressof(d), x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias),
          y.data_ptr(), _ptr(h), _ptr(stats))
    return y, h, stats


def wtconv_layer_norm_backward(dy, dh, h, weight, stats, want_db=True, workspace=None):
    """(dx, dw, db): dx is the gradient of x and of the residual.  h: the norm's
    input; dh: the gradient reaching h by its other use, or None."""
    dtype = _activation(h, "h", 2)
    rows, C = h.shape
    dev = h.device
    _check(dy, "dy", h.dtype, dev, h.shape)
    if dh is not None:
        _check(dh, "dh", h.dtype, dev, h.shape, True)
    _check(weight, "weight", torch.float32, dev, (C,), True)
    _check(stats, "stats", torch.float32, dev, (rows, 2), True)
    dx = torch.empty((rows, C), dtype=h.dtype, device=dev)
    dw = torch.empty(C, dtype=torch.float32, device=dev)
    db = torch.empty(C, dtype=torch.float32, device=dev) if want_db else None
    d = wtc_layer_desc(rows, h.stride(0), 0, dy.stride(0), C, dtype, 0.0)
    ws, size = _workspace(_load().wtconv_layer_norm_backward_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_layer_norm_backward", dev, ctypes.addressof(d), dy.data_ptr(), _ptr(dh), h.data_ptr(), weight.data_ptr(),
          stats.data_ptr(), dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ws), size)
    return dx, dw, db


def _scan_desc(x, gate, cu_seqlens, state, reverse):
    dtype = _activation(x, "x", 2)
    dev = x.device
    _check(gate, "gate", x.dtype, dev, x.shape)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [n + 1]")
    _narrow("cu_seqlens", *cu_seqlens.shape)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, cu_seqlens.shape, True)
    n = cu_seqlens.shape[0] - 1
    if state is not None:
        _check(state, "state", torch.float32, dev, (n, x.shape[1]), True)
    return wtc_scan_desc(x.shape[0], x.stride(0), gate.stride(0), 0, n, x.shape[1], dtype, reverse)


def wtconv_gated_scan_forward(x, gate, cu_seqlens, state=None, reverse=False, want_kept=False, workspace=None):
    """(y, last, kept) for x and gate [T, C]: last [n, C] float32; kept, what the
    backward pass needs, unless wanted None."""
    d = _scan_desc(x, gate, cu_seqlens, state, reverse)
    dev = x.device
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    last = torch.empty((d.n_seq, x.shape[1]), dtype=torch.float32, device=dev)
    lib = _load()
    kept = torch.empty(lib.wtconv_gated_scan_kept(ctypes.addressof(d)) // 4, dtype=torch.float32, device=dev) if want_kept else None
    ws, size = _workspace(lib.wtconv_gated_scan_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_gated_scan_forward", dev, ctypes.addressof(d), x.data_ptr(), gate.data_ptr(), cu_seqlens.data_ptr(),
          _ptr(state), y.data_ptr(), last.data_ptr(), _ptr(kept), _ptr(ws), size)
    return y, last, kept


def wtconv_gated_scan_backward(dy, dlast, x, gate, cu_seqlens, state, kept, reverse=False, workspace=None):
    """(dx, dgate, dstate): dlast or None (zeros); dstate None without a state."""
    d = _scan_desc(x, gate, cu_seqlens, state, reverse)
    dev = x.device
    _check(dy, "dy", x.dtype, dev, x.shape)
    if dlast is not None:
        _check(dlast, "dlast", torch.float32, dev, (d.n_seq, x.shape[1]), True)
    d.g_stride = dy.stride(0)
    lib = _load()
    _check(kept, "kept", torch.float32, dev, (lib.wtconv_gated_scan_kept(ctypes.addressof(d)) // 4,), True)
    dx, dgate = (torch.empty(x.shape, dtype=x.dtype, device=dev) for _ in range(2))
    dstate = None if state is None else torch.empty_like(state)
    ws, size = _workspace(lib.wtconv_gated_scan_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_gated_scan_backward", dev, ctypes.addressof(d), x.data_ptr(), gate.data_ptr(), cu_seqlens.data_ptr(),
          _ptr(state), kept.data_ptr(), dy.data_ptr(), _ptr(dlast), dx.data_ptr(), dgate.data_ptr(), _ptr(dstate), _ptr(ws), size)
    return dx, dgate, dstate


def wtconv_gated_scan_step(x, gate, state, out=None):
    """(y, new state) of one more token of each of n sequences.  out may be state."""
    dtype = _activation(x, "x", 2)
    dev = x.device
    _check(gate, "gate", x.dtype, dev, x.shape)
    _check(state, "state", torch.float32, dev, x.shape, True)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float32, device=dev)
    else:
        _check(out, "out", torch.float32, dev, x.shape, True)
    d = wtc_scan_desc(x.shape[0], x.stride(0), gate.stride(0), 0, 0, x.shape[1], dtype, 0)
    _call("wtconv_gated_scan_step", dev, ctypes.addressof(d), x.data_ptr(), gate.data_ptr(), state.data_ptr(), y.data_ptr(),
          out.data_ptr())
    return y, out


def wtconv_expert_order(experts, E, workspace=None):
    """(slot, pair, cu_experts) of experts [T, k] int32."""
    if not experts.is_cuda:
        raise ValueError("experts must be a CUDA tensor")
    dev = experts.device
    if experts.dim() != 2:
        raise ValueError(f"experts has shape {tuple(experts.shape)}, expected [T, k]")
    _check(experts, "experts", torch.int32, dev, experts.shape, True)
    _narrow("experts", E)
    n = experts.numel()
    slot = torch.empty_like(experts)
    pair = torch.empty(n, dtype=torch.int32, device=dev)
    cu = torch.empty(max(E, 0) + 1, dtype=torch.int32, device=dev)
    ws, size = _workspace(_load().wtconv_expert_order_workspace(n, E), dev, workspace)
    _call("wtconv_expert_order", dev, n, E, experts.data_ptr(), slot.data_ptr(), pair.data_ptr(), cu.data_ptr(), _ptr(ws), size)
    return slot, pair, cu


def _rows_desc(t, name, slot, cu_experts):
    dtype = _activation(t, name, 2)
    if slot.dim() != 2 or slot.shape[1] < 1:
        raise ValueError(f"slot has shape {tuple(slot.shape)}, expected [T, k]")
    _check(slot, "slot", torch.int32, t.device, slot.shape, True)
    E = 1
    if cu_experts is not None:
        if cu_experts.dim() != 1 or cu_experts.shape[0] < 2:
            raise ValueError("cu_experts must be [E + 1]")
        _check(cu_experts, "cu_experts", torch.int32, t.device, cu_experts.shape, True)
        E = cu_experts.shape[0] - 1
    _narrow("slot", slot.shape[1], E)
    return wtc_rows_desc(slot.shape[0], 0, 0, slot.shape[1], E, t.shape[1], dtype)


def wtconv_expert_gather(x, slot, cu_experts):
    """x [T, C] to the rows [T k, C] of slot [T, k]."""
    d = _rows_desc(x, "x", slot, cu_experts)
    if x.shape[0] != slot.shape[0]:
        raise ValueError(f"x has {x.shape[0]} rows, slot {slot.shape[0]}")
    d.x_stride = x.stride(0)
    rows = torch.empty((slot.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
    _call("wtconv_expert_gather", x.device, ctypes.addressof(d), x.data_ptr(), slot.data_ptr(), cu_experts.data_ptr(),
          rows.data_ptr())
    return rows


def wtconv_expert_combine(rows, weights, slot):
    """The sum of each token's rows, with weights [T, k] float32 or None (ones)."""
    d = _rows_desc(rows, "rows", slot, None)
    if rows.shape[0] != slot.numel():
        raise ValueError(f"rows has {rows.shape[0]} rows, slot {slot.numel()} places")
    if weights is not None:
        _check(weights, "weights", torch.float32, rows.device, slot.shape, True)
    d.r_stride = rows.stride(0)
    y = torch.empty((slot.shape[0], rows.shape[1]), dtype=rows.dtype, device=rows.device)
    _call("wtconv_expert_combine", rows.device, ctypes.addressof(d), rows.data_ptr(), _ptr(weights), slot.data_ptr(), y.data_ptr())
    return y


def wtconv_expert_combine_backward(dy, rows, weights, slot, cu_experts):
    """(drows, dweights)"""
    d = _rows_desc(rows, "rows", slot, cu_experts)
    dev = rows.device
    if rows.shape[0] != slot.numel():
        raise ValueError(f"rows has {rows.shape[0]} rows, slot {slot.numel()} places")
    _check(weights, "weights", torch.float32, dev, slot.shape, True)
    _check(dy, "dy", rows.dtype, dev, (slot.shape[0], rows.shape[1]))
    d.x_stride, d.r_stride = dy.stride(0), rows.stride(0)
    drows = torch.empty(rows.shape, dtype=rows.dtype, device=dev)
    dweights = torch.empty(slot.shape, dtype=torch.float32, device=dev)
    _call("wtconv_expert_combine_backward", dev, ctypes.addressof(d), dy.data_ptr(), rows.data_ptr(), weights.data_ptr(),
          slot.data_ptr(), cu_experts.data_ptr(), drows.data_ptr(), dweights.data_ptr())
    return drows, dweights


def _expert_desc(t, name, K, N, E, cu_experts):
    dtype = _activation(t, name, 2)
    _check(cu_experts, "cu_experts", torch.int32, t.device, (E + 1,), True)
    _narrow("weight", K, N, E)
    return wtc_expert_desc(t.shape[0], 0, 0, E, K, N, dtype)


def wtconv_expert_linear_forward(x, weight, cu_experts, bias=None):
    """x [R, K] weight[e]^T + bias[e], weight [E, N, K]."""
    if weight.dim() != 3:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected [E, N, K]")
    E, N, K = weight.shape
    d = _expert_desc(x, "x", K, N, E, cu_experts)
    dev = x.device
    _check(x, "x", x.dtype, dev, (x.shape[0], K))
    _check(weight, "weight", x.dtype, dev, weight.shape, True)
    if bias is not None:
        _check(bias, "bias", x.dtype, dev, (E, N), True)
    d.x_stride = x.stride(0)
    y = torch.empty((x.shape[0], N), dtype=x.dtype, device=dev)
    _call("wtconv_expert_linear_forward", dev, ctypes.addressof(d), x.data_ptr(), weight.data_ptr(), _ptr(bias),
          cu_experts.data_ptr(), y.data_ptr())
    return y


def wtconv_expert_linear_input_grad(dy, weight, cu_experts):
    """dy [R, N] weight[e], weight [E, N, K]."""
    if weight.dim() != 3:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected [E, N, K]")
    E, N, K = weight.shape
    d = _expert_desc(dy, "dy", K, N, E, cu_experts)
    dev = dy.device
    _check(dy, "dy", dy.dtype, dev, (dy.shape[0], N))
    _check(weight, "weight", dy.dtype, dev, weight.shape, True)
    d.g_stride = dy.stride(0)
    dx = torch.empty((dy.shape[0], K), dtype=dy.dtype, device=dev)
    _call("wtconv_expert_linear_input_grad", dev, ctypes.addressof(d), dy.data_ptr(), weight.data_ptr(), cu_experts.data_ptr(),
          dx.data_ptr())
    return dx


def wtconv_expert_linear_weight_grad(dy, x, cu_experts, want_db=True, workspace=None):
    """(dweight [E, N, K], dbias [E, N] or None) for dy [R, N] and x [R, K]."""
    _activation(dy, "dy", 2)
    E = cu_experts.shape[0] - 1
    d = _expert_desc(x, "x", x.shape[1], dy.shape[1], E, cu_experts)
    dev = x.device
    _check(dy, "dy", x.dtype, dev, (x.shape[0], dy.shape[1]))
    d.x_stride, d.g_stride = x.stride(0), dy.stride(0)
    dw = torch.empty((E, dy.shape[1], x.shape[1]), dtype=x.dtype, device=dev)
    db = torch.empty((E, dy.shape[1]), dtype=x.dtype, device=dev) if want_db else None
    ws, size = _workspace(_load().wtconv_expert_linear_weight_grad_workspace(ctypes.addressof(d)), dev, workspace)
    _call("wtconv_expert_linear_weight_grad", dev, ctypes.addressof(d), dy.data_ptr(), x.data_ptr(), cu_experts.data_ptr(),
          dw.data_ptr(), _ptr(db), _ptr(ws), size)
    return dw, db
