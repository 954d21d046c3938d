"""Operators over tokens with their gradients, and a block made of them.

A pixel of a channels-last plane is a token: B planes of H x W pixels are
B H W rows, and images of different sizes are packed one after another, with
their first rows in ``cu_seqlens``.

``rms_norm``, ``rms_norm_fp8``, ``rotary``, ``attention``, ``rotary_attention``
and ``dropout`` run in libwtconv's kernels (include/wtconv_tokens.h) on the
current stream and have gradients, except ``rms_norm_fp8``.  ``TokenBlock``
runs them together.
"""

import torch

from . import token_binding as tb

__all__ = ["rms_norm", "rms_norm_fp8", "rotary", "attention", "rotary_attention", "dropout", "image_positions",
           "rotary_frequencies", "RMSNorm", "TokenBlock"]


def _wants_grad(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _rows(t):
    """t as [rows, C] whose last axis is contiguous; a view where t allows it."""
    t = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    return t if t.stride(1) == 1 or t.shape[1] == 1 else t.contiguous()


def _dense(t):
    """t with a contiguous last axis."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _heads(t):
    """t [T, heads, D] as the attention kernels read it: tokens and heads start
    at multiples of 16 bytes; a copy where they do not."""
    unit = 16 // t.element_size()
    if t.stride(2) == 1 and t.stride(0) % unit == 0 and t.stride(1) % unit == 0 and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


# ------------------------------------------------------------------ root-mean-square norm
class _RMSNorm(torch.autograd.Function):
    """Saves the norm's input (h, or x without a residual) and one float per row."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        xr = _rows(x)
        y, h, rstd, _ = tb.wtconv_rms_norm_forward(xr, weight, None if residual is None else _rows(residual), eps,
                                                   want_rstd=True)
        if x.dim() != 2:
            y, h = y.view(x.shape), None if h is None else h.view(x.shape)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        if dy is None:
            return dh, None, dh, None
        dx, dw = tb._rms_norm_backward(_rows(dy), None if dh is None else _rows(dh).contiguous(), _rows(h), weight,
                                       rstd, ctx.eps)
        if h.dim() != 2:
            dx = dx.view(h.shape)
        return dx, dw, dx if ctx.needs_input_grad[2] else None, None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last axis, h = x +
    residual in x's type.  Returns y, or (y, h) with a residual.  x [..., C]
    float32 or bfloat16, weight [C] float32."""
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
    if _wants_grad(x, weight, residual):
        y, h = _RMSNorm.apply(x, weight, residual, eps)
    else:
        y, h, _, _ = tb.wtconv_rms_norm_forward(_rows(x), weight, None if residual is None else _rows(residual), eps)
        if x.dim() != 2:
            y, h = y.view(x.shape), None if h is None else h.view(x.shape)
    return y if residual is None else (y, h)


def rms_norm_fp8(x, weight, residual=None, eps=1e-6):
    """:func:`rms_norm` with its result in 8 bits: (y8, scale, h), y = y8 *
    scale[..., None] with y8 float8_e4m3fn and one float32 scale per row; h is
    None without a residual.  No gradient."""
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
    if _wants_grad(x, weight, residual):
        raise ValueError("rms_norm_fp8 has no gradient; call it under torch.no_grad()")
    y, h, _, scale = tb.wtconv_rms_norm_forward(_rows(x), weight, None if residual is None else _rows(residual), eps,
                                                fp8=True)
    return y.view(x.shape), scale.view(x.shape[:-1]), None if h is None else h.view(x.shape)


# ------------------------------------------------------------------ rotary positions
class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, inv_freq, sections, interleaved):
        ctx.sections, ctx.interleaved = sections, interleaved
        ctx.save_for_backward(positions, inv_freq)
        return tb.wtconv_rotary(_dense(x), positions, inv_freq, sections, interleaved)

    @staticmethod
    def backward(ctx, g):
        positions, inv_freq = ctx.saved_tensors
        dx = tb._rotary(_dense(g), positions, inv_freq, ctx.sections, ctx.interleaved, True,
                        torch.empty(g.shape, dtype=g.dtype, device=g.device))
        return dx, None, None, None, None


def rotary(x, positions, inv_freq, sections, interleaved=False):
    """x [T, heads, D] with channel pairs turned by position angles: pair p of
    axis a by positions[t, a] * inv_freq[p].  sections: the pairs of each axis
    (1 to 4 axes), sum(sections) <= D / 2; channels past the pairs stay.  Pairs
    are (p, sum(sections) + p), or (2p, 2p + 1) if interleaved.  positions [T,
    axes] int32, inv_freq [sum(sections)] float32; gradients of x only."""
    sections = tuple(int(n) for n in sections)
    if _wants_grad(x):
        return _Rotary.apply(x, positions, inv_freq, sections, interleaved)
    return tb.wtconv_rotary(_dense(x), positions, inv_freq, sections, interleaved)


def rotary_frequencies(sections, base=10000.0, device=None):
    """inv_freq: base^(-j / n) for pair j of an axis's n."""
    return torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections]).float().to(device)


def image_positions(sizes, device=None):
    """(positions, cu_seqlens) of images of sizes [(H, W), ...] packed one after
    another, pixels in row order: positions [T, 2] = (row, column), int32."""
    at = [torch.stack(torch.meshgrid(torch.arange(h), torch.arange(w), indexing="ij"), -1).reshape(-1, 2)
          for h, w in sizes]
    cu = torch.tensor([0] + [h * w for h, w in sizes]).cumsum(0)
    at = torch.cat(at) if at else torch.zeros(0, 2)
    return at.to(device=device, dtype=torch.int32), cu.to(device=device, dtype=torch.int32)


# ------------------------------------------------------------------ attention
class _Attention(torch.autograd.Function):
    """Saves its inputs, its output and one float per query and head."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, causal, scale):
        q, k, v = _heads(q), _heads(k), _heads(v)
        out, lse = tb.wtconv_attention_forward(q, k, v, cu_seqlens, causal, scale, want_lse=True)
        ctx.causal, ctx.scale = causal, scale
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        return out

    @staticmethod
    def backward(ctx, g):
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        return tb._attention_backward(q, k, v, out, lse, _heads(g), cu_seqlens, ctx.causal, ctx.scale) + \
            (None, None, None)


def attention(q, k, v, cu_seqlens, causal=False, scale=None):
    """softmax(scale q k^T) v inside each sequence of a pack: q [T, Hq, D], k
    and v [T, Hk, D] (views of one projection, or separate), Hq a multiple of
    Hk, D a multiple of 8 up to 128.  cu_seqlens [n + 1] int32 on the device:
    the first token of each sequence and the end; tokens of no sequence get
    zeros.  causal: a token sees itself and those before it.  scale: 1 /
    sqrt(D) unless given."""
    if _wants_grad(q, k, v):
        return _Attention.apply(q, k, v, cu_seqlens, causal, scale)
    return tb.wtconv_attention_forward(_heads(q), _heads(k), _heads(v), cu_seqlens, causal, scale)[0]


class _RotaryAttention(torch.autograd.Function):
    """rotary on q and k, then attention, on one projection: the gradients are
    written where the projection's are wanted, and turned back there."""

    @staticmethod
    def forward(ctx, qkv, Hq, Hk, positions, inv_freq, sections, cu_seqlens, interleaved, causal, scale):
        qkv = _heads(qkv)
        qk = tb.wtconv_rotary(qkv[:, :Hq + Hk], positions, inv_freq, sections, interleaved)
        out, lse = tb.wtconv_attention_forward(qk[:, :Hq], qk[:, Hq:], qkv[:, Hq + Hk:], cu_seqlens, causal, scale,
                                               want_lse=True)
        ctx.at = (Hq, Hk, sections, interleaved, causal, scale)
        ctx.save_for_backward(qkv, qk, out, lse, positions, inv_freq, cu_seqlens)
        return out

    @staticmethod
    def backward(ctx, g):
        Hq, Hk, sections, interleaved, causal, scale = ctx.at
        qkv, qk, out, lse, positions, inv_freq, cu_seqlens = ctx.saved_tensors
        d = torch.empty(qkv.shape, dtype=qkv.dtype, device=qkv.device)
        dqk = d[:, :Hq + Hk]
        tb._attention_backward(qk[:, :Hq], qk[:, Hq:], qkv[:, Hq + Hk:], out, lse, _heads(g), cu_seqlens, causal, scale,
                               grads=(d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]))
        tb._rotary(dqk, positions, inv_freq, sections, interleaved, True, dqk)
        return (d,) + (None,) * 9


def rotary_attention(qkv, Hq, Hk, positions, inv_freq, sections, cu_seqlens, interleaved=False, causal=False,
                     scale=None):
    """:func:`attention` of a projection qkv [T, Hq + 2 Hk, D] whose q and k
    are turned first (:func:`rotary`); its gradient is one tensor of qkv's
    shape, with no copies between."""
    if qkv.dim() != 3 or qkv.shape[1] != Hq + 2 * Hk:
        raise ValueError(f"qkv has shape {tuple(qkv.shape)}, expected [T, {Hq + 2 * Hk}, D]")
    return _RotaryAttention.apply(qkv, Hq, Hk, positions, inv_freq, tuple(int(n) for n in sections), cu_seqlens,
                                  interleaved, causal, scale)


# ------------------------------------------------------------------ dropout
class _Dropout(torch.autograd.Function):
    """Saves the generator's two words; the decisions are drawn again."""

    @staticmethod
    def forward(ctx, x, p, rng, residual):
        ctx.p = p
        ctx.save_for_backward(rng)
        return tb.wtconv_dropout(x.contiguous(), p, rng, None if residual is None else residual.contiguous())

    @staticmethod
    def backward(ctx, g):
        rng, = ctx.saved_tensors
        dx = None
        if ctx.needs_input_grad[0]:
            dx = tb._dropout(g.contiguous(), ctx.p, rng, None, torch.empty(g.shape, dtype=g.dtype, device=g.device))
        return dx, None, None, g if ctx.needs_input_grad[3] else None


def dropout(x, p, rng, residual=None):
    """residual + x where x is kept, with probability 1 - p, and divided by it.
    rng: int64 [2] on the device, (seed, offset); the same rng keeps the same
    elements, so every call of a step takes another offset.  p is taken to
    multiples of 2^-16."""
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
    if _wants_grad(x, residual):
        return _Dropout.apply(x, p, rng, residual)
    return tb.wtconv_dropout(x.contiguous(), p, rng, None if residual is None else residual.contiguous())


# ------------------------------------------------------------------ modules
class RMSNorm(torch.nn.Module):
    """:func:`rms_norm` with its weight."""

    def __init__(self, channels, eps=1e-6, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(channels, dtype=torch.float32, device=device))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps)


class TokenBlock(torch.nn.Module):
    """Pre-norm attention and two-layer branch over packed tokens:
        h = x + dropout(proj(attention(rotary(qkv(norm(x))))))
        out = h + dropout(down(gelu(up(norm(h)))))
    x [T, C], C = heads * D; kv_heads heads of k and v; sections: rotary pairs
    of each position axis (half of D / 2 each for images unless given)."""

    def __init__(self, channels, heads, kv_heads=None, sections=None, hidden=None, p=0.0, causal=False, seed=0,
                 device=None, dtype=torch.bfloat16):
        super().__init__()
        if channels % heads:
            raise ValueError(f"{channels} channels do not divide into {heads} heads")
        self.heads, self.kv_heads, self.D = heads, kv_heads or heads, channels // heads
        self.sections = tuple(sections) if sections else (self.D // 2 - self.D // 4, self.D // 4)
        self.p, self.causal = p, causal
        f = dict(device=device, dtype=dtype)
        self.norm1, self.norm2 = RMSNorm(channels, device=device), RMSNorm(channels, device=device)
        self.qkv = torch.nn.Linear(channels, (heads + 2 * self.kv_heads) * self.D, bias=False, **f)
        self.proj = torch.nn.Linear(channels, channels, bias=False, **f)
        self.up = torch.nn.Linear(channels, hidden or 4 * channels, **f)
        self.down = torch.nn.Linear(hidden or 4 * channels, channels, **f)
        self.register_buffer("inv_freq", rotary_frequencies(self.sections, device=device))
        self.register_buffer("rng", torch.tensor([seed, 0], device=device))

    def _dropout(self, x, residual):
        if not self.training or self.p == 0.0:
            return residual + x
        rng = self.rng.clone()   # this call's words; the next one takes another offset
        self.rng[1] += 1
        return dropout(x, self.p, rng, residual)

    def forward(self, x, positions, cu_seqlens):
        T = x.shape[0]
        qkv = self.qkv(self.norm1(x)).view(T, -1, self.D)
        a = rotary_attention(qkv, self.heads, self.kv_heads, positions, self.inv_freq, self.sections, cu_seqlens,
                             causal=self.causal)
        h = self._dropout(self.proj(a.reshape(T, -1)), x)
        return self._dropout(self.down(torch.nn.functional.gelu(self.up(self.norm2(h)))), h)
