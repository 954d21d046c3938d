"""Operators over tokens with their gradients, and a block made of them.

A pixel of a channels-last plane is a token: B planes of H x W pixels are
B H W rows, and images of different sizes are packed one after another, with
their first rows in ``cu_seqlens``.

``rms_norm``, ``rms_norm_fp8``, ``rotary``, ``attention``, ``rotary_attention``
and ``dropout`` run in libwtconv's kernels (include/wtconv_tokens.h) on the
current stream and have gradients (first ones only), except ``rms_norm_fp8``.
``TokenBlock`` runs them together.  So do ``layer_norm``, ``gated_scan`` and the
``expert_`` functions, and ``ScanBlock``, for planes too large for attention,
runs those together; ``gated_scan_step`` and ``expert_order`` have no gradient.

They go through the extension module ``_tokens`` (csrc/wtconv_tok_torch.cpp),
which is loaded by the first call and must have been built; ``token_binding``
has the same kernels without gradients, as the C functions.  The module
registers them as ``torch.ops.wtconv_tokens``, which is what traces hold: load
it (any call does) before running one that was saved.

Steps of small packs wait for the host, and most of that for PyTorch's handing
the backward pass to a thread of its own: within
``torch.autograd.set_multithreading_enabled(False)`` a forward and a backward
pass of 8 tokens take 32 us (norm) and 31 us (attention) instead of 75 and 72.

Forward and backward passes can be captured into graphs.  A backward pass is not,
while an eager pass of the same leaves lives: PyTorch ties a leaf's gradient to
the stream on which the leaf was used first.  ``layer_norm``, ``gated_scan`` and
the ``expert_`` functions refuse it for all leaves behind them, through whatever
other operators; leaves that a pass reaches before the first of these functions
(a linear layer's behind the last of them) are not looked at.
"""

from typing import NamedTuple

import torch

__all__ = ["rms_norm", "rms_norm_fp8", "rotary", "attention", "rotary_attention", "dropout", "layer_norm", "gated_scan",
           "gated_scan_step", "ExpertOrder", "expert_order", "expert_gather", "expert_linear", "expert_combine",
           "image_positions", "rotary_frequencies", "RMSNorm", "TokenBlock", "LayerNorm", "Experts", "ScanBlock"]

_ops = None


def _load():
    global _ops
    if _ops is None:
        try:
            from . import _tokens
        except ImportError as e:
            raise RuntimeError(f"the token operators are not built ({e}); run `python -m memory_bound_cnn_amd.build`") \
                from e
        _ops = _tokens
    return _ops


def rms_norm(x, weight, residual=None, eps=1e-6):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last axis, h = x +
    residual in x's type.  Returns y, or (y, h) with a residual.  x [..., C]
    float32 or bfloat16, weight [C] float32."""
    y, *h = (_ops or _load()).rms_norm(x, weight, residual, eps)
    return (y, *h) if h else y


def rms_norm_fp8(x, weight, residual=None, eps=1e-6):
    """:func:`rms_norm` with its result in 8 bits: (y8, scale, h), y = y8 *
    scale[..., None] with y8 float8_e4m3fn and one float32 scale per row; h is
    None without a residual.  No gradient."""
    y, scale, *h = (_ops or _load()).rms_norm_fp8(x, weight, residual, eps)
    return y, scale, h[0] if h else None


def rotary(x, positions, inv_freq, sections, interleaved=False):
    """x [T, heads, D] with channel pairs turned by position angles: pair p of
    axis a by positions[t, a] * inv_freq[p].  sections: the pairs of each axis
    (1 to 4 axes), sum(sections) <= D / 2; channels past the pairs stay.  Pairs
    are (p, sum(sections) + p), or (2p, 2p + 1) if interleaved.  positions [T,
    axes] int32, inv_freq [sum(sections)] float32; gradients of x only."""
    return (_ops or _load()).rotary(x, positions, inv_freq, sections, interleaved)


def attention(q, k, v, cu_seqlens, causal=False, scale=None):
    """softmax(scale q k^T) v inside each sequence of a pack: q [T, Hq, D], k
    and v [T, Hk, D] (views of one projection, or separate), Hq a multiple of
    Hk, D a multiple of 8 up to 128.  cu_seqlens [n + 1] int32 on the device:
    the first token of each sequence and the end; tokens of no sequence get
    zeros.  causal: a token sees itself and those before it.  scale: 1 /
    sqrt(D) unless given."""
    return (_ops or _load()).attention(q, k, v, cu_seqlens, causal, scale)


def rotary_attention(qkv, Hq, Hk, positions, inv_freq, sections, cu_seqlens, interleaved=False, causal=False,
                     scale=None):
    """:func:`attention` of a projection qkv [T, Hq + 2 Hk, D] whose q and k
    are turned first (:func:`rotary`); its gradient is one tensor of qkv's
    shape, with no copies between."""
    if qkv.dim() != 3 or qkv.shape[1] != Hq + 2 * Hk:
        raise ValueError(f"qkv has shape {tuple(qkv.shape)}, expected [T, {Hq + 2 * Hk}, D]")
    return (_ops or _load()).rotary_attention(qkv, Hq, Hk, positions, inv_freq, sections, cu_seqlens, interleaved,
                                              causal, scale)


def dropout(x, p, rng, residual=None):
    """residual + x where x is kept, with probability 1 - p, and divided by it.
    rng: int64 [2] on the device, (seed, offset); the same rng keeps the same
    elements, so every call of a step takes another offset.  p is taken to
    multiples of 2^-16."""
    return (_ops or _load()).dropout(x, p, rng, residual)


def layer_norm(x, weight, bias=None, residual=None, eps=1e-6):
    """y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias over the last
    axis, h = x + residual in x's type.  Returns y, or (y, h) with a residual.
    x [..., C] float32 or bfloat16, C up to 16384, weight and bias [C] float32."""
    y, *h = (_ops or _load()).layer_norm(x, weight, bias, residual, eps)
    return (y, *h) if h else y


def gated_scan(x, gate, cu_seqlens, state=None, reverse=False):
    """h_t = a_t h_(t-1) + (1 - a_t) x_t along each sequence of a pack, a =
    sigmoid(gate): (y, last).  x and gate [T, C] (views of one projection, or
    separate), y is h in x's type; h itself is float32.  cu_seqlens [n + 1] int32
    as for :func:`attention`; tokens of no sequence get zeros.  state [n, C]
    float32: what each sequence starts from, zeros unless given; last [n, C]
    float32: what it leaves.  reverse: from the last token to the first.  With
    gradients, half a byte a channel and token is kept beside the inputs.
    An infinity in a state, or in its gradient, stays one to the sequence's end (a
    NaN with one of the other sign); finite states and x are to stay below 2^127, as
    differences of two are taken."""
    y, last = (_ops or _load()).gated_scan(x, gate, cu_seqlens, state, reverse)
    return y, last


def gated_scan_step(x, gate, state, out=None):
    """:func:`gated_scan` of one more token of each sequence: (y, new state).  x
    and gate [n, C], state [n, C] float32.  out: where the new state goes (state
    itself, in a loop or a captured graph); a new tensor unless given.  No gradient."""
    return (_ops or _load()).gated_scan_step(x, gate, state, out)


class ExpertOrder(NamedTuple):
    """Pairs of a token and one of its k experts (pair t k + j) in the order of
    the experts, those of one in the order of the pairs.  int32."""
    slot: torch.Tensor         # [T, k]: each pair's place, -1 for pairs of no expert
    pair: torch.Tensor         # [T k]: the pair at each place, -1 past the last one
    cu_experts: torch.Tensor   # [E + 1]: expert e's places are cu_experts[e] up to cu_experts[e + 1]


def expert_order(experts, n_experts):
    """The order of tokens by expert.  experts [T, k] int32; a number outside of 0
    .. n_experts - 1 (-1, for a token that only pads a batch) is no expert's.
    n_experts up to 512."""
    return ExpertOrder(*(_ops or _load()).expert_order(experts, n_experts))


def expert_gather(x, order):
    """x [T, C] to the rows of the experts, [T k, C] in the order of ``order``
    (:func:`expert_order`); rows of no pair are zeros."""
    return (_ops or _load()).expert_gather(x, order.slot, order.cu_experts)


def expert_linear(x, weight, cu_experts, bias=None):
    """x weight[e]^T + bias[e] for the rows of each expert e, cu_experts[e] up to
    cu_experts[e + 1]; zeros for the rows of none.  x [R, K], weight [E, N, K] and
    bias [E, N] in x's type, K and N multiples of 8; cu_experts [E + 1] int32.
    float32 is computed to float32's precision, but from bfloat16 parts: finite
    values above 3.3895e38 count as infinite, and an infinity may give a NaN."""
    return (_ops or _load()).expert_linear(x, weight, bias, cu_experts)


def expert_combine(rows, weights, order):
    """The rows of the experts [T k, C] back to their tokens: y[t] = sum over j of
    weights[t, j] times the row of pair (t, j).  weights [T, k] float32."""
    return (_ops or _load()).expert_combine(rows, weights, order.slot, order.cu_experts)


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


# ------------------------------------------------------------------ modules
def _keep_dtype(fn):
    """A module's conversion that leaves types alone: what the operators take as
    float32 is not rounded by ``module.to(torch.bfloat16)``."""
    def convert(t):
        new = fn(t)
        return new if new.dtype == t.dtype else t.to(new.device)
    return convert


class RMSNorm(torch.nn.Module):
    """:func:`rms_norm` with its weight, which stays float32."""

    def __init__(self, channels, eps=1e-6, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(channels, dtype=torch.float32, device=device))

    def _apply(self, fn, recurse=True):
        return super()._apply(_keep_dtype(fn), recurse)

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps)


class TokenBlock(torch.nn.Module):
    """Pre-norm attention and two-layer branch over packed tokens:
        h = x + dropout(proj(attention(rotary(qkv(norm(x))))))
        out = h + dropout(down(gelu(up(norm(h)))))
    x [T, C], C = heads * D; kv_heads heads of k and v; sections: rotary pairs
    of each position axis (half of D / 2 each for images unless given).

    What a pass drops follows from a key that it draws from PyTorch's generator
    of the block's device: ``torch.manual_seed`` sets it, every block and pass
    gets its own, and activation checkpointing, which restores that generator,
    drops the same elements again.  seed tells blocks apart whose generators
    are in the same state (the ranks of a job that all started from one)."""

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
        # generator words of the latest pass: its key, and the offset after those of its two dropouts (0 and 1)
        self.register_buffer("rng", torch.tensor([0, 2], device=device))
        self.register_buffer("_to_words", torch.tensor([[seed, -2], [seed, -1]], device=device), persistent=False)

    def _apply(self, fn, recurse=True):
        inv_freq = self.inv_freq
        super()._apply(fn, recurse)
        self.inv_freq = _keep_dtype(fn)(inv_freq)
        return self

    def _dropout(self, x, residual, rng):
        if rng is None:
            return residual + x
        return dropout(x.to(residual.dtype), self.p, rng, residual)   # another type under autocast

    def forward(self, x, positions, cu_seqlens):
        T = x.shape[0]
        rng = (None, None)
        if self.training and self.p > 0.0:
            self.rng[0].random_()
            rng = self.rng + self._to_words   # new memory: it is saved for the backward pass
        qkv = self.qkv(self.norm1(x)).view(T, -1, self.D)
        a = rotary_attention(qkv, self.heads, self.kv_heads, positions, self.inv_freq, self.sections, cu_seqlens,
                             causal=self.causal)
        h = self._dropout(self.proj(a.reshape(T, -1)), x, rng[0])
        return self._dropout(self.down(torch.nn.functional.gelu(self.up(self.norm2(h)))), h, rng[1])


class LayerNorm(torch.nn.Module):
    """:func:`layer_norm` with its weight and bias, which stay float32."""

    def __init__(self, channels, eps=1e-6, bias=True, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(channels, dtype=torch.float32, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(channels, dtype=torch.float32, device=device)) if bias else None

    def _apply(self, fn, recurse=True):
        return super()._apply(_keep_dtype(fn), recurse)

    def forward(self, x, residual=None):
        return layer_norm(x, self.weight, self.bias, residual, self.eps)


def _autocast(x):
    """x in the type that autocast gives a linear layer."""
    return x.to(torch.get_autocast_dtype(x.device.type)) if torch.is_autocast_enabled(x.device.type) else x


class Experts(torch.nn.Module):
    """A two-layer branch in several versions, of which each token takes the k
    that a linear layer gives it the largest logits for, weighted by their softmax:
        sum_j w_j down_e(gelu(up_e(x))),  e = e_j(x).
    x [T, C] -> [T, C].  channels and hidden: multiples of 8."""

    def __init__(self, channels, hidden, experts, k=2, device=None, dtype=torch.bfloat16):
        super().__init__()
        if not 1 <= k <= experts:
            raise ValueError(f"{k} of {experts} experts a token")
        if experts > 512:
            raise ValueError(f"{experts} experts: up to 512 are supported")
        if channels % 8 or hidden % 8:
            raise ValueError(f"{channels} channels, {hidden} hidden: expert_linear takes multiples of 8")
        self.experts, self.k = experts, k
        f = dict(device=device, dtype=dtype)
        self.router = torch.nn.Linear(channels, experts, bias=False, **f)

        def uniform(*shape, fan):
            return torch.nn.Parameter(torch.empty(*shape, **f).uniform_(-fan ** -0.5, fan ** -0.5))

        self.up = uniform(experts, hidden, channels, fan=channels)
        self.up_bias = uniform(experts, hidden, fan=channels)
        self.down = uniform(experts, channels, hidden, fan=hidden)
        self.down_bias = uniform(experts, channels, fan=hidden)

    def forward(self, x):
        x = _autocast(x)
        top, chosen = self.router(x).float().topk(self.k, dim=1)
        order = expert_order(chosen.to(torch.int32), self.experts)
        up, up_bias, down, down_bias = (p.to(x.dtype) for p in (self.up, self.up_bias, self.down, self.down_bias))
        rows = expert_linear(expert_gather(x, order), up, order.cu_experts, up_bias)
        rows = expert_linear(torch.nn.functional.gelu(rows), down, order.cu_experts, down_bias)
        return expert_combine(rows, torch.softmax(top, 1), order)


class ScanBlock(torch.nn.Module):
    """Pre-norm gated recurrence and experts over packed tokens, for planes too
    large for attention:
        h = x + proj(scan(values, gates of in(norm(x))))
        out = h + experts(norm(h))
    x [T, C], C a multiple of 8.  Half of the channels run from each sequence's
    first token to its last and half the other way; with causal all from the first,
    and :meth:`step` takes one more token of each sequence."""

    def __init__(self, channels, hidden=None, experts=8, k=2, causal=False, device=None, dtype=torch.bfloat16):
        super().__init__()
        if not causal and channels % 2:
            raise ValueError(f"{channels} channels do not divide into two directions")
        f = dict(device=device, dtype=dtype)
        self.causal = causal
        self.norm1, self.norm2 = LayerNorm(channels, device=device), LayerNorm(channels, device=device)
        self.values = torch.nn.Linear(channels, 2 * channels, **f)   # and gates
        self.proj = torch.nn.Linear(channels, channels, bias=False, **f)
        self.experts = Experts(channels, hidden or 2 * channels, experts, k, **f)

    def _branch(self, x, mixed):
        n, h = self.norm2(self.proj(mixed).to(x.dtype), x)   # another type under autocast
        return h + self.experts(n).to(x.dtype)

    def forward(self, x, cu_seqlens):
        C = x.shape[1]
        if self.causal:
            v, g = self.values(self.norm1(x)).split(C, 1)
            mixed, _ = gated_scan(v, g, cu_seqlens)
        else:
            v, v_back, g, g_back = self.values(self.norm1(x)).split(C // 2, 1)
            mixed = torch.cat([gated_scan(v, g, cu_seqlens)[0], gated_scan(v_back, g_back, cu_seqlens, reverse=True)[0]], 1)
        return self._branch(x, mixed)

    def step(self, x, state):
        """One more token of each of n sequences: (out, state).  x [n, C]; state [n,
        C] float32, zeros at first, is updated in place.  No gradient."""
        if not self.causal:
            raise ValueError("only a causal block takes one token after another")
        with torch.no_grad():
            v, g = self.values(self.norm1(x)).split(x.shape[1], 1)
            mixed, state = gated_scan_step(v, g, state, out=state)
            return self._branch(x, mixed), state
