"""Attention on the GPU where packs have many sequences, and the precision of
its float32 products.

The bounds of test_tokens_gpu.py are worst cases; here float32 results are held
against what the same formula in plain float32 operations gives, as root mean
squares over the tensor: a product of float32 values from three bfloat16 parts
leaves out terms below 2^-24 of it, half a rounding, so that the kernels' errors
are those of float32 sums in another order.  Twice and a half of the plain
form's is allowed; without one of the six products, or all three small ones, they
are 7 to 30 times off."""

import math

import pytest
import torch

from memory_bound_cnn_amd import token_binding as tb, tokens

from .test_tokens_gpu import DEV, attn_check, gen, normal, pack

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ many sequences
def mixed_lengths(n):
    """n lengths of 0 to 400, those around a tile of 128 among them."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 401, (n,), generator=g).tolist()
    lens[:9] = [127, 128, 129, 0, 1, 256, 257, 400, 0]
    return lens


def gapped(lens, before, after, Hq, Hk, D, dtype, seed):
    """A pack with tokens of no sequence before the first and after the last one."""
    q, k, v, _ = pack([before + sum(lens) + after], Hq, Hk, D, dtype, seed=seed)
    return q, k, v, (before + torch.tensor([0] + lens, device=DEV).cumsum(0)).to(torch.int32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n", [61, 62, 63, 64, 130])
def test_attention_many_sequences_of_several_tiles(n, causal, dtype):
    """Tiles are handed out from the lengths in the wave's lanes up to 62
    sequences, and by searching cu_seqlens with more."""
    q, k, v, cu = gapped(mixed_lengths(n), 300, 517, 4, 2, 32, dtype, n)
    got = attn_check(q, k, v, cu, causal, what=f"{n} sequences")
    for t in got.values():
        assert not t[:300].any() and not t[int(cu[-1]):].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_empty_sequences_change_nothing(D, causal, dtype):
    """The same pack with empty sequences at its end, so many that the other
    way of handing out tiles is taken: the same bits."""
    q, k, v, cu = gapped(mixed_lengths(50), 140, 131, 6, 3, D, dtype, 7)
    dout = normal(gen(8), *q.shape, dtype=q.dtype)
    runs = []
    for empty in (0, 12, 13, 200):
        c = torch.cat([cu, cu[-1:].expand(empty)]).contiguous()
        d = tb._attn_desc(q, k, v, c, causal, None)
        assert tb._load().wtconv_attention_forward_workspace(tb.ctypes.addressof(d)) == 0    # not split
        out, lse = tb.wtconv_attention_forward(q, k, v, c, causal, want_lse=True)
        runs.append((out, lse) + tb.wtconv_attention_backward(q, k, v, out, lse, dout, c, causal))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ float32 products
def formula(q, k, v, dout, cu, causal, scale):
    """(out, lse, dq, dk, dv) in the type of q, one sequence and head at a time."""
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    out, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((Hq, T), math.inf, dtype=q.dtype, device=q.device)
    for lo, hi in zip(cu[:-1].tolist(), cu[1:].tolist()):
        for h in range(Hq):
            Q, K, V, G = q[lo:hi, h], k[lo:hi, h // group], v[lo:hi, h // group], dout[lo:hi, h]
            S = Q @ K.T * scale
            if causal:
                S = S.masked_fill(torch.ones(hi - lo, hi - lo, device=q.device, dtype=torch.bool).triu(1), -math.inf)
            top = S.amax(-1, keepdim=True)
            E = torch.exp(S - top)
            total = E.sum(-1, keepdim=True)
            P, lse[h, lo:hi] = E / total, (top + torch.log(total))[:, 0]
            O = P @ V
            dS = P * (G @ V.T - (G * O).sum(-1, keepdim=True)) * scale
            out[lo:hi, h], dq[lo:hi, h] = O, dS @ K
            dk[lo:hi, h // group] += dS.T @ Q
            dv[lo:hi, h // group] += P.T @ G
    return out, lse, dq, dk, dv


NAMES = ("out", "lse", "dq", "dk", "dv")


def as_precise_as_float32(got, plain, exact):
    """Each result's root mean square error within 2.5 times the plain form's."""
    for name, a, b, r in zip(NAMES, got, plain, exact):
        ours, theirs = ((t.double() - r).square().mean().sqrt().item() for t in (a, b))
        assert ours <= 2.5 * theirs, f"{name}: {ours:.3e}, plain float32 {theirs:.3e}"


def kernels(q, k, v, dout, cu, causal, scale):
    out, lse = tb.wtconv_attention_forward(q, k, v, cu, causal, scale, want_lse=True)
    return (out, lse) + tb.wtconv_attention_backward(q, k, v, out, lse, dout, cu, causal, scale)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,Hq,Hk,D,scale", [
    ([49, 196, 33], 2, 1, 64, None), ([300, 515], 2, 2, 32, None), ([257, 100], 2, 1, 128, None), ([190], 4, 2, 96, None),
    ([130, 70], 2, 1, 40, 0.5), ([1500], 1, 1, 64, None)])
def test_attention_float32_is_float32(lens, Hq, Hk, D, scale, causal):
    q, k, v, cu = pack(lens, Hq, Hk, D, "fp32", seed=D + len(lens))
    q, k, v = (t.contiguous() for t in (q, k, v))
    dout, s = normal(gen(9), *q.shape), D ** -0.5 if scale is None else scale
    plain = formula(q, k, v, dout, cu, causal, s)
    exact = formula(*(t.double() for t in (q, k, v, dout)), cu, causal, s)
    as_precise_as_float32(kernels(q, k, v, dout, cu, causal, s), plain, exact)


def test_attention_float32_one_key():
    """One key and q = 0: the logit and lse are 0 and P is 1, with nothing
    rounded, so that out is v's three parts put together again and dv dout's:
    the same bits."""
    _, k, v, cu = pack([1] * 300, 2, 2, 64, "fp32", seed=3)
    k, v = k.contiguous(), v.contiguous()
    dout = normal(gen(4), *k.shape)
    out, lse, _, _, dv = kernels(torch.zeros_like(k), k, v, dout, cu, False, 0.125)
    assert not lse.any() and torch.equal(out, v) and torch.equal(dv, dout)


@pytest.mark.parametrize("D", [8, 64, 128])
def test_attention_float32_low_parts_decide(D):
    """Logits a (b - b') with b' = b (1 + e), |e| <= 2^-12: the high parts
    cancel.  They come out to eight float32 roundings of a b."""
    n, g = 150, gen(D)
    a = 1 + torch.rand(n, 1, generator=g, device=DEV)
    b = 1 + torch.rand(n, 1, generator=g, device=DEV)
    c = b * (1 + 2.0 ** -12 * (2 * torch.rand(n, 1, generator=g, device=DEV) - 1))
    q, k = torch.zeros(n, 1, D, device=DEV), torch.zeros(n, 1, D, device=DEV)
    q[:, 0, 0:1], q[:, 0, D - 1:] = a, a
    k[:, 0, 0:1], k[:, 0, D - 1:] = b, -c
    scale, cu = 2.0 ** 13, torch.tensor([0, n], dtype=torch.int32, device=DEV)
    v = normal(g, n, 1, D)
    _, lse, *_ = kernels(q, k, v, normal(g, n, 1, D), cu, False, scale)
    want = torch.logsumexp(q[:, 0].double() @ k[:, 0].double().T * scale, -1)
    assert ((lse[0].double() - want).abs() <= 8 * 2.0 ** -24 * 4 * scale + 2.0 ** -20 * want.abs()).all()
