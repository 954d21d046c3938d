"""Token operators on the GPU against plain float64 implementations.

Tolerances follow from where bits are dropped.  U is the unit roundoff of the
storage type, 2^-p for p significant bits (24 of float32, 8 of bfloat16): it
bounds a rounding relative to the value.  float32 work on n terms is given
n 2^-23 relative to the sum of the terms' magnitudes."""

import math

import numpy as np
import pytest
import torch

from memory_bound_cnn_amd import token_binding as tb, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
F32 = 2.0 ** -23


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def within(got, ref, bound, what):
    """|got - ref| <= bound at every element (bound: of the same shape)."""
    assert got.shape == ref.shape, what
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / bound).max())} of the bound"


# ------------------------------------------------------------------ rms_norm
def rms_ref(x, w, r, eps):
    h = x.double() if r is None else (x.double() + r.double()).float().to(x.dtype).double()
    s = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, s, h * s * w.double()


RMS_SHAPES = [(1, 1), (1, 768), (3, 7), (5, 8), (49, 96), (130, 33), (257, 192), (7, 387), (300, 64), (64, 1024),
              (33, 1025), (9, 2048), (11, 2056), (5, 4100), (3, 8192), (2, 16384), (4, 5000), (1000, 16), (31, 640),
              (5600, 192), (5601, 91), (2803, 381), (1400, 768)]   # the last four: other shapes of lanes and vectors


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,C", RMS_SHAPES)
def test_rms_norm_forward_backward(rows, C, residual, dtype):
    g, dt, eps = gen(rows * 31 + C), TYPES[dtype], 1e-5
    x, w = normal(g, rows, C, dtype=dt), 1 + normal(g, C, scale=0.3)
    r = normal(g, rows, C, dtype=dt, scale=2.0) if residual else None
    leaves = [t.requires_grad_() for t in (x, w, r) if t is not None]
    dy, dh = normal(g, rows, C, dtype=dt), normal(g, rows, C, dtype=dt)
    if residual:
        y, h = tokens.rms_norm(x, w, r, eps=eps)
        grads = torch.autograd.grad((y, h), leaves, (dy, dh))
    else:
        y = tokens.rms_norm(x, w, eps=eps)
        grads = torch.autograd.grad(y, leaves, dy)
    with torch.no_grad():
        hr, s, yr = rms_ref(x, w, r, eps)
        n, u = C + 16, U[dtype]
        stat = n * F32   # of s, from a sum of C squares
        if residual:
            assert torch.equal(h.double(), hr)
        within(y.detach(), yr, (u + stat) * yr.abs() + 1e-30, "y")
        xh, uu = hr * s, dy.double() * w.double()
        along = (uu * xh).mean(1, keepdim=True)
        size = (uu * xh).abs().mean(1, keepdim=True)
        dx = s * (uu - xh * along) + (dh.double() if residual else 0)
        mag = s * (uu.abs() + xh.abs() * size) + (dh.double().abs() if residual else 0)
        within(grads[0], dx, u * dx.abs() + 4 * stat * mag + 1e-30, "dx")
        if residual:
            assert torch.equal(grads[0], grads[2])
        dw = (dy.double() * xh).sum(0)
        within(grads[1], dw, (rows + n) * F32 * (dy.double() * xh).abs().sum(0) + 1e-30, "dw")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1, 1), (49, 768), (7, 387), (130, 33), (5, 4100), (3, 16384), (64, 24),
                                    (5600, 192), (2803, 381), (1400, 768)])
def test_rms_norm_fp8(rows, C, dtype):
    """The scale to float32, the values to half a step of e4m3 (three bits after
    the leading one; 2^-9 below 2^-6) plus the rounding of y and its scale."""
    g, dt = gen(C), TYPES[dtype]
    x, r = normal(g, rows, C, dtype=dt), normal(g, rows, C, dtype=dt)
    w = 1 + normal(g, C, scale=0.3)
    if rows > 2:
        x[1], r[1] = 0, 0   # an all-zero row
        x[2], r[2] = x[2] * 1e-30, 0
    y8, scale, h = tokens.rms_norm_fp8(x, w, r)
    hr, s, yr = rms_ref(x, w, r, 1e-6)
    assert torch.equal(h.double(), hr) and y8.dtype == torch.float8_e4m3fn
    n = (C + 16) * F32
    want = (yr.abs().amax(1) / 448).clamp_min(2.0 ** -100)
    within(scale, want, 2 * n * want, "scale")
    q = yr / want[:, None]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    within(y8.double() * scale.double()[:, None], yr, (0.5 * step + 4 * n * q.abs()) * want[:, None] * (1 + 4 * n),
           "y8")
    if rows > 2:
        assert not y8[1].float().any()


def test_rms_norm_strided_rows_and_shapes():
    g = gen(5)
    big = normal(g, 40, 3, 100, dtype=torch.bfloat16)
    w = 1 + normal(g, 64, scale=0.1)
    x, r = big[:, 1, 5:69], big[:, 2, 30:94]          # rows 300 elements apart, 2-byte aligned
    y, h = tokens.rms_norm(x, w, r)
    yc, hc = tokens.rms_norm(x.contiguous(), w, r.contiguous())
    assert torch.equal(y, yc) and torch.equal(h, hc)
    x4 = normal(g, 2, 3, 5, 64)
    y4 = tokens.rms_norm(x4, w)
    assert y4.shape == x4.shape and torch.equal(y4.view(-1, 64), tokens.rms_norm(x4.view(-1, 64), w))
    xl = x4.permute(0, 1, 3, 2)[..., :5]              # last axis not contiguous
    assert torch.equal(tokens.rms_norm(xl, w[:5].contiguous()), tokens.rms_norm(xl.contiguous(), w[:5].contiguous()))
    # an upstream gradient without a row stride, and a broadcast residual
    xg, rg = normal(g, 6, 64).requires_grad_(), normal(g, 1, 64).requires_grad_()
    y, h = tokens.rms_norm(xg, w, rg.expand(6, 64))
    (y.sum() + h.sum()).backward()
    assert rg.grad.shape == (1, 64) and torch.allclose(rg.grad, xg.grad.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)


def test_rms_norm_parts_of_the_gradient():
    g = gen(6)
    w = (1 + normal(g, 48, scale=0.1)).requires_grad_()
    x, r = normal(g, 10, 48).requires_grad_(), normal(g, 10, 48).requires_grad_()
    y, h = tokens.rms_norm(x, w, r)
    dh = normal(g, 10, 48)
    a = torch.autograd.grad(h, (x, r), dh, retain_graph=True)
    assert torch.equal(a[0], dh) and torch.equal(a[1], dh)
    dy = normal(g, 10, 48)
    b = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    c = torch.autograd.grad((y, h), (x, w), (dy, torch.zeros_like(dh)))
    assert torch.equal(b[0], c[0]) and torch.equal(b[1], c[1])


def test_rms_norm_empty_and_repeatable():
    w = torch.ones(32, device=DEV)
    assert tokens.rms_norm(torch.zeros(0, 32, device=DEV), w).shape == (0, 32)
    dx, dw = tb.wtconv_rms_norm_backward(*[torch.zeros(0, 32, device=DEV)] * 3, w, torch.zeros(0, device=DEV))
    assert dx.shape == (0, 32) and not dw.any()
    g = gen(8)
    x, dy, w = normal(g, 5000, 192), normal(g, 5000, 192), 1 + normal(g, 192)
    _, _, rstd, _ = tb.wtconv_rms_norm_forward(x, w, want_rstd=True)
    a, b = (tb.wtconv_rms_norm_backward(dy, None, x, w, rstd) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ rotary
def rotary_ref(x, pos, f, sections, interleaved, sign=1):
    x, P = x.double(), sum(sections)
    axis = torch.cat([torch.full((n,), a, device=DEV) for a, n in enumerate(sections)]).long()
    angle = (pos.float()[:, axis] * f).double()      # the angle is the float32 product
    c, s = angle.cos()[:, None], sign * angle.sin()[:, None]
    y = x.clone()
    u, v = (x[..., 0:2 * P:2], x[..., 1:2 * P:2]) if interleaved else (x[..., :P], x[..., P:2 * P])
    a, b = u * c - v * s, u * s + v * c
    if interleaved:
        y[..., 0:2 * P:2], y[..., 1:2 * P:2] = a, b
    else:
        y[..., :P], y[..., P:2 * P] = a, b
    mag = torch.ones_like(y) * x.abs().amax(-1, keepdim=True)
    return y, mag


ROT = [(1, 1, 2, (1,)), (5, 3, 64, (16, 16)), (7, 12, 64, (32,)), (49, 4, 128, (16, 24, 24)), (33, 2, 80, (20, 20)),
       (10, 5, 48, (3, 8, 5, 4)), (9, 3, 7, (3,)), (6, 2, 30, (5, 0, 2)), (3, 1, 16, (0,)), (1000, 1, 96, (24, 24))]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,sections", ROT)
def test_rotary(T, H, D, sections, interleaved, dtype):
    g = gen(T + D)
    x = normal(g, T, H + 2, D, dtype=TYPES[dtype])[:, 1:H + 1].requires_grad_()
    pos = torch.randint(-50, 4096, (T, len(sections)), generator=g, device=DEV, dtype=torch.int32)
    f = tokens.rotary_frequencies(sections, device=DEV)
    y = tokens.rotary(x, pos, f, sections, interleaved=interleaved)
    dy = normal(g, T, H, D, dtype=TYPES[dtype])
    dx, = torch.autograd.grad(y, x, dy)
    with torch.no_grad():
        for got, src, sign in ((y, x, 1), (dx, dy, -1)):
            ref, mag = rotary_ref(src, pos, f, sections, interleaved, sign)
            within(got.detach(), ref, U[dtype] * ref.abs() + 8 * F32 * mag, "rotary")
        # in place, and inverse of the turn
        z = x.detach().clone()
        assert torch.equal(tb.wtconv_rotary(z, pos, f, sections, interleaved, out=z), y.detach())


def test_rotary_empty():
    f = tokens.rotary_frequencies((4,), device=DEV)
    x = torch.zeros(0, 2, 8, device=DEV)
    assert tokens.rotary(x, torch.zeros(0, 1, dtype=torch.int32, device=DEV), f, (4,)).shape == (0, 2, 8)


# ------------------------------------------------------------------ dropout
def philox_words(block, offset, seed):
    """Words of one counter, in Python integers."""
    c = [block & 0xFFFFFFFF, block >> 32, offset & 0xFFFFFFFF, offset >> 32]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_ref(n, p, seed, offset):
    least = int(round(p * 65536))
    words = [w for b in range(-(-n // 8)) for w in philox_words(b, offset, seed)]
    half = np.array(words, dtype="<u4").view("<u2")[:n]
    return torch.from_numpy(half.astype(np.int64) >= least).to(DEV), 65536 / (65536 - least) if least < 65536 else 0.0


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.uint64).view(torch.int64).to(DEV)


def test_generator_known_answers():
    """Published vectors of the generator (its authors' test files)."""
    assert philox_words(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = (1 << 64) - 1
    assert philox_words(ones, ones, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,p", [(1, 0.5), (7, 0.1), (8, 0.1), (9, 0.9), (4099, 0.25), (100, 0.0), (100, 1.0),
                                 (65, 1e-6)])
def test_dropout(n, p, residual, dtype):
    g, seed, offset = gen(n), 0xFEDCBA9876543210, 0x8000000000000005
    x = normal(g, n, dtype=TYPES[dtype]).requires_grad_()
    r = normal(g, n, dtype=TYPES[dtype]).requires_grad_() if residual else None
    rng = rng_of(seed, offset)
    y = tokens.dropout(x, p, rng, residual=r)
    dy = normal(g, n, dtype=TYPES[dtype])
    grads = torch.autograd.grad(y, [t for t in (x, r) if t is not None], dy)
    keep, f = keep_ref(n, p, seed, offset)
    with torch.no_grad():
        xk = torch.where(keep, x.double() * f, torch.zeros((), dtype=torch.float64, device=DEV))
        ref = xk + (r.double() if residual else 0)
        within(y.detach(), ref, U[dtype] * ref.abs() + 2 * F32 * xk.abs() + 1e-30, "y")
        dk = torch.where(keep, dy.double() * f, torch.zeros((), dtype=torch.float64, device=DEV))
        within(grads[0], dk, (U[dtype] + 2 * F32) * dk.abs() + 1e-30, "dx")
        if residual:
            assert torch.equal(grads[1], dy)


def test_dropout_drops_what_is_not_finite():
    x = torch.full((4096,), float("nan"), device=DEV)
    y = tokens.dropout(x, 0.5, rng_of(3, 4))
    keep, _ = keep_ref(4096, 0.5, 3, 4)
    assert torch.equal(torch.isnan(y), keep) and not y[~keep].any()


def test_dropout_unaligned_views_and_rates():
    g = gen(2)
    x = normal(g, 1 << 20, dtype=torch.bfloat16)
    a = tokens.dropout(x[3:-2], 0.3, rng_of(1, 2))
    b = tokens.dropout(x[3:-2].clone(), 0.3, rng_of(1, 2))
    assert torch.equal(a, b)
    n = a.numel()
    kept = int((tokens.dropout(torch.ones(n, device=DEV), 0.3, rng_of(1, 2)) != 0).sum())
    assert abs(kept - 0.7 * n) < 5 * math.sqrt(n * 0.21)      # five standard deviations
    other = tokens.dropout(torch.ones(n, device=DEV), 0.3, rng_of(1, 3)) != 0
    same = int((other == (tokens.dropout(torch.ones(n, device=DEV), 0.3, rng_of(1, 2)) != 0)).sum())
    assert abs(same - 0.58 * n) < 5 * math.sqrt(n * 0.25)
    assert tokens.dropout(x[:0], 0.3, rng_of(1, 2)).shape == (0,)


# ------------------------------------------------------------------ attention
def attention_ref(q, k, v, cu, causal, scale, dout=None, u=0.0):
    """out, lse (and dq, dk, dv), each with a bound on the error of float32
    work with P and dS rounded relatively by u."""
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=DEV)
    r = {n: z(t) for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    b = {n: z(t) for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    lse = torch.full((Hq, T), math.inf, dtype=torch.float64, device=DEV)
    for s in range(cu.numel() - 1):
        lo, hi = int(cu[s]), int(cu[s + 1])
        if hi <= lo:
            continue
        n = hi - lo
        for h in range(Hq):
            Q, K, V = (t[lo:hi, i].double() for t, i in ((q, h), (k, h // group), (v, h // group)))
            S = Q @ K.T * scale
            if causal:
                S = S.masked_fill(torch.ones(n, n, device=DEV, dtype=torch.bool).triu(1), -math.inf)
            lse[h, lo:hi] = torch.logsumexp(S, -1)
            P = torch.softmax(S, -1)
            # relative error of P: the logit's error, the maximum's rounding, the exponential, and u
            e = u + F32 * ((D + 8) * abs(scale) * (Q.abs() @ K.abs().T) + S.masked_fill(S == -math.inf, 0).abs() * 4
                           + n + 32)
            Pe = P * (e + (P * e).sum(-1, keepdim=True))      # of the quotient by the row's sum
            O = P @ V
            Oe = Pe @ V.abs() + n * F32 * (P @ V.abs()) + u * O.abs() + F32 * O.abs()
            r["out"][lo:hi, h], b["out"][lo:hi, h] = O, Oe
            if dout is None:
                continue
            G = dout[lo:hi, h].double()
            dP = G @ V.T
            dPe = (D + 2) * F32 * (G.abs() @ V.abs().T)
            delta = (G * O).sum(-1, keepdim=True)
            de = (G.abs() * Oe).sum(-1, keepdim=True) + (D + 2) * F32 * (G * O).abs().sum(-1, keepdim=True)
            dS = P * (dP - delta)
            dSe = Pe * (dP - delta).abs() + P * (dPe + de) + (u + 2 * F32) * dS.abs()
            a = abs(scale)
            r["dq"][lo:hi, h] = scale * dS @ K
            b["dq"][lo:hi, h] = a * ((dSe + n * F32 * dS.abs()) @ K.abs())
            r["dk"][lo:hi, h // group] += scale * dS.T @ Q
            b["dk"][lo:hi, h // group] += a * ((dSe + n * group * F32 * dS.abs()).T @ Q.abs())
            r["dv"][lo:hi, h // group] += P.T @ G
            b["dv"][lo:hi, h // group] += (Pe + n * group * F32 * P).T @ G.abs()
    return r, b, lse


def attn_check(q, k, v, cu, causal=False, scale=None, train=True, what=""):
    dtype = "bf16" if q.dtype == torch.bfloat16 else "fp32"
    u = U[dtype]
    q, k, v = (t.detach().requires_grad_(train) for t in (q, k, v))
    out = tokens.attention(q, k, v, cu, causal=causal, scale=scale)
    dout = normal(gen(99), *q.shape, dtype=q.dtype)
    got = {"out": out.detach()}
    if train:
        got.update(zip(("dq", "dk", "dv"), torch.autograd.grad(out, (q, k, v), dout)))
    sc = q.shape[2] ** -0.5 if scale is None else scale
    with torch.no_grad():
        r, b, lse = attention_ref(q, k, v, cu, causal, sc, dout if train else None, 0.0 if dtype == "fp32" else u)
        for n, t in got.items():
            within(t, r[n], 1.02 * (b[n] + u * (r[n].abs() + b[n])) + 1e-30, f"{what} {n}")
        _, ls = tb.wtconv_attention_forward(q.contiguous(), k.contiguous(), v.contiguous(), cu, causal, scale,
                                            want_lse=True)
        fin = torch.isfinite(lse)
        assert torch.equal(torch.isposinf(ls), ~fin)
        # 1.5 times the bound of P's relative error, without u
        qa, ka = q.double().abs().amax(), k.double().abs().amax()
        assert ((ls.double() - lse)[fin].abs() <= F32 * (lse[fin].abs() * 8 + 64 + 8 * q.shape[2] ** 2 * abs(sc) * qa * ka
                                                          + int(cu.max()))).all()
    return got


def pack(lens, Hq, Hk, D, dtype, seed=0, scale=1.0):
    T = sum(lens)
    qkv = normal(gen(seed), T, Hq + 2 * Hk, D, dtype=TYPES[dtype], scale=scale)
    cu = torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], cu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,Hq,Hk,D", [
    ([1], 1, 1, 64), ([2], 2, 1, 32), ([0, 1, 0, 3, 0], 2, 2, 64), ([49], 12, 12, 64), ([196, 196], 3, 3, 64),
    ([31, 32, 33], 2, 1, 128), ([63, 64, 65], 4, 2, 64), ([127, 128, 129], 2, 2, 128), ([257, 5, 300], 6, 2, 64),
    ([100, 77], 2, 1, 8), ([130], 1, 1, 40), ([90, 200], 4, 1, 72), ([150], 2, 2, 96), ([70, 140], 3, 1, 104),
    ([1] * 200, 1, 1, 32), ([515], 2, 1, 128),
])
def test_attention(lens, Hq, Hk, D, causal, dtype):
    q, k, v, cu = pack(lens, Hq, Hk, D, dtype, seed=sum(lens))
    attn_check(q, k, v, cu, causal, what=f"{lens[:4]} {Hq}/{Hk} {D}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu,Hq,Hk,D", [([0, 1500], 1, 1, 64), ([0, 1300], 2, 1, 128), ([3, 3, 1200, 1290], 1, 1, 32),
                                        ([0, 1000, 1003, 1900], 2, 2, 104), ([7, 2610], 2, 1, 64),
                                        ([0, 1, 4000], 1, 1, 128)])
def test_attention_split(cu, Hq, Hk, D, causal, dtype):
    """Few long sequences and heads: a tile's other side is split over
    workgroups, some of which have nothing of a short sequence or of the tokens
    of none."""
    q, k, v, _ = pack([cu[-1] + 20], Hq, Hk, D, dtype, seed=cu[-1])
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if cu[-1] - cu[0] > 2000 and not causal:
        d = tb._attn_desc(q, k, v, cu, causal, None)
        assert tb._load().wtconv_attention_forward_workspace(tb.ctypes.addressof(d)) > 0
    attn_check(q, k, v, cu, causal, what=f"split {cu.tolist()}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attention_scales(scale, dtype):
    q, k, v, cu = pack([70, 131], 2, 1, 64, dtype, seed=1)
    attn_check(q, k, v, cu, True, scale, what=f"scale {scale}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_rising_maxima(dtype):
    """Keys that grow along the sequence raise the running maximum tile after
    tile, far beyond what is left unscaled."""
    q, k, v, cu = pack([400], 2, 2, 64, dtype, seed=2)
    k = (k.float() * torch.linspace(0.01, 6, 400, device=DEV)[:, None, None]).to(k.dtype)
    attn_check(q.float().abs().to(q.dtype), k.float().abs().to(k.dtype), v, cu, False, what="rising")
    attn_check(q.float().abs().to(q.dtype), k.float().abs().flip(0).contiguous().to(k.dtype), v, cu, True, what="falling")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_tokens_of_no_sequence(dtype):
    q, k, v, _ = pack([300], 2, 1, 64, dtype, seed=3)
    for cu in ([17, 17, 150, 283], [0], [300], [5, 6], [130]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        got = attn_check(q, k, v, cu, False, what=str(cu.tolist()))
        for t in got.values():
            assert not t[:int(cu[0])].any() and not t[int(cu[-1]):].any()


def test_attention_many_sequences():
    """More sequences than one probe of the search covers, some empty."""
    rng = np.random.RandomState(0)
    lens = [int(n) for n in rng.randint(0, 12, 5000)]
    q, k, v, cu = pack(lens, 1, 1, 32, "bf16", seed=4)
    out = tokens.attention(q, k, v, cu)
    L, n = 12, len(lens)
    at = cu[:-1, None].long() + torch.arange(L, device=DEV)
    there = torch.arange(L, device=DEV) < (cu[1:] - cu[:-1])[:, None]
    at = at.clamp_max(q.shape[0] - 1)
    Q, K, V = (t[at, 0].double() for t in (q, k, v))
    S = (Q @ K.transpose(1, 2) * 32 ** -0.5).masked_fill(~there[:, None], -math.inf)
    O = torch.softmax(S, -1) @ V
    bound = 3 * U["bf16"] * (torch.softmax(S, -1) @ V.abs()) + 1e-4
    within(out[at, 0][there], O[there], bound[there], "many")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_keeps_sequences_apart(dtype):
    """Infinities and NaN in one sequence, and in tokens of none, change no bit of another."""
    lens, first = [70, 90, 130], 11
    q, k, v, _ = pack([first + sum(lens) + 9], 2, 1, 64, dtype, seed=5)
    cu = torch.tensor([first, first + 70, first + 160, first + 290], dtype=torch.int32, device=DEV)
    dout = normal(gen(6), *q.shape, dtype=q.dtype)

    def all_of(q, k, v, dout):
        out, lse = tb.wtconv_attention_forward(q, k, v, cu, True, want_lse=True)
        return (out,) + tb.wtconv_attention_backward(q, k, v, out, lse, dout, cu, True)

    clean = all_of(*(t.contiguous() for t in (q, k, v, dout)))
    bad = [t.contiguous().clone() for t in (q, k, v, dout)]
    for i, t in enumerate(bad):
        t[:first] = float("nan")
        t[first + 290:] = float("inf")
        t[first + 70 + i] = float("nan") if i % 2 else float("-inf")
    for a, b in zip(clean, all_of(*bad)):
        for lo, hi in ((0, first + 70), (first + 160, first + 299)):
            assert torch.equal(a[lo:hi], b[lo:hi])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attention_split_scales(scale, dtype):
    q, k, v, cu = pack([1600], 1, 1, 64, dtype, seed=21)
    attn_check(q, k, v, cu, False, scale, what=f"split scale {scale}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_split_rising_maxima(dtype):
    """Parts of the keys whose maxima lie far apart: the weights of most vanish."""
    q, k, v, cu = pack([1600], 1, 1, 64, dtype, seed=22)
    k = (k.float().abs() * torch.linspace(0.01, 6, 1600, device=DEV)[:, None, None]).to(k.dtype)
    q = q.float().abs().to(q.dtype)
    attn_check(q, k, v, cu, False, what="split rising")
    attn_check(q, k.flip(0).contiguous(), v, cu, False, what="split falling")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_split_keeps_sequences_apart(dtype):
    """As above for sequences whose keys are split: not even through a
    workspace that held NaN, on another stream, and into outputs with strides."""
    q, k, v, _ = pack([1700], 1, 1, 64, dtype, seed=23)
    cu = torch.tensor([5, 805, 1690], dtype=torch.int32, device=DEV)
    dout = normal(gen(24), *q.shape, dtype=q.dtype)

    def all_of(q, k, v, dout, wide):
        d = tb._attn_desc(q, k, v, cu, False, None)
        need = [f(tb.ctypes.addressof(d)) for f in (tb._load().wtconv_attention_forward_workspace,
                                                    tb._load().wtconv_attention_backward_workspace)]
        assert need[0] > 0
        ws = [torch.full((n // 4 + 1,), float("nan"), device=DEV).view(torch.uint8) for n in need]
        out = torch.full((q.shape[0], 1, 64 + wide), 7.0, device=DEV, dtype=q.dtype)[..., :64]
        _, lse = tb.wtconv_attention_forward(q, k, v, cu, False, want_lse=True, out=out, workspace=ws[0])
        return (out, lse.t()) + tb.wtconv_attention_backward(q, k, v, out, lse, dout, cu, False, workspace=ws[1])

    clean = all_of(*(t.contiguous() for t in (q, k, v, dout)), 0)
    assert not clean[0][:5].any() and not clean[0][1690:].any() and torch.isposinf(clean[1][:5]).all()
    bad = [t.contiguous().clone() for t in (q, k, v, dout)]
    for i, t in enumerate(bad):
        t[:5] = float("nan")
        t[1690:] = float("inf")
        t[900 + 300 * i % 700] = float("nan") if i % 2 else float("-inf")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = all_of(*bad, 8)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(clean, got):
        assert torch.equal(a[5:805], b[5:805]) and torch.equal(a[:5], b[:5]) and torch.equal(a[1690:], b[1690:])


def test_attention_repeatable_and_other_streams():
    q, k, v, cu = pack([300, 41, 777], 4, 2, 64, "bf16", seed=7)
    dout = normal(gen(8), *q.shape, dtype=q.dtype)

    def once():
        out, lse = tb.wtconv_attention_forward(q, k, v, cu, True, want_lse=True)
        return (out, lse) + tb.wtconv_attention_backward(q, k, v, out, lse, dout, cu, True)
    a = once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = once()
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_attention_layouts():
    """[Hq, T, D] storage, views that do not start at 16 bytes, and gradients
    from expanded upstream gradients."""
    q, k, v, cu = pack([100, 60], 4, 2, 64, "bf16", seed=9)
    ref = tokens.attention(q, k, v, cu)
    qt, kt, vt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    assert torch.equal(tokens.attention(qt, kt, vt, cu), ref)
    odd = torch.empty(160, 4, 67, dtype=q.dtype, device=DEV)
    odd[..., 3:] = q
    assert torch.equal(tokens.attention(odd[..., 3:], k, v, cu), ref)
    a = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    tokens.attention(*a, cu).sum().backward()
    b = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    tokens.attention(*b, cu).backward(torch.ones_like(ref))
    for x, y in zip(a, b):
        assert torch.equal(x.grad, y.grad)
    # one k and v head for all, by expansion: the gradient sums the broadcast heads
    k1, v1 = (t[:, :1].detach().clone().requires_grad_() for t in (k, v))
    tokens.attention(q, k1.expand(-1, 4, -1), v1.expand(-1, 4, -1), cu).sum().backward()
    k2, v2 = (t[:, :1].detach().clone().requires_grad_() for t in (k, v))
    tokens.attention(q, k2, v2, cu).sum().backward()
    for x, y in ((k1, k2), (v1, v2)):
        assert torch.allclose(x.grad.float(), y.grad.float(), rtol=4 * 2 ** -8, atol=0.05 * float(y.grad.float().abs().max()))


def test_attention_offsets_beyond_32_bits():
    """Tokens 65536 elements apart: the last ones lie beyond 2^31 elements."""
    T, D = 33000, 64
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free device memory")
    big = torch.empty(T, 65536, dtype=torch.bfloat16, device=DEV)
    g = gen(10)
    small = normal(g, T, 3, D, dtype=torch.bfloat16)
    wide = big[:, :3 * D].view(T, 3, D)
    wide.copy_(small)
    cu = torch.tensor([0, T - 200, T], dtype=torch.int32, device=DEV)
    for f in (lambda t: t[T - 200:], lambda t: t[:300]):
        a = tokens.attention(wide[:, 0:1], wide[:, 1:2], wide[:, 2:3], cu)
        b = tokens.attention(small[:, 0:1], small[:, 1:2], small[:, 2:3], cu)
        assert torch.equal(f(a), f(b))
    x, w = wide.view(T, 3 * D)[:, :D], torch.ones(D, device=DEV)
    assert torch.equal(tokens.rms_norm(x, w), tokens.rms_norm(small[:, 0].contiguous(), w))


def test_attention_gradient_by_differences():
    """Central differences of <out, g> along one direction, from the forward
    pass alone.  Third-order terms at a step of 2^-6 and float32 sums of some
    2^12 terms are within 1e-3 of the gradient's and the direction's norms."""
    q, k, v, cu = pack([37, 80], 4, 2, 32, "fp32", seed=11)
    dout = normal(gen(12), *q.shape)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(tokens.attention(*leaves, cu, causal=True), leaves, dout)
    e = 2.0 ** -6
    for i in range(3):
        d = normal(gen(20 + i), *leaves[i].shape)

        def f(t):
            a = [x.detach() for x in leaves]
            a[i] = a[i] + t * d
            return (tokens.attention(*a, cu, causal=True).double() * dout.double()).sum()
        diff = float((f(e) - f(-e)) / (2 * e))
        want = float((grads[i].double() * d.double()).sum())
        assert abs(diff - want) <= 1e-3 * float(grads[i].norm() * d.norm()) , (i, diff, want)


def test_rms_norm_and_rotary_gradients_by_differences():
    g = gen(13)
    w = 1 + normal(g, 48, scale=0.2)
    x, r, dy, dh, d = (normal(g, 20, 48) for _ in range(5))
    a = [t.clone().requires_grad_() for t in (x, w, r)]
    grads = torch.autograd.grad(tokens.rms_norm(*a), a, (dy, dh))
    e = 2.0 ** -7
    for i, dirn in ((0, d), (1, normal(g, 48))):
        def f(t):
            b = [x, w, r]
            b[i] = b[i] + t * dirn
            y, h = tokens.rms_norm(*b)
            return (y.double() * dy.double()).sum() + (h.double() * dh.double()).sum()
        diff, want = float((f(e) - f(-e)) / (2 * e)), float((grads[i].double() * dirn.double()).sum())
        assert abs(diff - want) <= 1e-3 * float(grads[i].norm() * dirn.norm())


# ------------------------------------------------------------------ together
def test_rotary_attention_is_its_parts():
    qkv = normal(gen(14), 160, 8, 64, dtype=torch.bfloat16)
    pos, cu = tokens.image_positions([(10, 10), (6, 10)], device=DEV)
    sections = (16, 16)
    f = tokens.rotary_frequencies(sections, device=DEV)
    a, b = qkv.clone().requires_grad_(), qkv.clone().requires_grad_()
    out = tokens.rotary_attention(a, 4, 2, pos, f, sections, cu)
    q, k = tokens.rotary(b[:, :4], pos, f, sections), tokens.rotary(b[:, 4:6], pos, f, sections)
    ref = tokens.attention(q, k, b[:, 6:], cu)
    g = normal(gen(15), 160, 4, 64, dtype=torch.bfloat16)
    assert torch.equal(out, ref)
    assert torch.equal(torch.autograd.grad(out, a, g)[0], torch.autograd.grad(ref, b, g)[0])


def test_token_block_trains_and_repeats():
    torch.manual_seed(0)
    m = tokens.TokenBlock(96, 3, kv_heads=1, p=0.1, device=DEV, dtype=torch.float32)
    pos, cu = tokens.image_positions([(7, 7), (4, 9)], device=DEV)
    x = torch.randn(85, 96, device=DEV, requires_grad=True)
    y = m(x, pos, cu)
    (y * y).sum().backward()
    for name, p in m.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().sum() > 0, name
    assert torch.isfinite(x.grad).all() and int(m.rng[1]) == 2
    assert not torch.equal(m(x, pos, cu), y)           # another offset drops other elements
    m.eval()
    a, b = m(x, pos, cu), m(x, pos, cu)
    assert torch.equal(a, b)
    # images do not see each other
    x2 = x.detach().clone()
    x2[49:] += 1
    assert torch.equal(m(x2, pos, cu)[:49], a[:49])


def test_second_derivatives_are_refused():
    x, w = torch.randn(4, 16, device=DEV, requires_grad=True), torch.ones(16, device=DEV, requires_grad=True)
    y = tokens.rms_norm(x, w)
    dy = torch.randn(4, 16, device=DEV, requires_grad=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(y, x, dy, create_graph=True)
    q = torch.randn(5, 2, 32, device=DEV, requires_grad=True)
    cu = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    g = torch.randn(5, 2, 32, device=DEV, requires_grad=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(tokens.attention(q, q, q, cu), q, g, create_graph=True)


def test_second_derivatives_by_the_inputs_are_refused():
    """An output's gradient that needs none itself: the norm's and the
    attention's gradients depend on their inputs all the same, those of the
    rotation and of dropout do not."""
    x, w = torch.randn(4, 16, device=DEV, requires_grad=True), torch.ones(16, device=DEV)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(tokens.rms_norm(x, w).sum(), x, create_graph=True)
    q = torch.randn(5, 3, 32, device=DEV, requires_grad=True)
    cu, pos = torch.tensor([0, 5], dtype=torch.int32, device=DEV), torch.zeros(5, 1, dtype=torch.int32, device=DEV)
    f, rng = tokens.rotary_frequencies((4,), device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(tokens.attention(q, q, q, cu).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(tokens.rotary_attention(q, 1, 1, pos, f, (4,), cu).sum(), q, create_graph=True)
    for y in (tokens.rotary(q, pos, f, (4,)), tokens.dropout(q, 0.5, rng)):
        torch.autograd.grad(y.sum(), q, create_graph=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rotary_attention_without_gradients_is_the_same(dtype):
    """Without gradients nothing is kept for them; the outputs are the same bits."""
    qkv = torch.randn(300, 8, 64, device=DEV, dtype=dtype, requires_grad=True)
    cu = torch.tensor([0, 7, 300], dtype=torch.int32, device=DEV)
    pos = torch.arange(300, device=DEV, dtype=torch.int32)[:, None].contiguous()
    f = tokens.rotary_frequencies((32,), device=DEV)
    y = tokens.rotary_attention(qkv, 4, 2, pos, f, (32,), cu, causal=True)
    with torch.no_grad():
        z = tokens.rotary_attention(qkv, 4, 2, pos, f, (32,), cu, causal=True)
    assert y.requires_grad and not z.requires_grad and torch.equal(y, z)


def test_entry_points_refuse():
    """Device tensors of wrong types, shapes and places, through the public functions."""
    x, w = torch.zeros(4, 16, device=DEV), torch.ones(16, device=DEV)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    pos, f = torch.zeros(4, 1, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV)
    x3 = x.view(4, 1, 16)
    for call, message in (
            (lambda: tokens.rms_norm(x.half(), w), "expected float32 or bfloat16"),
            (lambda: tokens.rms_norm(x, w[:8]), "weight has shape"),
            (lambda: tokens.rms_norm(x, w.bfloat16()), "weight has dtype"),
            (lambda: tokens.rms_norm(x, w.cpu()), "weight must be a CUDA tensor"),
            (lambda: tokens.rms_norm(x, w, x.bfloat16()), "residual has dtype"),
            (lambda: tokens.rms_norm_fp8(x.clone().requires_grad_(), w), "no gradient"),
            (lambda: tokens.rotary(x3, pos, f, (9,)), "pairs do not fit"),
            (lambda: tokens.rotary(x3, pos, f, (4,)), "inv_freq has shape"),
            (lambda: tokens.rotary(x3, pos.long(), f, (8,)), "positions has dtype"),
            (lambda: tokens.rotary(x3, pos, f, ()), "axes are supported"),
            (lambda: tokens.rotary(x, pos, f, (8,)), "expected 3 axes"),
            (lambda: tokens.attention(x3, x3, x3, cu.long()), "cu_seqlens has dtype"),
            (lambda: tokens.attention(x3, x3, x3[:3], cu), "v has shape"),
            (lambda: tokens.attention(x3, x3.expand(4, 2, 16), x3.expand(4, 2, 16), cu), "do not divide"),
            (lambda: tokens.attention(x3, x3, x3.bfloat16(), cu), "v has dtype"),
            (lambda: tokens.dropout(x, 1.5, torch.zeros(2, dtype=torch.int64, device=DEV)), "no probability"),
            (lambda: tokens.dropout(x, 0.5, torch.zeros(2, device=DEV)), "rng has dtype"),
            (lambda: tokens.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64, device=DEV), x[:2]), "residual has shape")):
        with pytest.raises(ValueError, match=message):
            call()
    x60 = torch.zeros(4, 1, 60, device=DEV)
    with pytest.raises(RuntimeError, match="shape outside the supported limits"):
        tokens.attention(x60, x60, x60, cu)


def test_operators_replay_in_a_graph():
    """Captured once, replayed with eager work between: each replay is the eager result."""
    q, k, v, cu = pack([64, 100], 2, 1, 64, "bf16", seed=16)
    w = torch.ones(64, device=DEV)
    rng = rng_of(1, 1)
    x = normal(gen(17), 164, 64, dtype=torch.bfloat16)

    def step():
        y, h = tokens.rms_norm(x, w, x)
        return tokens.attention(q, k, v, cu), y, tokens.dropout(h, 0.2, rng, residual=x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(normal(gen(30 + i), 164, 64, dtype=torch.bfloat16))
        rng[1] += 1
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_hybrid_network_learns(dtype):
    """WTConv stage, packed token blocks and their gradients together: the loss
    of eight images, seen 30 times, falls well below that of a guess."""
    from memory_bound_cnn_amd import hybrid
    losses = hybrid.train(steps=30, dtype=dtype, log=None)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0], losses
