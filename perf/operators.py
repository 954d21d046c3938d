"""The token operators' cases: what they are measured on, their plain forms and their values in 64 bits.

A case names one operator (rms_norm, rotary, attention, dropout) with its sizes.  The sizes follow the image planes the
package is built for: a pixel of a channels-last plane is a token, so B planes of H x W pixels with C channels are
B H W tokens of C channels, and images of different sizes are packed one after another.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
F8_MAX = 448.0            # the largest e4m3 value
F8_LEAST = 2.0 ** -100    # the smallest row scale of the 8-bit output
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# --------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm of one 7 x 7 image in a network's last stage, at inference: latency
        dict(name="rms_one_image", op="rms_norm", dtype="bf16", rows=49, C=768, residual=True, fp8=False, train=False),
        # a training step of a 32 x 32 stage, 64 images
        dict(name="rms_train", op="rms_norm", dtype="bf16", rows=65536, C=192, residual=True, fp8=False, train=True),
        # a float32 training step with rows and channels that divide by nothing, no residual
        dict(name="rms_train_odd", op="rms_norm", dtype="fp32", rows=100003, C=387, residual=False, fp8=False,
             train=True),
        # the norm ahead of an 8-bit product, 128 images of 14 x 14
        dict(name="rms_fp8", op="rms_norm", dtype="bf16", rows=25088, C=384, residual=True, fp8=True, train=False),
        # queries and keys of 14 x 14 images where the projection left them, two axes, at inference
        dict(name="rotary_images", op="rotary", dtype="bf16", frames=128, h=14, w=14, T=25088, heads=12, extra=6, D=64,
             axes=2, interleaved=False, train=False),
        # clips of 32 x 32 frames with a token more than the frames fill, three axes, both directions
        dict(name="rotary_video", op="rotary", dtype="fp32", frames=64, h=32, w=32, T=65537, heads=10, extra=2, D=128,
             axes=3, interleaved=True, train=True),
        # attention inside one 7 x 7 image, at inference: latency
        dict(name="attn_one_image", op="attention", dtype="bf16", seqs=1, lo=49, hi=49, pack=1, Hq=12, Hk=12, D=64,
             causal=False, train=False),
        # a training step over a pack of images between 7 x 7 and 32 x 32 pixels
        dict(name="attn_images", op="attention", dtype="bf16", seqs=48, lo=49, hi=1024, pack=2, Hq=6, Hk=6, D=64,
             causal=False, train=True),
        # a training step over long clips, each token seeing those before it, grouped heads
        dict(name="attn_video", op="attention", dtype="bf16", seqs=3, lo=3500, hi=8192, pack=4, Hq=16, Hk=4, D=128,
             causal=True, train=True),
        # a float32 training step of a 14 x 14 stage
        dict(name="attn_fp32", op="attention", dtype="fp32", seqs=32, lo=196, hi=196, pack=5, Hq=6, Hk=3, D=64,
             causal=False, train=True),
        # dropout on a branch before its residual, 64 images of 128 x 128 x 96, a training step
        dict(name="dropout_planes", op="dropout", dtype="bf16", n=64 * 128 * 128 * 96, p=0.1, residual=True,
             train=True),
        # one image of 7 x 7 with an odd number of channels, no residual: latency
        dict(name="dropout_odd", op="dropout", dtype="fp32", n=49 * 767, p=0.25, residual=False, train=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms_norm", "rotary", "attention", "attention", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "rms_norm":
        C = _log(rng, 16, 8192)
        fp8 = rng.random() < 0.25
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(200000, 40_000_000 // C)), C=C,
                    residual=rng.random() < 0.6, fp8=fp8, train=not fp8 and rng.random() < 0.6)
    if op == "rotary":
        axes = rng.choice([1, 2, 3])
        frames, h, w = _log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 1, 64)
        heads, D = rng.choice([1, 3, 6, 12, 24]), rng.choice([32, 48, 64, 80, 96, 128])
        T = max(1, min(frames * h * w, 60_000_000 // (heads * D)))
        return dict(op=op, dtype=dtype, frames=frames, h=h, w=w, T=T, heads=heads, extra=rng.choice([0, 1, 6]), D=D,
                    axes=axes, interleaved=rng.random() < 0.5, train=rng.random() < 0.5)
    if op == "attention":
        D, Hk, group = rng.choice([32, 64, 64, 80, 96, 128, 128]), rng.choice([1, 2, 3, 4, 6]), rng.choice([1, 1, 2, 4])
        hi = _log(rng, 1, 8192 if dtype == "bf16" else 2048)
        seqs = min(_log(rng, 1, 64), max(1, 2_000_000_000 // (hi * hi * Hk * group)))
        return dict(op=op, dtype=dtype, seqs=seqs, lo=rng.choice([0, hi // 4, hi]), hi=hi, pack=rng.randrange(1 << 20),
                    Hq=Hk * group, Hk=Hk, D=D, causal=rng.random() < 0.5, train=rng.random() < 0.6)
    return dict(op=op, dtype=dtype, n=_log(rng, 1, 60_000_000), p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                residual=rng.random() < 0.6, train=rng.random() < 0.6)


def _lengths(c):
    rng = random.Random(c["pack"])
    got = [rng.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return got if sum(got) else [1] + got[1:]


def _sections(c):
    """Pairs per axis: the head's D / 2 pairs split as evenly as they go, the first axes getting the odd ones."""
    pairs, axes = c["D"] // 2, c["axes"]
    return [pairs // axes + (a < pairs % axes) for a in range(axes)]


def work(c):
    e = SIZE[c["dtype"]]
    if c["op"] == "rms_norm":
        n, r = c["rows"] * c["C"], int(c["residual"])
        read, wrote = (1 + r) * n * e, (r * e + (1 if c["fp8"] else e)) * n
        both = n * e * (3 + r) if c["train"] else 0          # dy, dh and h in, dx out
        return {"bytes": read + wrote + both + 4 * c["C"], "flops": (4 + 8 * bool(c["train"])) * n}
    if c["op"] == "rotary":
        n = c["T"] * c["heads"] * c["D"]
        passes = 2 if c["train"] else 1
        return {"bytes": passes * (2 * n * e + 4 * c["T"] * c["axes"]), "flops": passes * 3 * n}
    if c["op"] == "attention":
        lens = _lengths(c)
        pairs = sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lens)
        T, q, kv = sum(lens), c["Hq"] * c["D"] * e, 2 * c["Hk"] * c["D"] * e
        # forward: q, k, v in, out out; backward: q, k, v, out, dout in, dq, dk, dv out
        return {"bytes": T * (2 * q + kv + (4 * q + 2 * kv if c["train"] else 0)),
                "flops": pairs * c["Hq"] * c["D"] * (14 if c["train"] else 4)}
    n = c["n"]
    return {"bytes": n * e * (2 + int(c["residual"]) + (2 if c["train"] else 0)), "flops": 2 * n}


# -------------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": c}
    if c["op"] == "rms_norm":
        shape = (c["rows"], c["C"])
        s.update(x=normal(*shape), weight=1.0 + normal(c["C"], scale=0.2, dtype=torch.float32),
                 residual=normal(*shape, scale=3.0) if c["residual"] else None)
        if c["train"]:
            s.update(dy=normal(*shape), dh=normal(*shape) if c["residual"] else None)
    elif c["op"] == "rotary":
        T, n = c["T"], c["T"]
        at = torch.arange(n, device="cuda") % (c["frames"] * c["h"] * c["w"])
        at = at + seed % 5      # a clip starts anywhere
        t, y, x = at // (c["h"] * c["w"]), at // c["w"] % c["h"], at % c["w"]
        s["positions"] = torch.stack([at] if c["axes"] == 1 else [t, y, x][3 - c["axes"]:], 1).to(torch.int32)
        s["sections"] = tuple(_sections(c))
        s["inv_freq"] = torch.cat([10000.0 ** (-torch.arange(m, device="cuda", dtype=torch.float64) / m)
                                   for m in s["sections"]]).float()
        s["x"] = normal(T, c["heads"] + c["extra"], c["D"])[:, :c["heads"]]   # q and k; v stays beside them
        if c["train"]:
            s["dy"] = normal(T, c["heads"], c["D"])
    elif c["op"] == "attention":
        lens = _lengths(c)
        T, Hq, Hk, D = sum(lens), c["Hq"], c["Hk"], c["D"]
        qkv = normal(T, Hq + 2 * Hk, D)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:], max_len=max(lens),
                 cu_seqlens=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32))
        if c["train"]:
            s["dout"] = normal(T, Hq, D)
    else:
        s.update(x=normal(c["n"]), residual=normal(c["n"]) if c["residual"] else None,
                 rng=torch.randint(-(1 << 62), 1 << 62, (2,), generator=g, device="cuda"))
        if c["train"]:
            s["dy"] = normal(c["n"])
    if c["train"]:
        s.update({k: s[k].requires_grad_() for k in ("x", "q", "k", "v", "weight") if k in s})
        if s.get("residual") is not None:
            s["residual"].requires_grad_()
    return s


# ----------------------------------------------------------------------------------------------------- the calls
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rms_norm": _own_rms_norm, "rotary": _own_rotary, "attention": _own_attention,
                "dropout": _own_dropout}[op](s)
    with torch.no_grad():
        return {"rms_norm": _plain_rms_norm, "rotary": _plain_rotary, "attention": _plain_attention,
                "dropout": _plain_dropout}[op](s)


def _own_rms_norm(s):
    from memory_bound_cnn_amd import tokens
    c = s["case"]
    if c["fp8"]:
        q, scale, h = tokens.rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS)
        y = (q.float() * scale[:, None]).to(s["x"].dtype)
        return {"y": y, "scale": scale, "h": h if c["residual"] else None}
    if not c["residual"]:
        y = tokens.rms_norm(s["x"], s["weight"], eps=EPS)
        if not c["train"]:
            return {"y": y}
        dx, dw = torch.autograd.grad(y, (s["x"], s["weight"]), s["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    y, h = tokens.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
    if not c["train"]:
        return {"y": y, "h": h}
    dx, dr, dw = torch.autograd.grad((y, h), (s["x"], s["residual"], s["weight"]), (s["dy"], s["dh"]))
    return {"y": y, "h": h, "dx": dx, "dr": dr, "dw": dw}


def _own_rotary(s):
    from memory_bound_cnn_amd import tokens
    y = tokens.rotary(s["x"], s["positions"], s["inv_freq"], s["sections"], interleaved=s["case"]["interleaved"])
    if not s["case"]["train"]:
        return {"y": y}
    return {"y": y, "dx": torch.autograd.grad(y, s["x"], s["dy"])[0]}


def _own_attention(s):
    from memory_bound_cnn_amd import tokens
    out = tokens.attention(s["q"], s["k"], s["v"], s["cu_seqlens"], causal=s["case"]["causal"])
    if not s["case"]["train"]:
        return {"out": out}
    dq, dk, dv = torch.autograd.grad(out, (s["q"], s["k"], s["v"]), s["dout"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _own_dropout(s):
    from memory_bound_cnn_amd import tokens
    c = s["case"]
    y = tokens.dropout(s["x"], c["p"], s["rng"], residual=s["residual"])
    if not c["train"]:
        return {"y": y}
    return {"y": y, "dx": torch.autograd.grad(y, s["x"], s["dy"])[0]}


# --------------------------------------------------------------------------------------------------- plain forms
def _plain_rms_norm(s):
    """h = x + r as it is stored; y = h / sqrt(mean h^2 + eps) w; 8 bits: y over its row's scale, as e4m3."""
    c, x, w = s["case"], s["x"], s["weight"]
    h = (x.float() + s["residual"].float()).to(x.dtype) if c["residual"] else x
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1, keepdim=True) + EPS)
    xh = hf * rstd
    y = xh * w
    out = {"y": y.to(x.dtype)}
    if c["residual"]:
        out["h"] = h
    if c["fp8"]:
        scale = (y.abs().amax(1, keepdim=True) / F8_MAX).clamp_min(F8_LEAST)
        held = (y / scale).to(torch.float8_e4m3fn).float() * scale
        return {"y": held.to(x.dtype), "scale": scale[:, 0], "h": out.get("h")}
    if not c["train"]:
        return out
    dy = s["dy"].float()
    u = dy * w
    dx = rstd * (u - xh * (u * xh).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + s["dh"].float()
    out["dx"] = dx.to(x.dtype)
    if c["residual"]:
        out["dr"] = out["dx"]
    out["dw"] = (dy * xh).sum(0)
    return out


def _turn(x, cos, sin, interleaved):
    """The pairs (u, v) of each head turned to (u cos - v sin, u sin + v cos); channels past the pairs stay."""
    P = cos.shape[1]
    cos, sin, xf = cos[:, None], sin[:, None], x.float()
    u, v = (xf[..., 0:2 * P:2], xf[..., 1:2 * P:2]) if interleaved else (xf[..., :P], xf[..., P:2 * P])
    a, b = u * cos - v * sin, u * sin + v * cos
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, xf[..., 2 * P:]), -1).to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    axis = torch.cat([torch.full((m,), a, device="cuda") for a, m in enumerate(s["sections"])])
    angle = s["positions"].float()[:, axis] * s["inv_freq"]
    cos, sin = angle.cos(), angle.sin()
    out = {"y": _turn(s["x"], cos, sin, c["interleaved"])}
    if c["train"]:
        out["dx"] = _turn(s["dy"], cos, -sin, c["interleaved"])
    return out


def _plain_attention(s):
    """Each sequence padded to the longest one; softmax over the keys that are there, and that the query may see."""
    c, cu, L = s["case"], s["cu_seqlens"].long(), s["max_len"]
    Hq, Hk, D, scale = c["Hq"], c["Hk"], c["D"], 1.0 / math.sqrt(c["D"])
    T, group = s["q"].shape[0], c["Hq"] // c["Hk"]
    lens = cu[1:] - cu[:-1]
    at = torch.arange(L, device="cuda")
    there = at < lens[:, None]                                            # [n, L]
    token = (cu[:-1, None] + at).clamp_max(T - 1)                         # the token in each padded place
    seq = torch.searchsorted(cu[1:], torch.arange(T, device="cuda"), right=True)
    place = seq * L + torch.arange(T, device="cuda") - cu[seq]            # the padded place of each token
    head = torch.arange(Hq, device="cuda") // group

    def pad(x):
        return (x.float()[token] * there[:, :, None, None]).transpose(1, 2).contiguous()      # [n, H, L, D]

    def back(x, dtype):
        return x.transpose(1, 2).reshape(-1, x.shape[1], D)[place].to(dtype)

    q, k, v = pad(s["q"]), pad(s["k"])[:, head], pad(s["v"])[:, head]
    S = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    seen = there[:, None, None, :]
    if c["causal"]:
        seen = seen & (at[None, :] <= at[:, None])
    S.masked_fill_(~seen, float("-inf"))
    S.sub_(S.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()              # empty sequences: rows of -inf
    P = S.div_(S.sum(-1, keepdim=True).clamp_min(1e-30))
    O = torch.matmul(P, v)
    out = {"out": back(O, s["q"].dtype)}
    if not c["train"]:
        return out
    dO = pad(s["dout"])
    dV = torch.matmul(P.transpose(-1, -2), dO)
    dS = torch.matmul(dO, v.transpose(-1, -2)).sub_((dO * O).sum(-1, keepdim=True)).mul_(P).mul_(scale)
    dQ, dK = torch.matmul(dS, k), torch.matmul(dS.transpose(-1, -2), q)
    n = dK.shape[0]
    out["dq"] = back(dQ, s["q"].dtype)
    out["dk"] = back(dK.view(n, Hk, group, L, D).sum(2), s["k"].dtype)
    out["dv"] = back(dV.view(n, Hk, group, L, D).sum(2), s["v"].dtype)
    return out


LOW = 0xFFFFFFFF


def _philox(counter, key):
    """Ten rounds of Philox 4x32 (Salmon, Moraes, Dror, Shaw, 2011) on int64 tensors that hold 32-bit words."""
    def rounds(n, c0, c1, c2, c3, k0, k1):
        if n == 0:
            return c0, c1, c2, c3
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57          # 64-bit products: the wrapped sign bit is masked off
        return rounds(n - 1, (q >> 32 & LOW) ^ c1 ^ k0, q & LOW, (p >> 32 & LOW) ^ c3 ^ k1, p & LOW,
                      (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW)
    return rounds(10, *counter, *key)


def _plain_dropout(s):
    """Element i takes half-word i % 8 of the words at counter i // 8; it is kept where that is at least 65536 p."""
    c, x = s["case"], s["x"]
    n, least = c["n"], int(round(c["p"] * 65536))
    seed, offset = s["rng"][0], s["rng"][1]
    block = torch.arange((n + 7) // 8, device="cuda")
    words = _philox((block & LOW, block >> 32, (offset & LOW).expand_as(block), (offset >> 32 & LOW).expand_as(block)),
                    (seed & LOW, seed >> 32 & LOW))
    halves = torch.stack([h for word in words for h in (word & 0xFFFF, word >> 16)], 1).flatten()[:n]
    keep, scale = halves >= least, 65536.0 / (65536 - least)
    zero = torch.zeros((), device="cuda")
    y = torch.where(keep, x.float() * scale, zero)
    if c["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(x.dtype)}
    if c["train"]:
        out["dx"] = torch.where(keep, s["dy"].float() * scale, zero).to(x.dtype)
    return out


# ----------------------------------------------------------------------------------------------- values in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        return {"rms_norm": _exact_rms_norm, "rotary": _exact_rotary, "attention": _exact_attention,
                "dropout": _exact_dropout}[c["op"]](c, s)


def _e4m3(v):
    """The nearest e4m3 values, ties to even: 3 bits after the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-F8_MAX, F8_MAX)


def _exact_rms_norm(c, s):
    """From the definition: the sum as the residual stream holds it, everything after that in 64 bits."""
    h = s["x"].double()
    if c["residual"]:
        h = (h + s["residual"].double()).float().to(TYPES[c["dtype"]]).double()
    w = s["weight"].double()
    norm = torch.linalg.vector_norm(h, dim=1)
    t = torch.sqrt(norm ** 2 / c["C"] + EPS)
    y = h / t[:, None] * w
    if c["fp8"]:
        scale = torch.clamp(y.abs().max(1).values / F8_MAX, min=F8_LEAST)
        return {"y": _e4m3(y / scale[:, None]) * scale[:, None], "scale": scale, "h": h if c["residual"] else None}
    out = {"y": y}
    if c["residual"]:
        out["h"] = h
    if c["train"]:
        dy = s["dy"].double()
        # d(h_c / t) = dh_c / t - h_c sum_k(h_k dh_k) / (C t^3)
        along = torch.einsum("rc,rc->r", dy * w, h) / (c["C"] * t ** 3)
        dx = dy * w / t[:, None] - h * along[:, None]
        if c["residual"]:
            dx = dx + s["dh"].double()
            out["dr"] = dx
        out["dx"] = dx
        out["dw"] = torch.einsum("rc,rc,r->c", dy, h, 1 / t)
    return out


def _exact_rotary(c, s):
    """Each pair as a complex number times e^(i angle)."""
    def turn(x, sign):
        x, first, y = x.double(), 0, x.double().clone()
        half = sum(s["sections"])
        for a, m in enumerate(s["sections"]):
            angle = s["positions"][:, a, None].double() * s["inv_freq"][None, first:first + m].double()
            e = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
            at = torch.arange(first, first + m, device="cuda")
            u, v = (2 * at, 2 * at + 1) if c["interleaved"] else (at, at + half)
            z = torch.complex(x[..., u], x[..., v]) * e
            y[..., u], y[..., v] = z.real, z.imag
            first += m
        return y
    out = {"y": turn(s["x"], 1)}
    if c["train"]:
        out["dx"] = turn(s["dy"], -1)
    return out


def _exact_attention(c, s):
    """One sequence and one head of queries at a time."""
    lens, group, scale, first = _lengths(c), c["Hq"] // c["Hk"], 1 / math.sqrt(c["D"]), 0
    names = ("out", "dq", "dk", "dv") if c["train"] else ("out",)
    like = {"out": s["q"], "dq": s["q"], "dk": s["k"], "dv": s["v"]}
    out = {m: torch.zeros(like[m].shape, dtype=torch.float64, device="cuda") for m in names}
    for n in lens:
        rows, first = slice(first, first + n), first + n
        if n == 0:
            continue
        for h in range(c["Hq"]):
            q, k, v = s["q"][rows, h].double(), s["k"][rows, h // group].double(), s["v"][rows, h // group].double()
            logits = q @ k.T * scale
            if c["causal"]:
                logits = logits.masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), -math.inf)
            p = torch.softmax(logits, -1)
            out["out"][rows, h] = p @ v
            if c["train"]:
                do = s["dout"][rows, h].double()
                out["dv"][rows, h // group] += p.T @ do
                dp = do @ v.T
                ds = p * (dp - (dp * p).sum(-1, keepdim=True))
                out["dq"][rows, h] = ds @ k * scale
                out["dk"][rows, h // group] += ds.T @ q * scale
    return out


def _exact_dropout(c, s):
    """The generator on NumPy words, the sums in 64 bits."""
    n, least = c["n"], int(round(c["p"] * 65536))
    seed, offset = (int(v) & 0xFFFFFFFFFFFFFFFF for v in s["rng"].tolist())
    keep, m32 = np.empty(-(-n // 8) * 8, dtype=bool), np.uint64(LOW)
    for b in range(0, -(-n // 8), 1 << 15):
        at = np.arange(b, min(b + (1 << 15), -(-n // 8)), dtype=np.uint64)
        w = [at & m32, at >> np.uint64(32), np.full_like(at, offset & LOW), np.full_like(at, offset >> 32)]
        for r in range(10):
            k = [np.uint64((seed + r * 0x9E3779B9) & LOW), np.uint64(((seed >> 32) + r * 0xBB67AE85) & LOW)]
            left, right = w[0] * np.uint64(0xD2511F53), w[2] * np.uint64(0xCD9E8D57)
            w = [right >> np.uint64(32) ^ w[1] ^ k[0], right & m32, left >> np.uint64(32) ^ w[3] ^ k[1], left & m32]
        bits = np.stack(w, 1).astype("<u4").view("<u2").reshape(-1)
        keep[8 * b:8 * b + bits.size] = bits >= least
    keep = torch.from_numpy(keep[:n]).cuda()
    factor = keep.double() * 65536 / (65536 - least)
    y = s["x"].double() * factor
    out = {"y": y + s["residual"].double() if c["residual"] else y}
    if c["train"]:
        out["dx"] = s["dy"].double() * factor
    return out
