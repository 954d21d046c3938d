"""Cases of the operators that a block for large planes and wide branches is made of: what they are measured on, their
plain forms and their values in 64 bits.

A case names one operator with its sizes: layer_norm; gated_scan, a gated linear recurrence inside each sequence of a
pack, and scan_step, its form for one token a sequence; expert_rows, the rows of tokens sorted by expert and brought
back; expert_linear, the products of each expert's rows.  The sizes follow the image planes the package is built for: a
pixel of a channels-last plane is a token, and images of different sizes are packed one after another.
"""
import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# --------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm of one 7 x 7 image in a network's last stage, at inference: latency
        dict(name="layer_one_image", op="layer_norm", dtype="bf16", rows=49, C=768, residual=False, bias=True,
             train=False),
        # a training step of a 32 x 32 stage, 128 images, the norm behind a residual
        dict(name="layer_train", op="layer_norm", dtype="bf16", rows=131072, C=384, residual=True, bias=True,
             train=True),
        # a float32 training step with rows and channels that divide by nothing
        dict(name="layer_train_odd", op="layer_norm", dtype="fp32", rows=50021, C=389, residual=False, bias=False,
             train=True),
        # one more token for each of 128 streams of frames: latency
        dict(name="scan_step", op="scan_step", dtype="bf16", B=128, C=768),
        # a training step over a pack of images between 7 x 7 and 64 x 64 pixels, last pixel to first
        dict(name="scan_images", op="gated_scan", dtype="bf16", seqs=64, lo=49, hi=4096, pack=1, C=384, state=False,
             reverse=True, train=True),
        # a training step over two planes of 256 x 256 pixels: few sequences, long ones
        dict(name="scan_planes", op="gated_scan", dtype="bf16", seqs=2, lo=65536, hi=65536, pack=2, C=512, state=False,
             reverse=False, train=True),
        # clips that go on from a state, float32, odd lengths and channels, inference
        dict(name="scan_odd", op="gated_scan", dtype="fp32", seqs=5, lo=1, hi=9001, pack=3, C=387, state=True,
             reverse=False, train=False),
        # the rows of 128 images of 14 x 14, two of 8 experts a token, a training step
        dict(name="rows_train", op="expert_rows", dtype="bf16", T=25088, k=2, E=8, C=384, absent=0.0, train=True),
        # a padded batch with an odd number of channels, three of 37 experts a token, float32
        dict(name="rows_odd", op="expert_rows", dtype="fp32", T=20011, k=3, E=37, C=771, absent=0.1, train=True),
        # the products of one 7 x 7 image, two of 8 experts a token, at inference: the weights' way from memory
        dict(name="products_one_image", op="expert_linear", dtype="bf16", rows=98, pad=0, E=8, K=512, N=2048, bias=True,
             pack=4, train=False),
        # a training step of a wide branch, 128 images of 14 x 14, two of 8 experts a token
        dict(name="products_train", op="expert_linear", dtype="bf16", rows=50176, pad=0, E=8, K=1024, N=4096, bias=True,
             pack=5, train=True),
        # float32, sizes that fill no tile, rows that no expert has
        dict(name="products_odd", op="expert_linear", dtype="fp32", rows=6007, pad=93, E=5, K=392, N=1544, bias=False,
             pack=6, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "gated_scan", "gated_scan", "scan_step", "expert_rows", "expert_linear",
                     "expert_linear"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "layer_norm":
        C = _log(rng, 16, 8192)
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(200000, (50 if dtype == "bf16" else 25) * 1000000 // C)),
                    C=C, residual=rng.random() < 0.5, bias=rng.random() < 0.7, train=rng.random() < 0.6)
    if op == "scan_step":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 4096), C=_log(rng, 1, 4096))
    if op == "gated_scan":
        C, hi = _log(rng, 16, 2048), _log(rng, 1, 65536)
        seqs = min(_log(rng, 1, 512), max(1, (60 if dtype == "bf16" else 30) * 1000000 // (hi * C)))
        if hi * C > 30000000:
            C = 30000000 // hi
        return dict(op=op, dtype=dtype, seqs=seqs, lo=rng.choice([0, hi // 4, hi]), hi=hi, pack=rng.randrange(1 << 20),
                    C=C, state=rng.random() < 0.4, reverse=rng.random() < 0.4, train=rng.random() < 0.6)
    if op == "expert_rows":
        k, C, E = rng.choice([1, 2, 2, 3, 4, 6, 8]), _log(rng, 16, 2048), _log(rng, 1, 256)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(65536, 40000000 // (k * C))), k=min(k, E), E=E, C=C,
                    absent=rng.choice([0.0, 0.0, 0.2]), train=rng.random() < 0.6)
    K, N, E = 8 * _log(rng, 4, 512), 8 * _log(rng, 4, 512), _log(rng, 1, 64)
    while E * K * N > 200000000:
        E //= 2
    most = (200000000000 if dtype == "bf16" else 10000000000) // (K * N)
    return dict(op=op, dtype=dtype, rows=_log(rng, 1, max(1, min(65536, most))), pad=rng.choice([0, 0, 17]), E=E, K=K,
                N=N, bias=rng.random() < 0.5, pack=rng.randrange(1 << 20), train=rng.random() < 0.6)


def _lengths(c):
    rng = random.Random(c["pack"])
    got = [rng.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return got if sum(got) else [1] + got[1:]


def _counts(c):
    """Rows of each expert: some have several times the others', and may have none."""
    rng = random.Random(c["pack"])
    share = [rng.random() ** 2 + 0.02 for _ in range(c["E"])]
    at = [int(c["rows"] * sum(share[:e]) / sum(share)) for e in range(c["E"])] + [c["rows"]]
    return [b - a for a, b in zip(at, at[1:])]


def work(c):
    op, e = c["op"], SIZE[c["dtype"]]
    train = bool(c.get("train"))
    if op == "layer_norm":
        n, r = c["rows"] * c["C"], int(c["residual"])
        return {"bytes": (2 + 2 * r) * n * e + (3 + r) * n * e * train, "flops": (6 + 10 * train) * n}
    if op == "scan_step":
        n = c["B"] * c["C"]
        return {"bytes": n * (3 * e + 8), "flops": 6 * n}
    if op == "gated_scan":
        n, s = sum(_lengths(c)) * c["C"], 4 * c["seqs"] * c["C"] * (1 + int(c["state"]))
        return {"bytes": (3 + 5 * train) * n * e + s * (1 + train), "flops": (6 + 12 * train) * n}
    if op == "expert_rows":
        n, k = c["T"] * c["C"] * e, c["k"]
        # the rows out, the weighted sum back; their gradients: the sum of the rows', and each row's with its weight's
        return {"bytes": n * (2 * (1 + k) + ((1 + k) + (1 + 2 * k)) * train) + 16 * c["T"] * k,
                "flops": c["T"] * c["C"] * k * (2 + 4 * train)}
    R, E, K, N = c["rows"], c["E"], c["K"], c["N"]
    live = sum(n > 0 for n in _counts(c))
    return {"bytes": e * (R * (K + N) + live * K * N + train * (R * (2 * K + N) + (live + E) * K * N)),
            "flops": 2 * R * K * N * (1 + 2 * train)}


# -------------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = c["op"], TYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def gates(n, C):     # what a channel keeps of its state: from half of it to nearly all, and by the token
        return (torch.rand(C, generator=g, device="cuda") * 6 + torch.randn(n, C, generator=g, device="cuda")).to(dtype)

    s = {"case": c}
    leaves = []
    if op == "layer_norm":
        shape = (c["rows"], c["C"])
        s.update(x=normal(*shape) + normal(c["rows"], 1), weight=1.0 + normal(c["C"], scale=0.2, dtype=torch.float32),
                 bias=normal(c["C"], scale=0.2, dtype=torch.float32) if c["bias"] else None,
                 residual=normal(*shape, scale=3.0) if c["residual"] else None)
        if c["train"]:
            s.update(dy=normal(*shape), dh=normal(*shape) if c["residual"] else None)
            leaves = ["x", "weight", "bias", "residual"]
    elif op == "scan_step":
        s.update(x=normal(c["B"], c["C"]), gate=gates(c["B"], c["C"]), state=normal(c["B"], c["C"], dtype=torch.float32))
    elif op == "gated_scan":
        lens, C = _lengths(c), c["C"]
        T = sum(lens)
        s.update(x=normal(T, C), gate=gates(T, C), lens=lens,
                 cu_seqlens=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
                 state=normal(len(lens), C, dtype=torch.float32) if c["state"] else None)
        if c["train"]:
            s.update(dy=normal(T, C), dlast=normal(len(lens), C, dtype=torch.float32))
            leaves = ["x", "gate", "state"]
    elif op == "expert_rows":
        T, k, E, C = c["T"], c["k"], c["E"], c["C"]
        logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        top, experts = logits.topk(k, dim=1)
        absent = torch.rand(T, 1, generator=g, device="cuda") < c["absent"]      # tokens that only pad a batch
        s.update(experts=torch.where(absent, -1, experts).to(torch.int32), weights=torch.softmax(top, 1).contiguous(),
                 x=normal(T, C), rows=normal(T * k, C))     # rows: what the experts gave
        if c["train"]:
            s.update(dxs=normal(T * k, C), dy=normal(T, C))
            leaves = ["x", "rows", "weights"]
    else:
        R, E, K, N = c["rows"] + c["pad"], c["E"], c["K"], c["N"]
        counts = _counts(c)
        s.update(x=normal(R, K), weight=normal(E, N, K, scale=K ** -0.5), bias=normal(E, N) if c["bias"] else None,
                 counts=counts, cu_experts=torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32))
        if c["train"]:
            s["dy"] = normal(R, N)
            leaves = ["x", "weight", "bias"]
    s["leaves"] = [name for name in leaves if s[name] is not None]
    for name in s["leaves"]:
        s[name].requires_grad_()
    return s


# ----------------------------------------------------------------------------------------------------- the calls
def run(s):
    op = s["case"]["op"]
    if own:
        return {"layer_norm": _own_layer_norm, "gated_scan": _own_gated_scan, "scan_step": _own_scan_step,
                "expert_rows": _own_expert_rows, "expert_linear": _own_expert_linear}[op](s)
    with torch.no_grad():
        return {"layer_norm": _plain_layer_norm, "gated_scan": _plain_gated_scan, "scan_step": _plain_scan_step,
                "expert_rows": _plain_expert_rows, "expert_linear": _plain_expert_linear}[op](s)


def _gradients(s, outputs, grads):
    got = torch.autograd.grad(outputs, [s[name] for name in s["leaves"]], grads)
    return {"d" + name: d for name, d in zip(s["leaves"], got)}


def _own_layer_norm(s):
    from memory_bound_cnn_amd import tokens
    c = s["case"]
    if not c["residual"]:
        y = tokens.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": y, **(_gradients(s, y, s["dy"]) if c["train"] else {})}
    y, h = tokens.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
    return {"y": y, "h": h, **(_gradients(s, (y, h), (s["dy"], s["dh"])) if c["train"] else {})}


def _own_gated_scan(s):
    from memory_bound_cnn_amd import tokens
    c = s["case"]
    y, last = tokens.gated_scan(s["x"], s["gate"], s["cu_seqlens"], state=s["state"], reverse=c["reverse"])
    return {"y": y, "last": last, **(_gradients(s, (y, last), (s["dy"], s["dlast"])) if c["train"] else {})}


def _own_scan_step(s):
    from memory_bound_cnn_amd import tokens
    y, state = tokens.gated_scan_step(s["x"], s["gate"], s["state"])
    return {"y": y, "state": state}


def _own_expert_rows(s):
    from memory_bound_cnn_amd import tokens
    order = tokens.expert_order(s["experts"], s["case"]["E"])
    xs = tokens.expert_gather(s["x"], order)
    y = tokens.expert_combine(s["rows"], s["weights"], order)
    out = {"slot": order.slot, "pair": order.pair, "cu_experts": order.cu_experts, "xs": xs, "y": y}
    return {**out, **(_gradients(s, (xs, y), (s["dxs"], s["dy"])) if s["case"]["train"] else {})}


def _own_expert_linear(s):
    from memory_bound_cnn_amd import tokens
    y = tokens.expert_linear(s["x"], s["weight"], s["cu_experts"], bias=s["bias"])
    return {"y": y, **(_gradients(s, y, s["dy"]) if s["case"]["train"] else {})}


# --------------------------------------------------------------------------------------------------- plain forms
def _plain_layer_norm(s):
    """h = x + r as it is stored; y = (h - mean h) / sqrt(mean (h - mean h)^2 + eps) w + b."""
    c, x, w = s["case"], s["x"], s["weight"]
    h = (x.float() + s["residual"].float()).to(x.dtype) if c["residual"] else x
    xh = h.float()
    xh = xh - xh.mean(1, keepdim=True)
    rstd = torch.rsqrt((xh * xh).mean(1, keepdim=True) + EPS)
    xh = xh * rstd
    y = xh * w
    if c["bias"]:
        y = y + s["bias"]
    out = {"y": y.to(x.dtype)}
    if c["residual"]:
        out["h"] = h
    if c["train"]:
        dy = s["dy"].float()
        u = dy * w
        dx = rstd * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dh"].float()
            out["dresidual"] = dx.to(x.dtype)
        out["dx"] = dx.to(x.dtype)
        out["dweight"] = (dy * xh).sum(0)
        if c["bias"]:
            out["dbias"] = dy.sum(0)
    return out


def _gate(f):
    """What is kept of the state, and what is taken of the input: 1 - sigmoid(f) = sigmoid(-f) loses no bits."""
    f = f.float()
    return 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(f))


def _scan(A, B):
    """B[:, t] = A[:, t] B[:, t - 1] + B[:, t], the steps taken 1, 2, 4, ... at once."""
    d, L = 1, A.shape[1]
    while d < L:
        B = torch.cat((B[:, :d], A[:, d:] * B[:, :-d] + B[:, d:]), 1)
        A = torch.cat((A[:, :d], A[:, d:] * A[:, :-d]), 1)
        d *= 2
    return B


def _places(s):
    """The token in each place of sequences padded to the longest one, in the order they are walked; the place of each
    token; which places are there."""
    cu, T, L = s["cu_seqlens"].long(), s["x"].shape[0], max(s["lens"])
    at, lens = torch.arange(L, device="cuda"), (cu[1:] - cu[:-1])[:, None]
    there = at < lens
    token = cu[:-1, None] + (lens - 1 - at if s["case"]["reverse"] else at)
    place = torch.zeros(T, dtype=torch.long, device="cuda")
    place[token[there]] = torch.arange(there.numel(), device="cuda").view_as(there)[there]
    return token.clamp(0, T - 1), place, there[:, :, None], lens


def _plain_gated_scan(s):
    """h_t = a_t h_(t-1) + (1 - a_t) x_t, a = sigmoid(gate); places past a sequence's end keep its state."""
    c, C = s["case"], s["case"]["C"]
    token, place, there, lens = _places(s)
    x = s["x"].float()[token]
    a, take = _gate(s["gate"][token])
    first = s["state"] if c["state"] else torch.zeros(len(s["lens"]), C, device="cuda")
    one = torch.ones((), device="cuda")
    A, B = torch.where(there, a, one), torch.where(there, take * x, 0 * one)
    B[:, 0] += A[:, 0] * first
    h = _scan(A, B)
    out = {"y": h.reshape(-1, C)[place].to(s["x"].dtype), "last": h[:, -1].clone()}
    if not c["train"]:
        return out
    dy = s["dy"].float()[token] * there
    dy[:, -1] += s["dlast"]
    after = torch.cat((A[:, 1:], torch.zeros_like(A[:, :1])), 1)
    dh = _scan(after.flip(1), dy.flip(1)).flip(1)
    before = torch.cat((first[:, None], h[:, :-1]), 1)
    out["dx"] = (dh * take).reshape(-1, C)[place].to(s["x"].dtype)
    out["dgate"] = (dh * (before - x) * a * take).reshape(-1, C)[place].to(s["x"].dtype)
    if c["state"]:
        out["dstate"] = A[:, 0] * dh[:, 0]
    return out


def _plain_scan_step(s):
    a, take = _gate(s["gate"])
    h = a * s["state"] + take * s["x"].float()
    return {"y": h.to(s["x"].dtype), "state": h}


def _plain_expert_rows(s):
    """The pairs of a token and an expert in the order of the experts, those of one in the order of the tokens; a
    pair's rank among its expert's is the number of those before it."""
    c, T, k, E, C = s["case"], s["case"]["T"], s["case"]["k"], s["case"]["E"], s["case"]["C"]
    e = s["experts"].reshape(-1).long()
    there = e >= 0
    mine = torch.zeros(T * k, E + 1, dtype=torch.int32, device="cuda")
    mine[torch.arange(T * k, device="cuda"), torch.where(there, e, E)] = 1
    before = mine.cumsum(0, dtype=torch.int32) - mine
    counts = mine.sum(0)[:E]
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0)))
    rank = before[torch.arange(T * k, device="cuda"), torch.where(there, e, E)]
    slot = torch.where(there, cu[e.clamp_min(0)] + rank, -1)
    pair = torch.full((T * k + 1,), -1, dtype=torch.long, device="cuda")
    pair[torch.where(there, slot, T * k)] = torch.arange(T * k, device="cuda")
    pair = pair[:-1]
    pair_of = torch.where(pair >= 0, pair, 0)
    has, on = (pair >= 0)[:, None], there.view(T, k)[:, :, None]
    slots = slot.view(T, k).clamp_min(0)
    dtype = s["x"].dtype
    xs = s["x"][pair_of // k] * has
    w = s["weights"]
    y = (s["rows"].float()[slots] * w[:, :, None] * on).sum(1)
    out = {"slot": slot.view(T, k).int(), "pair": pair.int(), "cu_experts": cu.int(), "xs": xs, "y": y.to(dtype)}
    if c["train"]:
        dy = s["dy"].float()
        out["dx"] = (s["dxs"].float()[slots] * on).sum(1).to(dtype)
        out["drows"] = (dy[pair_of // k] * w.reshape(-1)[pair_of][:, None] * has).to(dtype)
        out["dweights"] = (s["rows"].float()[slots] * dy[:, None, :] * on).sum(2)
    return out


def _plain_expert_linear(s):
    """One expert's rows after another's."""
    c, x, w, dtype = s["case"], s["x"], s["weight"], s["x"].dtype
    y = torch.zeros(x.shape[0], c["N"], dtype=dtype, device="cuda")
    out = {"y": y}
    if c["train"]:
        out["dx"], out["dweight"] = torch.zeros_like(x), torch.zeros_like(w)
        if c["bias"]:
            out["dbias"] = torch.zeros_like(s["bias"])
    at = 0
    for e, n in enumerate(s["counts"]):
        rows, at = slice(at, at + n), at + n
        if n == 0:
            continue
        xe, we = x[rows].float(), w[e].float()
        ye = torch.matmul(xe, we.T)
        y[rows] = (ye + s["bias"][e].float() if c["bias"] else ye).to(dtype)
        if c["train"]:
            dy = s["dy"][rows].float()
            out["dx"][rows] = torch.matmul(dy, we).to(dtype)
            out["dweight"][e] = torch.matmul(dy.T, xe).to(dtype)
            if c["bias"]:
                out["dbias"][e] = dy.sum(0).to(dtype)
    return out


# ----------------------------------------------------------------------------------------------- values in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        return {"layer_norm": _exact_layer_norm, "gated_scan": _exact_gated_scan, "scan_step": _exact_scan_step,
                "expert_rows": _exact_expert_rows, "expert_linear": _exact_expert_linear}[c["op"]](c, s)


def _exact_layer_norm(c, s):
    """From the definition: the sum as the residual stream holds it, everything after that in 64 bits."""
    h = s["x"].double()
    if c["residual"]:
        h = (h + s["residual"].double()).float().to(TYPES[c["dtype"]]).double()
    C, w = c["C"], s["weight"].double()
    off = h - (h.sum(1) / C)[:, None]
    t = torch.sqrt(torch.linalg.vector_norm(off, dim=1) ** 2 / C + EPS)
    y = off / t[:, None] * w
    out = {"y": y + s["bias"].double() if c["bias"] else y}
    if c["residual"]:
        out["h"] = h
    if c["train"]:
        dy = s["dy"].double()
        # d(off_c / t) = d off_c / t - off_c sum_k(off_k d off_k) / (C t^3), and off takes the mean's part away
        along = torch.einsum("rc,rc->r", dy * w, off) / (C * t ** 3)
        doff = dy * w / t[:, None] - off * along[:, None]
        dx = doff - (doff.sum(1) / C)[:, None]
        if c["residual"]:
            dx = dx + s["dh"].double()
            out["dresidual"] = dx
        out["dx"] = dx
        out["dweight"] = torch.einsum("rc,rc,r->c", dy, off, 1 / t)
        if c["bias"]:
            out["dbias"] = torch.einsum("rc->c", dy)
    return out


def _exact_gated_scan(c, s):
    """One token of every sequence after another, sequences with the most tokens first."""
    lens, C = s["lens"], c["C"]
    T, L = sum(lens), max(lens)
    start = s["cu_seqlens"].long()
    by_length = sorted(range(len(lens)), key=lambda i: -lens[i])
    ids = torch.tensor(by_length, device="cuda")
    still = [0] * (L + 1)                 # sequences that have a token number t
    for n in lens:
        still[n] += 1
    for t in range(L - 1, -1, -1):
        still[t] += still[t + 1]
    still = still[1:]
    length = torch.tensor(lens, device="cuda")

    def tokens_at(t):
        of = ids[:still[t]]
        return start[of + 1] - 1 - t if c["reverse"] else start[of] + t

    x, f = s["x"].double(), s["gate"].double()
    h = s["state"].double()[ids] if c["state"] else torch.zeros(len(lens), C, dtype=torch.float64, device="cuda")
    y, before = torch.empty_like(x), torch.empty_like(x)
    for t in range(L):
        at, n = tokens_at(t), still[t]
        a = torch.sigmoid(f[at])
        before[at] = h[:n]
        h[:n] = a * h[:n] + torch.sigmoid(-f[at]) * x[at]
        y[at] = h[:n]
    last = torch.empty_like(h)
    last[ids] = h
    out = {"y": y, "last": last}
    if not c["train"]:
        return out
    dh, dy = s["dlast"].double()[ids], s["dy"].double()
    dx, df = torch.empty_like(x), torch.empty_like(x)
    for t in range(L - 1, -1, -1):
        at, n = tokens_at(t), still[t]
        a, take = torch.sigmoid(f[at]), torch.sigmoid(-f[at])
        dh[:n] += dy[at]
        dx[at] = dh[:n] * take
        df[at] = dh[:n] * (before[at] - x[at]) * (a * take)
        dh[:n] *= a
    out.update(dx=dx, dgate=df)
    if c["state"]:
        out["dstate"] = torch.empty_like(dh)
        out["dstate"][ids] = dh
    return out


def _exact_scan_step(c, s):
    a = torch.sigmoid(s["gate"].double())
    h = s["x"].double() + a * (s["state"].double() - s["x"].double())
    return {"y": h, "state": h}


def _exact_expert_rows(c, s):
    """Lists of each expert's pairs, then the sums one choice of all tokens after another."""
    T, k, E, C = c["T"], c["k"], c["E"], c["C"]
    lists = [[] for _ in range(E)]
    for p, e in enumerate(s["experts"].reshape(-1).tolist()):
        if e >= 0:
            lists[e].append(p)
    pair, cu = [], [0]
    for mine in lists:
        pair += mine
        cu.append(len(pair))
    live = len(pair)
    slot = [-1] * (T * k)
    for r, p in enumerate(pair):
        slot[p] = r
    slot = torch.tensor(slot, device="cuda").view(T, k)
    at = torch.tensor(pair, dtype=torch.long, device="cuda")
    x, rows, w = s["x"].double(), s["rows"].double(), s["weights"].double()
    xs, y = torch.zeros(T * k, C, dtype=torch.float64, device="cuda"), torch.zeros_like(x)
    xs[:live] = x[at // k]
    y.index_add_(0, at // k, rows[:live] * w.view(-1)[at][:, None])
    out = {"slot": slot.int(), "pair": torch.tensor(pair + [-1] * (T * k - live), device="cuda").int(),
           "cu_experts": torch.tensor(cu, device="cuda").int(), "xs": xs, "y": y}
    if c["train"]:
        dy, dx = s["dy"].double(), torch.zeros_like(x)
        dx.index_add_(0, at // k, s["dxs"].double()[:live])
        drows, dw = torch.zeros_like(rows), torch.zeros_like(w)
        drows[:live] = dy[at // k] * w.view(-1)[at][:, None]
        dw.view(-1)[at] = torch.einsum("rc,rc->r", dy[at // k], rows[:live])
        out.update(dx=dx, drows=drows, dweights=dw)
    return out


def _exact_expert_linear(c, s):
    """Products of blocks of rows, each with its expert's weights."""
    R, E, K, N = s["x"].shape[0], c["E"], c["K"], c["N"]
    f64 = dict(dtype=torch.float64, device="cuda")
    cu = s["cu_experts"].tolist()
    out = {"y": torch.zeros(R, N, **f64)}
    if c["train"]:
        out.update(dx=torch.zeros(R, K, **f64), dweight=torch.zeros(E, N, K, **f64))
        if c["bias"]:
            out["dbias"] = torch.zeros(E, N, **f64)
    for e in range(E):
        w = s["weight"][e].double()
        for r in range(cu[e], cu[e + 1], 4096):
            rows = slice(r, min(r + 4096, cu[e + 1]))
            x = s["x"][rows].double()
            out["y"][rows] = x @ w.t() + (s["bias"][e].double() if c["bias"] else 0)
            if c["train"]:
                dy = s["dy"][rows].double()
                out["dx"][rows] = dy @ w
                out["dweight"][e] += dy.t() @ x
                if c["bias"]:
                    out["dbias"][e] += dy.sum(0)
    return out
