"""Layer norm, gated scan and the experts' rows and products on the GPU against
plain float64 implementations.

Tolerances follow from where bits are dropped.  U is the unit roundoff of the
storage type (2^-24 float32, 2^-8 bfloat16), relative to the value; float32 work
on n terms is given n 2^-23 relative to the sum of the terms' magnitudes."""

import ctypes
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
BOTH = pytest.mark.parametrize("dtype", ["fp32", "bf16"])


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def within(got, ref, bound, what):
    """|got - ref| <= bound at every element (bound: of the same shape)."""
    assert got.shape == ref.shape, what
    got, ref, bound = got.detach().double().cpu(), ref.cpu(), bound.cpu()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / bound).max())} of the bound"


# ------------------------------------------------------------------ layer_norm
SHAPES = [(1, 1), (1, 768), (3, 7), (5, 8), (49, 96), (130, 33), (257, 192), (7, 387), (64, 1024), (33, 1025), (11, 2056),
          (5, 4100), (2, 16384), (1000, 16), (5600, 192), (5601, 91), (2803, 381), (1400, 768)]


@BOTH
@pytest.mark.parametrize("residual,bias", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_layer_norm_forward_backward(rows, C, residual, bias, dtype):
    g, dt, eps = gen(rows * 31 + C), TYPES[dtype], 1e-5
    x, w = normal(g, rows, C, dtype=dt) + 0.5, 1 + normal(g, C, scale=0.3)
    b = normal(g, C) if bias else None
    r = normal(g, rows, C, dtype=dt, scale=2.0) if residual else None
    names = [n for n, t in (("x", x), ("w", w), ("b", b), ("r", r)) if t is not None]
    leaves = [t.requires_grad_() for t in (x, w, b, r) if t is not None]
    dy, dh = normal(g, rows, C, dtype=dt), normal(g, rows, C, dtype=dt)
    out = tokens.layer_norm(x, w, b, r, eps=eps)
    y, h = out if residual else (out, None)
    grads = dict(zip(names, torch.autograd.grad((y, h) if residual else y, leaves, (dy, dh) if residual else dy)))
    with torch.no_grad():
        hr = x.double() if r is None else (x.double() + r.double()).float().to(dt).double()
        m = hr.mean(1, keepdim=True)
        off = hr - m
        s = 1 / torch.sqrt((off * off).mean(1, keepdim=True) + eps)
        wd, u, stat = w.double(), U[dtype], (C + 16) * F32
        yr = off * s * wd + (b.double() if bias else 0)
        size = hr.abs().mean(1, keepdim=True)            # the mean is off by stat of it
        if residual:
            assert torch.equal(h.double(), hr)
        xh = off * s
        dxh = xh.abs() + s * size                        # times stat: how far xh is off
        within(y, yr, u * yr.abs() + 4 * stat * (dxh * wd.abs() + (b.double().abs() if bias else 0)) + 1e-30, "y")
        dyd = dy.double()
        v = dyd * wd
        dx = s * (v - v.mean(1, keepdim=True) - xh * (v * xh).mean(1, keepdim=True)) + (dh.double() if residual else 0)
        mag = s * (v.abs() + v.abs().mean(1, keepdim=True) + dxh * (v * xh).abs().mean(1, keepdim=True)
                   + xh.abs() * (v.abs() * dxh).mean(1, keepdim=True)) + (dh.double().abs() if residual else 0)
        within(grads["x"], dx, u * dx.abs() + 4 * stat * mag + 1e-30, "dx")
        if residual:
            assert torch.equal(grads["x"], grads["r"])
        within(grads["w"], (dyd * xh).sum(0), (rows * F32 + 4 * stat) * (dyd.abs() * dxh).sum(0) + 1e-30, "dw")
        if bias:
            within(grads["b"], dyd.sum(0), (rows + 16) * F32 * dyd.abs().sum(0) + 1e-30, "db")


def test_layer_norm_far_from_zero():
    """A mean of 10^4 deviations: the variance is of differences from the mean.  The mean is off by half a bit of it
    (2^-24 10^4, rounded once from sums of 64 numbers that are exact here)."""
    g = gen(3)
    x = (10000 + torch.randint(-4, 5, (200, 64), generator=g, device=DEV) / 4.0)
    y = tokens.layer_norm(x, torch.ones(64, device=DEV))
    off = x.double() - x.double().mean(1, keepdim=True)
    s = 1 / torch.sqrt((off * off).mean(1, keepdim=True) + 1e-6)
    within(y, off * s, s * 10000 * 2 * F32 + 100 * F32 * (off * s).abs(), "y")


def test_layer_norm_strided_shapes_parts_and_empty():
    g = gen(5)
    w, b = 1 + normal(g, 64, scale=0.1), normal(g, 64)
    big = normal(g, 40, 3, 100, dtype=torch.bfloat16)
    x, r = big[:, 1, 5:69], big[:, 2, 30:94]          # rows 300 elements apart, 2-byte aligned
    for a, c in zip(tokens.layer_norm(x, w, b, r), tokens.layer_norm(x.contiguous(), w, b, r.contiguous())):
        assert torch.equal(a, c)
    x4 = normal(g, 2, 3, 5, 64)
    assert torch.equal(tokens.layer_norm(x4, w, b).view(-1, 64), tokens.layer_norm(x4.view(-1, 64), w, b))
    xl = x4.permute(0, 1, 3, 2)[..., :5]              # last axis not contiguous
    assert torch.equal(tokens.layer_norm(xl, w[:5].contiguous()), tokens.layer_norm(xl.contiguous(), w[:5].contiguous()))
    w, b = w.requires_grad_(), b.requires_grad_()
    x, r = normal(g, 10, 64).requires_grad_(), normal(g, 1, 64).requires_grad_()      # a broadcast residual
    y, h = tokens.layer_norm(x, w, b, r.expand(10, 64))
    dh, dy = normal(g, 10, 64), normal(g, 10, 64)
    a = torch.autograd.grad(h, (x, r), dh, retain_graph=True)                         # y is not used
    assert torch.equal(a[0], dh) and torch.allclose(a[1], dh.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)
    only_y = torch.autograd.grad(y, (x, w, b), dy, retain_graph=True)
    both = torch.autograd.grad((y, h), (x, w, b), (dy, torch.zeros_like(dy)), retain_graph=True)
    for p, q in zip(only_y, both):
        assert torch.equal(p, q)
    y.sum().backward()                                                                # a gradient without strides
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
    e = torch.zeros(0, 64, device=DEV, requires_grad=True)
    y = tokens.layer_norm(e, w, b)
    de, dw, db = torch.autograd.grad(y, (e, w, b), torch.zeros(0, 64, device=DEV))
    assert y.shape == de.shape == (0, 64) and not dw.any() and not db.any()


def test_layer_norm_rows_do_not_meet():
    g = gen(6)
    x, w = normal(g, 50, 200, dtype=torch.bfloat16), 1 + normal(g, 200, scale=0.1)
    clean = tokens.layer_norm(x, w)
    for bad in (math.nan, math.inf):
        z = x.clone()
        z[7, 3] = bad
        y = tokens.layer_norm(z, w)
        assert y[7].isnan().all() and torch.equal(y[:7], clean[:7]) and torch.equal(y[8:], clean[8:])


# ------------------------------------------------------------------ gated_scan
def scan_ref(x, gate, cu, state, reverse, dy=None, dlast=None):
    """One token after another, on the CPU in float64: values, and bounds of float32 work in units of its roundoff
    (E of h: each step adds what it rounds of its terms' magnitudes H and keeps a times the error before)."""
    T, C = x.shape
    n = len(cu) - 1
    x, f = x.detach().cpu().double(), gate.detach().cpu().double()
    a, take = torch.sigmoid(f), torch.sigmoid(-f)
    z = torch.zeros(T, C, dtype=torch.float64)
    y, before, H, Hb, E, Eb = (z.clone() for _ in range(6))
    last = torch.zeros(n, C, dtype=torch.float64) if state is None else state.detach().cpu().double().clone()
    lastE, lastH = torch.zeros_like(last), last.abs()
    order = []
    for s in range(n):
        span = range(cu[s], cu[s + 1])
        order.append(list(reversed(span)) if reverse else list(span))
        for t in order[-1]:
            before[t], Hb[t], Eb[t] = last[s], lastH[s], lastE[s]
            last[s] = a[t] * last[s] + take[t] * x[t]
            lastH[s] = a[t] * lastH[s] + take[t] * x[t].abs()
            lastE[s] = a[t] * lastE[s] + lastH[s]
            y[t], H[t], E[t] = last[s], lastH[s], lastE[s]
    out = dict(y=y, last=last, E=E, lastE=lastE)
    if dy is None:
        return out
    dy = dy.detach().cpu().double()
    dx, df, eg, ef = (z.clone() for _ in range(4))
    G = torch.zeros(n, C, dtype=torch.float64) if dlast is None else dlast.detach().cpu().double().clone()
    GM, GE = G.abs(), torch.zeros_like(G)
    for s in range(n):
        for t in reversed(order[s]):
            d, M = dy[t] + G[s], dy[t].abs() + GM[s]
            e = GE[s] + M
            dx[t], df[t] = take[t] * d, d * (before[t] - x[t]) * a[t] * take[t]
            eg[t] = take[t] * (e + M)
            ef[t] = a[t] * take[t] * ((e + 4 * M) * (Hb[t] + x[t].abs()) + M * Eb[t])
            G[s], GM[s], GE[s] = a[t] * d, a[t] * M, a[t] * (e + M)
    out.update(dx=dx, df=df, dstate=G, eg=eg, ef=ef, eG=GE)
    return out


def check_scan(x, gate, cu, state, reverse, dtype, seed=0):
    g = gen(seed)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    n, C = len(cu) - 1, x.shape[1]
    dy, dlast = normal(g, *x.shape, dtype=x.dtype), normal(g, n, C)
    leaves = [t.detach().requires_grad_() for t in (x, gate) + (() if state is None else (state,))]
    y, last = tokens.gated_scan(leaves[0], leaves[1], cut, leaves[2] if state is not None else None, reverse)
    grads = torch.autograd.grad((y, last), leaves, (dy, dlast))
    r = scan_ref(x, gate, cu, state, reverse, dy, dlast)
    # a gate is 1 / (1 + exp): its exponent is off by a roundoff of |f|, and exp, the sum, the reciprocal and the
    # product each by one or two; the step adds two more
    k = (float(gate.float().abs().max()) + 10) * F32
    u = U[dtype]
    within(y, r["y"], u * r["y"].abs() + k * r["E"] + 1e-30, "y")
    within(last, r["last"], k * r["lastE"] + F32 * r["last"].abs() + 1e-30, "last")
    within(grads[0], r["dx"], u * r["dx"].abs() + k * r["eg"] + 1e-30, "dx")
    within(grads[1], r["df"], u * r["df"].abs() + k * r["ef"] + 1e-30, "dgate")
    if state is not None:
        within(grads[2], r["dstate"], k * r["eG"] + F32 * r["dstate"].abs() + 1e-30, "dstate")


def scan_inputs(T, C, dtype, seed, spread=6.0):
    g = gen(seed)
    gate = torch.rand(C, generator=g, device=DEV) * spread + torch.randn(T, C, generator=g, device=DEV)
    return normal(g, T, C, dtype=TYPES[dtype]), gate.to(TYPES[dtype])


PACKS = [[0, 1], [0, 3], [0, 17], [0, 64], [0, 65], [0, 200], [0, 700], [0, 1, 2, 3, 4], [0, 0, 5, 5, 5, 70, 200, 200],
         [0, 63, 127, 128, 129, 300], [0, 16, 32, 48, 64, 80], [0, 49, 98, 147, 196]]


@BOTH
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("cu", PACKS)
def test_gated_scan(cu, reverse, dtype):
    for C, with_state in ((1, True), (2, False), (3, True), (34, False)):
        x, gate = scan_inputs(cu[-1], C, dtype, seed=cu[-1] + C)
        state = normal(gen(C), len(cu) - 1, C) if with_state else None
        check_scan(x, gate, cu, state, reverse, dtype)


@BOTH
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens", [[3000], [1, 2500, 0, 3], [900, 1100, 40, 700]])
def test_gated_scan_long(lens, reverse, dtype):
    """Many parts, whose states come from the parts before them (and gradients from those after)."""
    cu = [0] + list(np.cumsum(lens))
    x, gate = scan_inputs(cu[-1], 6, dtype, seed=len(lens), spread=9.0)
    check_scan(x, gate, cu, normal(gen(1), len(lens), 6), reverse, dtype)


@BOTH
def test_gated_scan_tokens_of_no_sequence(dtype):
    """Before the first sequence and after the last: zeros, and zero gradients, whatever is there."""
    for reverse in (False, True):
        x, gate = scan_inputs(300, 5, dtype, seed=9)
        cu = [70, 71, 71, 200]
        keep = slice(70, 200)
        inner = [c - 70 for c in cu]
        state, dl = normal(gen(2), 3, 5), normal(gen(3), 3, 5)
        dy = normal(gen(4), 300, 5, dtype=TYPES[dtype])
        for t in (x, gate, dy):
            t[:70], t[200:] = math.nan, math.inf

        def run(x, gate, dy, cu):
            leaves = [t.detach().clone().requires_grad_() for t in (x, gate, state)]
            y, last = tokens.gated_scan(*leaves[:2], torch.tensor(cu, dtype=torch.int32, device=DEV), leaves[2], reverse)
            return (y, last) + torch.autograd.grad((y, last), leaves, (dy, dl))
        whole, part = run(x, gate, dy, cu), run(x[keep].contiguous(), gate[keep].contiguous(), dy[keep].contiguous(), inner)
        for i in (0, 2, 3):
            assert not whole[i][:70].any() and not whole[i][200:].any()
        # parts of the two packs begin at other tokens: their sums are in another order
        for a, b in zip(whole, part):
            a = a[keep] if a.shape[0] == 300 else a
            assert torch.allclose(a.float(), b.float(), rtol=2 * U[dtype] + 400 * F32, atol=400 * F32)


@BOTH
@pytest.mark.parametrize("reverse", [False, True])
def test_gated_scan_keeps_sequences_apart(reverse, dtype):
    """A sequence with values that are not finite reaches no other; parts begin and end in each."""
    cu = torch.tensor([0, 500, 1200, 1800], dtype=torch.int32, device=DEV)
    x, gate = scan_inputs(1800, 4, dtype, seed=12, spread=12.0)
    dy, state = normal(gen(5), 1800, 4, dtype=TYPES[dtype]), normal(gen(6), 3, 4)

    def run(x, gate, dy, state):
        leaves = [t.detach().clone().requires_grad_() for t in (x, gate, state)]
        y, last = tokens.gated_scan(leaves[0], leaves[1], cu, leaves[2], reverse)
        return (y, last) + torch.autograd.grad((y, last), leaves, (dy, torch.ones_like(last)))
    clean = run(x, gate, dy, state)
    for which in range(4):
        for bad in (math.nan, math.inf, -math.inf):
            args = [t.clone() for t in (x, gate, dy, state)]
            if which < 3:
                args[which][500:1200] = bad
            else:
                args[3][1] = bad
            got = run(*args)
            for i, (a, b) in enumerate(zip(got, clean)):
                if a.shape[0] == 1800:
                    assert torch.equal(a[:500], b[:500]) and torch.equal(a[1200:], b[1200:]), (which, bad, i)
                else:
                    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]), (which, bad, i)


@BOTH
@pytest.mark.parametrize("reverse", [False, True])
def test_gated_scan_not_finite_is_not_forgotten(reverse, dtype):
    """Gates that forget all but 1e-4 of the state in a step, whose product over a part is 0 in float32: what is not finite
    stays in the states of its channel up to the sequence's end, and a gradient's up to its start, and reach no other."""
    T, n, C = 9000, 5000, 8
    x, gate = scan_inputs(T, C, dtype, seed=21)
    gate = gate * 0 - 9
    x[100, 3], x[4800, 5], x[6000, 2] = float("nan"), float("inf"), float("nan")
    dy = torch.ones_like(x)
    dy[4100, 1], dy[8000, 7] = float("nan"), float("-inf")
    cu = torch.tensor([0, n, T], dtype=torch.int32, device=DEV)
    leaves = [t.clone().requires_grad_() for t in (x, gate)]
    y, last = tokens.gated_scan(*leaves, cu, reverse=reverse)
    dx, = torch.autograd.grad(y, leaves[:1], dy)
    bad = torch.zeros(T, C, dtype=torch.bool)
    bad_dx = bad.clone()
    for t, c, to in ((100, 3, bad), (4800, 5, bad), (6000, 2, bad), (4100, 1, bad_dx), (8000, 7, bad_dx)):
        a, b = (0, n) if t < n else (n, T)
        to[t:b, c] = True
        if reverse == (to is bad):   # from t towards the start
            to[t:b, c], to[a:t + 1, c] = False, True
    assert torch.equal(~y.isfinite().cpu(), bad)
    assert torch.equal(~dx.isfinite().cpu(), bad_dx)
    ends = [0, n] if reverse else [n - 1, T - 1]
    assert torch.equal(~last.isfinite().cpu(), bad[ends])


@BOTH
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("cu", [[0, 1900, 3000], [0, 45], [0, 3, 20, 20, 61]])
def test_gated_scan_infinities_stay(cu, reverse, dtype):
    """An infinity that enters a state, or a gradient, stays one of its sign where the gates keep most of it, where they keep
    little (over a part 0 in float32), and where some do; it becomes a NaN with one of the other sign or a NaN gate alone.
    What is finite is as without it."""
    T, C, n, inf = cu[-1], 8, len(cu) - 1, math.inf
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    x0, some = scan_inputs(T, C, dtype, seed=T)
    at, later = (T // 3, T // 2) if not reverse else (T // 2, T // 3)
    for gate0 in (some - 3, some * 0 + 9, some * 0 - 9):
        x, gate = x0.clone(), gate0.clone()
        state, dlast, dy = normal(gen(1), n, C), normal(gen(2), n, C), normal(gen(3), T, C, dtype=TYPES[dtype])
        clean = [t.clone() for t in (x, gate, state, dy, dlast)]
        state[:, 0] = inf
        x[at, 1], x[at, 2] = inf, -inf
        x[at, 3], x[later, 3] = inf, -inf
        dlast[:, 4], dy[later, 5] = -inf, inf
        state[:, 6], gate[later, 6] = -inf, math.nan

        def run(x, gate, state, dy, dlast):
            leaves = [t.detach().clone().requires_grad_() for t in (x, gate, state)]
            y, last = tokens.gated_scan(leaves[0], leaves[1], cut, leaves[2], reverse)
            return [t.detach() for t in (y, last) + torch.autograd.grad((y, last), leaves, (dy, dlast))]
        got, want = run(x, gate, state, dy, dlast), run(*clean)
        r = scan_ref(x, gate, cu, state, reverse, dy, dlast)
        for name, a, b in zip(("y", "last", "dx", "df", "dstate"), got, want):
            ref, a, b = r[name], a.cpu(), b.cpu()
            assert torch.equal(a.isnan(), ref.isnan()), name
            there = ref.isinf()
            assert torch.equal(a.isinf(), there) and torch.equal(a[there].double(), ref[there]), name
            assert torch.equal(a[ref.isfinite()], b[ref.isfinite()]), name
        # a token at a time
        y, new = tokens.gated_scan_step(x[at:at + 1].expand(n, C), gate[later:later + 1].expand(n, C), state)
        a = torch.sigmoid(gate[later].double())
        ref = a * state.double() + torch.sigmoid(-gate[later].double()) * x[at].double()
        assert torch.equal(new.isnan(), ref.isnan()) and torch.equal(new.isinf(), ref.isinf())
        assert torch.equal(new[ref.isinf()].double(), ref[ref.isinf()])


@BOTH
def test_gated_scan_gates_at_their_ends(dtype):
    """Gates of +-infinity and beyond what exp holds: all of the state, or none of it."""
    C, T = 6, 40
    x, _ = scan_inputs(T, C, dtype, seed=1)
    state = normal(gen(2), 1, C)
    for v in (math.inf, 200.0, 1e30):
        gate = torch.full_like(x, v)
        y, last = tokens.gated_scan(x, gate, torch.tensor([0, T], dtype=torch.int32, device=DEV), state)
        assert torch.equal(last, state) and torch.equal(y, state.to(x.dtype).expand(T, C))
        y, last = tokens.gated_scan(x, -gate, torch.tensor([0, T], dtype=torch.int32, device=DEV), state)
        # 1 - a is e / (1 + e), e = exp(87) or 2^126: the reciprocal is off by a last bit, 2^-23, the sum and the product
        # by half a bit each, and a is below 2^-125; so what is taken is 1 within 2 2^-23
        xd = x.double()
        within(y, xd, (U[dtype] + 2 * F32) * xd.abs() + 2.0 ** -120, "y")
        within(last, xd[-1:], 2 * F32 * xd[-1:].abs() + 2.0 ** -120, "last")
        leaves = [t.clone().requires_grad_() for t in (x, gate)]
        y, _ = tokens.gated_scan(*leaves, torch.tensor([0, T], dtype=torch.int32, device=DEV), state)
        dx, df = torch.autograd.grad(y, leaves, torch.ones_like(y))
        assert not dx.any() and not df.any()


def test_gated_scan_layouts_and_parts_of_the_gradient():
    g = gen(8)
    cu = torch.tensor([0, 30, 100, 301], dtype=torch.int32, device=DEV)
    proj = normal(g, 301, 3 * 7, dtype=torch.bfloat16)
    x, gate = proj[:, 1:8], proj[:, 9:16]                        # views of one projection, odd offsets
    y, last = tokens.gated_scan(x, gate, cu)
    yc, lc = tokens.gated_scan(x.contiguous(), gate.contiguous(), cu)
    assert torch.equal(y, yc) and torch.equal(last, lc)
    xt = x.t().contiguous().t()                                  # last axis not contiguous
    assert torch.equal(tokens.gated_scan(xt, gate, cu)[0], yc)
    first = normal(g, 1, 7).requires_grad_()                     # one state for all sequences
    y, last = tokens.gated_scan(x, gate, cu, first.expand(3, 7))
    each = first.detach().repeat(3, 1).requires_grad_()
    ye, le = tokens.gated_scan(x, gate, cu, each)
    assert torch.equal(y, ye) and torch.equal(last, le)
    d, = torch.autograd.grad((y, last), first, (torch.ones_like(y), torch.ones_like(last)))
    de, = torch.autograd.grad((ye, le), each, (torch.ones_like(y), torch.ones_like(last)))
    assert torch.allclose(d, de.sum(0, keepdim=True), rtol=4 * F32, atol=4 * F32 * float(de.abs().sum(0).max()))
    x, gate, state = (t.detach().clone().requires_grad_() for t in (x, gate, normal(g, 3, 7)))
    y, last = tokens.gated_scan(x, gate, cu, state)
    dl, dy = normal(g, 3, 7), normal(g, 301, 7, dtype=torch.bfloat16)
    only_last = torch.autograd.grad(last, (x, gate, state), dl, retain_graph=True)
    both = torch.autograd.grad((y, last), (x, gate, state), (torch.zeros_like(y), dl), retain_graph=True)
    only_y = torch.autograd.grad(y, (x, gate, state), dy, retain_graph=True)
    zero = torch.autograd.grad((y, last), (x, gate, state), (dy, torch.zeros_like(last)), retain_graph=True)
    for a, b in zip(only_last + only_y, both + zero):
        assert torch.equal(a, b)
    (y.float().sum() + last.sum()).backward()                    # gradients without strides
    assert x.grad.isfinite().all() and state.grad.isfinite().all()


def test_gated_scan_empty_packs():
    state = normal(gen(1), 3, 5).requires_grad_()
    for cu in ([0, 0, 0, 0],):
        x = torch.zeros(0, 5, device=DEV, requires_grad=True)
        y, last = tokens.gated_scan(x, x * 1, torch.tensor(cu, dtype=torch.int32, device=DEV), state)
        assert y.shape == (0, 5) and torch.equal(last, state)
        dx, ds = torch.autograd.grad((y, last), (x, state), (torch.zeros(0, 5, device=DEV), torch.ones(3, 5, device=DEV)))
        assert dx.shape == (0, 5) and torch.equal(ds, torch.ones(3, 5, device=DEV))
    x = normal(gen(2), 4, 5)
    y, last = tokens.gated_scan(x, x, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert not y.any() and last.shape == (0, 5)
    assert torch.equal(tokens.gated_scan(x, x, torch.tensor([2, 2, 2], dtype=torch.int32, device=DEV), state[:2].detach())[1], state[:2])


def test_gated_scan_bounds_outside_of_the_pack():
    """Entries of cu_seqlens below 0 and above T mean 0 and T; a decreasing one reads and writes nothing out of range
    (the outputs of such a pack mean nothing, but its memory's neighbours stay as they are)."""
    x, gate = scan_inputs(100, 8, "fp32", seed=4)
    got = tokens.gated_scan(x, gate, torch.tensor([-5, 40, 1 << 30], dtype=torch.int32, device=DEV))
    want = tokens.gated_scan(x, gate, torch.tensor([0, 40, 100], dtype=torch.int32, device=DEV))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    tokens.gated_scan(x, gate, torch.tensor([50, 20, 90, 10, 100], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()


def test_gated_scan_many_sequences():
    """More sequences than a search step looks at, some empty: each is its own scan."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 6, (700,), generator=g)
    cu = [0] + lens.cumsum(0).tolist()
    x, gate = scan_inputs(cu[-1], 4, "fp32", seed=5)
    check_scan(x, gate, cu, normal(gen(6), 700, 4), False, "fp32")


@pytest.mark.parametrize("reverse", [False, True])
def test_gated_scan_of_mostly_empty_sequences(reverse):
    """A short pack beside many sequences with no token: their states are passed on by many threads (one that walks all of
    them takes 0.2 us each, 0.2 s), and so are their gradients."""
    n, T, C = 1 << 20, 37, 3
    cu = torch.full((n + 1,), T, dtype=torch.int32, device=DEV)
    cu[:500], cu[500:n // 2] = 0, 21
    x, gate = scan_inputs(T, C, "fp32", seed=2)
    state, dlast, dy = normal(gen(3), n, C), normal(gen(4), n, C), normal(gen(5), T, C)

    def timed(f):
        f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        got = f()
        b.record()
        torch.cuda.synchronize()
        assert a.elapsed_time(b) < 20
        return got
    y, last, kept = timed(lambda: tb.wtconv_gated_scan_forward(x, gate, cu, state, reverse, want_kept=True))
    dx, dgate, dstate = timed(lambda: tb.wtconv_gated_scan_backward(dy, dlast, x, gate, cu, state, kept, reverse))
    full = [499, n // 2 - 1]
    few = lambda t: t[full].contiguous()
    cuf = torch.tensor([0, 21, T], dtype=torch.int32, device=DEV)
    yf, lastf, keptf = tb.wtconv_gated_scan_forward(x, gate, cuf, few(state), reverse, want_kept=True)
    dxf, dgatef, dstatef = tb.wtconv_gated_scan_backward(dy, few(dlast), x, gate, cuf, few(state), keptf, reverse)
    for a, b in ((y, yf), (last[full], lastf), (dx, dxf), (dgate, dgatef), (dstate[full], dstatef)):
        assert torch.equal(a, b)
    empty = torch.ones(n, dtype=torch.bool, device=DEV)
    empty[full] = False
    assert torch.equal(last[empty], state[empty]) and torch.equal(dstate[empty], dlast[empty])


def test_gated_scan_of_the_largest_pack():
    """2^31 - 1025 tokens of one channel, whose last part ends 2^31 tokens after the first one's begin if it is taken whole:
    every 2^20th token sets the state, the others keep it, and the last one's gradient goes back to the last that set it."""
    T, each = (1 << 31) - (1 << 10) - 1, 1 << 20
    n = (T + each - 1) // each
    value = (torch.arange(n, device=DEV) % 128 + 1).bfloat16()                  # exact
    x, gate = (torch.full((T, 1), v, dtype=torch.bfloat16, device=DEV) for v in (0.0, 200.0))
    x[::each, 0], gate[::each] = value, -200.0
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    y, last, kept = tb.wtconv_gated_scan_forward(x, gate, cu, want_kept=True)
    for i in range(n):
        assert (y[i * each:(i + 1) * each] == value[i]).all(), i
    assert last.item() == value[-1].item()
    dy = torch.zeros_like(y)
    dy[-1] = 3.0
    dx, dgate, _ = tb.wtconv_gated_scan_backward(dy, torch.full_like(last, 2.0), x, gate, cu, None, kept)
    assert dx[(n - 1) * each].item() == 5.0 and not dgate.any()
    dx[(n - 1) * each] = 0
    assert not dx.any()


def test_gated_scan_is_the_same_again():
    cu = torch.tensor([0, 5000, 9000], dtype=torch.int32, device=DEV)
    x, gate = (t.requires_grad_() for t in scan_inputs(9000, 33, "bf16", seed=7))
    dy = normal(gen(8), 9000, 33, dtype=torch.bfloat16)

    def run():
        y, last = tokens.gated_scan(x, gate, cu)
        return (y, last) + torch.autograd.grad((y, last), (x, gate), (dy, torch.ones_like(last)))
    first = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@BOTH
@pytest.mark.parametrize("n,C", [(1, 1), (3, 7), (128, 768), (5, 4099)])
def test_gated_scan_step(n, C, dtype):
    x, gate = scan_inputs(n, C, dtype, seed=n + C)
    state = normal(gen(C), n, C)
    y, new = tokens.gated_scan_step(x, gate, state)
    a, take = torch.sigmoid(gate.double()), torch.sigmoid(-gate.double())
    h = a * state.double() + take * x.double()
    k = (float(gate.float().abs().max()) + 10) * F32
    size = a * state.double().abs() + take * x.double().abs()
    within(new, h, k * size, "state")
    assert torch.equal(y, new.to(y.dtype))
    same = state.clone()
    y2, out = tokens.gated_scan_step(x, gate, same, out=same)     # in place
    assert out is same and torch.equal(same, new) and torch.equal(y2, y)
    # one token a sequence of a pack is the same, bit for bit
    yp, last = tokens.gated_scan(x, gate, torch.arange(n + 1, dtype=torch.int32, device=DEV), state)
    assert torch.equal(yp, y) and torch.equal(last, new)


def test_gated_scan_step_strided_and_empty():
    proj = normal(gen(1), 9, 30, dtype=torch.bfloat16)
    state = normal(gen(2), 9, 7)
    a = tokens.gated_scan_step(proj[:, 3:10], proj[:, 11:18], state)
    b = tokens.gated_scan_step(proj[:, 3:10].contiguous(), proj[:, 11:18].contiguous(), state)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    e = torch.zeros(0, 7, device=DEV)
    assert tokens.gated_scan_step(e, e, e)[0].shape == (0, 7)


# ------------------------------------------------------------------ experts' rows
def order_ref(experts, E):
    e = experts.cpu().numpy().reshape(-1)
    there = (e >= 0) & (e < E)
    at = np.argsort(np.where(there, e, E), kind="stable")
    live = int(there.sum())
    slot = np.full(e.size, -1)
    slot[at[:live]] = np.arange(live)
    pair = np.where(np.arange(e.size) < live, at, -1)
    return slot.reshape(experts.shape), pair, np.concatenate(([0], np.cumsum(np.bincount(e[there], minlength=E))))


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 8), (63, 1, 3), (64, 2, 7), (1000, 3, 5), (4096, 2, 8), (4097, 2, 512),
                                   (8193, 1, 64), (30000, 2, 37), (100, 4, 512), (70000, 1, 1), (20011, 8, 300)])
@pytest.mark.parametrize("absent", [0.0, 0.3, 1.0])
def test_expert_order(T, k, E, absent):
    g = gen(T + E)
    experts = (torch.rand(T, k, generator=g, device=DEV) ** 2 * E).int()     # low numbers more often
    gone = torch.rand(T, k, generator=g, device=DEV) < absent
    experts = torch.where(gone, torch.randint(-3, 0, (T, k), generator=g, device=DEV).int(), experts)
    if absent == 0.3:
        experts[:, 0] = torch.where(gone[:, 0], E + 5, experts[:, 0])        # too large is none's too
    slot, pair, cu = tokens.expert_order(experts, E)
    for got, want in zip((slot, pair, cu), order_ref(experts, E)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)


def test_expert_order_of_nothing():
    slot, pair, cu = tokens.expert_order(torch.zeros(0, 2, dtype=torch.int32, device=DEV), 5)
    assert slot.shape == (0, 2) and pair.shape == (0,) and cu.tolist() == [0] * 6


@BOTH
@pytest.mark.parametrize("T,k,E,C", [(1, 1, 1, 1), (5, 2, 3, 7), (49, 2, 8, 768), (1000, 1, 4, 24), (301, 3, 5, 387),
                                     (777, 5, 11, 130), (64, 8, 8, 16), (20, 2, 4, 5000), (2000, 6, 40, 96)])
def test_expert_gather_and_combine(T, k, E, C, dtype):
    g, dt, u = gen(T * 7 + C), TYPES[dtype], U[dtype]
    experts = torch.rand(T, E, generator=g, device=DEV).topk(min(k, E), 1).indices.int()
    k = experts.shape[1]
    experts[torch.rand(T, k, generator=g, device=DEV) < 0.2] = -1
    order = tokens.expert_order(experts, E)
    x, rows = normal(g, T, C, dtype=dt).requires_grad_(), normal(g, T * k, C, dtype=dt)
    live = int(order.cu_experts[-1])
    rows[live:] = math.nan                                   # what no expert has does not matter
    rows.requires_grad_()
    w = torch.rand(T, k, generator=g, device=DEV).requires_grad_()
    xs = tokens.expert_gather(x, order)
    pair = order.pair.long()
    assert torch.equal(xs[:live], x[pair[:live] // k]) and not xs[live:].any()
    y = tokens.expert_combine(rows, w, order)
    dxs, dy = normal(g, T * k, C, dtype=dt), normal(g, T, C, dtype=dt)
    dxs[live:] = math.nan
    dx, = torch.autograd.grad(xs, x, dxs)
    dr, dw = torch.autograd.grad(y, (rows, w), dy)
    with torch.no_grad():
        there = (order.slot >= 0)
        at = order.slot.long().clamp_min(0)
        picked = torch.where(there[..., None], rows.double()[at], 0.0)
        terms = picked * w.double()[..., None]
        within(y, terms.sum(1), u * terms.sum(1).abs() + (k + 1) * F32 * terms.abs().sum(1) + 1e-30, "y")
        parts = torch.where(there[..., None], dxs.double()[at], 0.0)
        within(dx, parts.sum(1), u * parts.sum(1).abs() + (k + 1) * F32 * parts.abs().sum(1) + 1e-30, "dx")
        want = dy.double()[pair[:live] // k] * w.double().view(-1)[pair[:live]][:, None]
        within(dr[:live], want, u * want.abs() * (1 + F32) + F32 * want.abs() + 1e-30, "drows")
        assert not dr[live:].any()
        dots = picked * dy.double()[:, None]
        within(dw, dots.sum(2), (C + 1) * F32 * dots.abs().sum(2) + 1e-30, "dweights")


def test_expert_rows_layouts():
    g = gen(4)
    experts = torch.tensor([[0, 1], [1, 2], [2, 0], [-1, 1]], dtype=torch.int32, device=DEV)
    order = tokens.expert_order(experts.t().contiguous().t(), 3)           # not contiguous
    assert torch.equal(order.slot, tokens.expert_order(experts, 3).slot)
    big = normal(g, 8, 3 * 9, dtype=torch.bfloat16)
    x, rows, w = big[:4, 1:10], big[:, 11:20], torch.rand(4, 2, device=DEV)
    assert torch.equal(tokens.expert_gather(x, order), tokens.expert_gather(x.contiguous(), order))
    assert torch.equal(tokens.expert_combine(rows, w, order), tokens.expert_combine(rows.contiguous(), w, order))
    xt = x.t().contiguous().t()
    assert torch.equal(tokens.expert_gather(xt, order), tokens.expert_gather(x.contiguous(), order))
    wt = w.t().contiguous().t().requires_grad_()                           # weights in another order, and broadcast ones
    y = tokens.expert_combine(rows.contiguous().requires_grad_(), wt, order)
    assert torch.equal(y, tokens.expert_combine(rows, w, order))
    one = torch.rand(1, 1, device=DEV, requires_grad=True)
    tokens.expert_combine(rows, one.expand(4, 2), order).float().sum().backward()
    assert one.grad.shape == (1, 1)
    x = x.detach().clone().requires_grad_()
    tokens.expert_gather(x, order).float().sum().backward()                # a gradient without strides
    assert torch.equal(x.grad.float(), (experts >= 0).sum(1, keepdim=True).expand(4, 9).float())
    empty = tokens.expert_order(torch.zeros(0, 2, dtype=torch.int32, device=DEV), 3)
    e = torch.zeros(0, 9, device=DEV)
    assert tokens.expert_gather(e, empty).shape == (0, 9) and tokens.expert_combine(e, torch.zeros(0, 2, device=DEV), empty).shape == (0, 9)


# ------------------------------------------------------------------ experts' products
def product_case(counts, K, N, dtype, bias, seed, before=0, after=0, scale=1.0):
    g, dt = gen(seed), TYPES[dtype]
    R, E = before + sum(counts) + after, len(counts)
    cu = torch.tensor([before] + counts, device=DEV).cumsum(0).to(torch.int32)
    x, w = normal(g, R, K, dtype=dt, scale=scale), normal(g, E, N, K, dtype=dt, scale=K ** -0.5)
    b = normal(g, E, N, dtype=dt) if bias else None
    return x, w, b, cu, normal(g, R, N, dtype=dt)


def check_product(x, w, b, cu, dy, dtype):
    leaves = [t.requires_grad_() for t in (x, w, b) if t is not None]
    y = tokens.expert_linear(x, w, cu, b)
    grads = torch.autograd.grad(y, leaves, dy)
    u, at = U[dtype], cu.tolist()
    E, N, K = w.shape
    with torch.no_grad():
        none = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
        none[at[0]:at[-1]] = False
        assert not y[none].any() and not grads[0][none].any()
        for e in range(E):
            rows = slice(at[e], at[e + 1])
            n = at[e + 1] - at[e]
            xe, we, ge = x[rows].double(), w[e].double(), dy[rows].double()
            be = b[e].double() if b is not None else torch.zeros(N, dtype=torch.float64, device=DEV)
            ref = xe @ we.T + be
            within(y[rows], ref, u * ref.abs() + (K + 16) * F32 * (xe.abs() @ we.abs().T + be.abs()) + 1e-30, f"y of expert {e}")
            ref = ge @ we
            within(grads[0][rows], ref, u * ref.abs() + (N + 16) * F32 * (ge.abs() @ we.abs()) + 1e-30, f"dx of expert {e}")
            ref = ge.T @ xe
            within(grads[1][e], ref, u * ref.abs() + (n + 16) * F32 * (ge.abs().T @ xe.abs()) + 1e-30, f"dweight of expert {e}")
            if b is not None:
                ref = ge.sum(0)
                within(grads[2][e], ref, u * ref.abs() + (n + 16) * F32 * ge.abs().sum(0) + 1e-30, f"dbias of expert {e}")


@BOTH
@pytest.mark.parametrize("counts,K,N", [([1], 8, 8), ([3, 0, 5], 16, 24), ([0, 0, 0], 64, 64), ([40, 7, 1, 130], 72, 136),
                                        ([128, 128], 64, 128), ([129, 255, 31], 200, 264), ([1] * 9, 104, 40),
                                        ([64, 65, 63, 0, 1], 128, 96), ([500], 392, 8), ([5, 300], 8, 520),
                                        ([33, 32, 31] * 7, 64, 64), ([0] * 70 + [5] * 80, 32, 48)])
def test_expert_linear(counts, K, N, dtype):
    check_product(*product_case(counts, K, N, dtype, bias=True, seed=K + N), dtype)


@BOTH
@pytest.mark.parametrize("counts,K,N", [([9000, 100, 0, 300], 520, 264), ([40] * 20 + [3000, 0, 1500] + [17] * 25, 520, 1000),
                                        ([8] * 70 + [2500, 0, 1300] + [5] * 30, 64, 40), ([1200, 1300], 72, 80),
                                        ([14000, 0, 3001, 70, 4000], 1000, 1016), ([30] * 20 + [9000] + [500] * 30, 1000, 1016)])
def test_expert_linear_of_uneven_experts(counts, K, N, dtype):
    """Gradients of weights in parts of an expert's rows: some experts whole, some in parts, up to 64 of them and more."""
    check_product(*product_case(counts, K, N, dtype, bias=True, seed=len(counts)), dtype)


def test_expert_linear_with_bounds_in_no_order():
    """Experts whose rows overlap have more together than there are: their gradients are anything, but stay where they belong."""
    x, w, b, cu, dy = product_case([3000, 0, 0, 0], 64, 48, "fp32", True, seed=8)
    guard = torch.full((4 * 48 * 64,), 7.0, device=DEV)
    bad = torch.tensor([0, 3000, 0, 3000, -5], dtype=torch.int32, device=DEV)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    torch.autograd.grad(tokens.expert_linear(leaves[0], leaves[1], bad, leaves[2]), leaves, dy)
    torch.cuda.synchronize()
    assert torch.equal(guard, torch.full_like(guard, 7.0))
    check_product(x, w, b, cu, dy, "fp32")


class Guarded:
    """Outputs and workspaces of C calls one after another in one allocation, 4 KB of a known byte around each."""
    PAD, BYTE = 4096, 0xA5

    def __init__(self, *sizes):
        self.at, end = [], self.PAD
        for n in sizes:
            self.at.append((end, n))
            end += (n + 255) // 256 * 256 + self.PAD
        self.memory = torch.full((end,), self.BYTE, dtype=torch.uint8, device=DEV)

    def __getitem__(self, i):
        return self.memory.data_ptr() + self.at[i][0]

    def tensor(self, i, dtype):
        a, n = self.at[i]
        return self.memory[a:a + n].view(dtype)

    def check(self):
        torch.cuda.synchronize()
        outside = torch.ones_like(self.memory, dtype=torch.bool)
        for a, n in self.at:
            outside[a:a + n] = False
        assert (self.memory[outside] == self.BYTE).all()


@BOTH
@pytest.mark.parametrize("R,K,N,E,bounds", [
    (3000, 64, 48, 4, [0, 3000, 0, 3000, -5]), (3000, 64, 48, 4, [0, 3000, 3000, 3000, 3000]), (12000, 8, 8, 3, [0, 12000, 0, 12000]),
    (20000, 264, 136, 4, [9000, 20000, -7, 20000, 0]), (9, 520, 24, 5, [9, 0, 9, 3, 5, 1 << 30]), (400, 64, 264, 3, [400, 0, 399, 1]),
    (6000, 1000, 1016, 6, [0, 6000, 0, 6000, 0, 6000, 0])])
def test_expert_linear_writes_its_outputs_alone(R, K, N, E, bounds, dtype):
    """Bounds of experts in any order: outputs and sums of parts are anything, but what lies around them in memory stays."""
    g, dt = gen(R), TYPES[dtype]
    size = dt.itemsize
    x, dy, w, b = (normal(g, *s, dtype=dt) for s in ((R, K), (R, N), (E, N, K), (E, N)))
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    d = tb.wtc_expert_desc(R, K, N, E, K, N, 0 if dtype == "fp32" else 1)
    ref, lib = ctypes.addressof(d), tb._load()
    need = lib.wtconv_expert_linear_weight_grad_workspace(ref)
    out = Guarded(R * N * size, R * K * size, E * N * K * size, E * N * size, need)
    dev = x.device
    tb._call("wtconv_expert_linear_forward", dev, ref, x.data_ptr(), w.data_ptr(), b.data_ptr(), cu.data_ptr(), out[0])
    out.check()
    tb._call("wtconv_expert_linear_input_grad", dev, ref, dy.data_ptr(), w.data_ptr(), cu.data_ptr(), out[1])
    out.check()
    tb._call("wtconv_expert_linear_weight_grad", dev, ref, dy.data_ptr(), x.data_ptr(), cu.data_ptr(), out[2], out[3], out[4], need)
    out.check()
    if bounds == sorted(bounds):
        y = tokens.expert_linear(x, w, cu, b)
        dw, db = tb.wtconv_expert_linear_weight_grad(dy, x, cu)
        dx = tb.wtconv_expert_linear_input_grad(dy, w, cu)
        for i, t in enumerate((y, dx, dw, db)):
            assert torch.equal(out.tensor(i, dt), t.reshape(-1))


@BOTH
@pytest.mark.parametrize("reverse", [0, 1])
@pytest.mark.parametrize("T,C,bounds", [(300, 7, [0, 100, 300]), (300, 7, [250, 20, 280, 10, 300, -3, 400]), (41, 1, [40, 0, 41]),
                                        (2000, 34, [1999, 0, 2000, 5]), (64, 3, [0, 0, 64, 64, 2])])
def test_gated_scan_writes_its_outputs_alone(T, C, bounds, reverse, dtype):
    x, gate = scan_inputs(T, C, dtype, seed=T)
    n, dt = len(bounds) - 1, TYPES[dtype]
    dy, state, dlast = normal(gen(1), T, C, dtype=dt), normal(gen(2), n, C), normal(gen(3), n, C)
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    d = tb.wtc_scan_desc(T, C, C, C, n, C, 0 if dtype == "fp32" else 1, reverse)
    ref, lib = ctypes.addressof(d), tb._load()
    kept, need = lib.wtconv_gated_scan_kept(ref), lib.wtconv_gated_scan_workspace(ref)
    row, states = T * C * dt.itemsize, n * C * 4
    out = Guarded(row, states, kept, need, row, row, states)
    tb._call("wtconv_gated_scan_forward", x.device, ref, x.data_ptr(), gate.data_ptr(), cu.data_ptr(), state.data_ptr(), out[0],
             out[1], out[2], out[3], need)
    out.check()
    tb._call("wtconv_gated_scan_backward", x.device, ref, x.data_ptr(), gate.data_ptr(), cu.data_ptr(), state.data_ptr(), out[2],
             dy.data_ptr(), dlast.data_ptr(), out[4], out[5], out[6], out[3], need)
    out.check()
    if bounds == sorted(bounds):
        y, last, k = tb.wtconv_gated_scan_forward(x, gate, cu, state, reverse, want_kept=True)
        grads = tb.wtconv_gated_scan_backward(dy, dlast, x, gate, cu, state, k, reverse)
        for i, t in zip((0, 1, 4, 5, 6), (y, last) + grads):
            assert torch.equal(out.tensor(i, t.dtype), t.reshape(-1))


@BOTH
@pytest.mark.parametrize("T,k,E,C", [(1, 1, 1, 1), (63, 3, 5, 33), (700, 2, 9, 130), (5000, 2, 70, 9)])
def test_expert_rows_write_their_outputs_alone(T, k, E, C, dtype):
    g, dt, dev = gen(T), TYPES[dtype], torch.device(DEV, 0)
    experts = torch.randint(-1, E, (T, k), generator=g, device=DEV).int()
    x, rows, dy, weights = normal(g, T, C, dtype=dt), normal(g, T * k, C, dtype=dt), normal(g, T, C, dtype=dt), normal(g, T, k)
    lib, n = tb._load(), T * k
    need = lib.wtconv_expert_order_workspace(n, E)
    d = tb.wtc_rows_desc(T, C, C, k, E, C, 0 if dtype == "fp32" else 1)
    ref, one, all_rows = ctypes.addressof(d), T * C * dt.itemsize, n * C * dt.itemsize
    out = Guarded(4 * n, 4 * n, 4 * (E + 1), need, all_rows, one, all_rows, 4 * n)
    tb._call("wtconv_expert_order", dev, n, E, experts.data_ptr(), out[0], out[1], out[2], out[3], need)
    out.check()
    tb._call("wtconv_expert_gather", dev, ref, x.data_ptr(), out[0], out[2], out[4])
    tb._call("wtconv_expert_combine", dev, ref, rows.data_ptr(), weights.data_ptr(), out[0], out[5])
    tb._call("wtconv_expert_combine_backward", dev, ref, dy.data_ptr(), rows.data_ptr(), weights.data_ptr(), out[0], out[2], out[6], out[7])
    out.check()
    order = tokens.expert_order(experts, E)
    want = tuple(order) + (tokens.expert_gather(x, order), tokens.expert_combine(rows, weights, order))
    for i, t in zip((0, 1, 2, 4, 5, 6, 7), want + tb.wtconv_expert_combine_backward(dy, rows, weights, order.slot, order.cu_experts)):
        assert torch.equal(out.tensor(i, t.dtype), t.reshape(-1))


@BOTH
@pytest.mark.parametrize("counts,K,N", [([1], 2048, 64), ([0, 2, 0, 1], 1000, 72), ([0] * 100 + [1] + [0] * 50 + [2, 0, 1] + [0] * 300, 520, 40),
                                        ([16, 17, 0, 15], 264, 136), ([33, 1], 72, 24), ([1] * 3, 8, 8), ([3, 2, 4], 4104, 16)])
def test_expert_linear_of_few_rows(counts, K, N, dtype):
    """A step of a few sequences: fewer rows than experts or not, rows of no expert on both sides, terms that end inside a
    read, waves with none."""
    x, w, b, cu, dy = product_case(counts, K, N, dtype, True, seed=K + N, before=2, after=3)
    x[:2], x[-3:] = math.nan, math.inf
    check_product(x, w, b, cu, dy, dtype)


@BOTH
def test_expert_linear_of_the_largest_tiles(dtype):
    """Enough tiles for those of 256 x 256 in both directions (bfloat16), with a part of a step, of a tile's rows and of its
    columns left over, experts of one row and of none; in float32 the weights' gradient of three parts."""
    check_product(*product_case([1, 3000, 0, 2543, 128, 4000, 257, 2615], 1000, 1016, dtype, bias=True, seed=77), dtype)


@BOTH
@pytest.mark.parametrize("counts,K,N", [([30000, 2769], 64, 256), ([5000, 0, 9000, 2400], 264, 1032), ([700, 900, 2000], 1096, 512),
                                        ([3000], 64, 64), ([9000], 72, 40)])
def test_expert_linear_large(counts, K, N, dtype):
    """The larger tiles, and sums over rows that several workgroups share."""
    check_product(*product_case(counts, K, N, dtype, bias=False, seed=K + N), dtype)


def test_expert_linear_of_more_tiles_than_a_launch_has():
    """1.2 billion rows of 8 channels: tiles of rows in three launches.  Whole numbers that come again every 2^20 + 7 rows, so
    that every sum is exact: products up to 48; the gradients' 10^6 (random walks of 10^6 steps of at most 2, 400 times)."""
    R, E, P = (1 << 30) + (1 << 27), 3, (1 << 20) + 7
    at = [77, R // 3, R // 3, R - 1000]
    g = gen(5)
    px, pdy = (torch.randint(-n, n + 1, (P, 8), generator=g, device=DEV).bfloat16() for n in (2, 1))
    x, dy = (t.repeat(R // P + 1, 1)[:R] for t in (px, pdy))
    w = torch.randint(-3, 4, (E, 8, 8), generator=g, device=DEV).bfloat16()
    cu = torch.tensor(at, dtype=torch.int32, device=DEV)
    # an expert's runs of rows from one multiple of P to the next
    runs = [(e, max(r, at[e]), min(r + P, at[e + 1])) for e in range(E) for r in range(at[e] // P * P, at[e + 1], P)]
    for out, of, turned in ((tokens.expert_linear(x, w, cu), px, w.transpose(1, 2)),
                            (tb.wtconv_expert_linear_input_grad(dy, w, cu), pdy, w)):
        assert not out[:at[0]].any() and not out[at[-1]:].any()
        want = [(of.float() @ turned[e].float().contiguous()).bfloat16() for e in range(E)]
        for e, a, b in runs:
            assert torch.equal(out[a:b], want[e][a % P:a % P + b - a]), (e, a)
    del out
    dw, db = tb.wtconv_expert_linear_weight_grad(dy, x, cu)
    # products and dy of rows 0 .. r - 1 of the first P summed: 64 and 8 columns
    both = torch.cat([(pdy[:, :, None] * px[:, None]).view(P, 64), pdy], 1).double().cumsum(0)
    both = torch.cat([torch.zeros_like(both[:1]), both])
    want = torch.zeros(E, 72, dtype=torch.float64, device=DEV)
    for e, a, b in runs:
        want[e] += both[a % P + b - a] - both[a % P]
    assert torch.equal(dw, want[:, :64].view(E, 8, 8).bfloat16()) and torch.equal(db, want[:, 64:].bfloat16())


@BOTH
def test_expert_linear_rows_of_no_expert(dtype):
    """Before the first expert's rows and after the last's: zeros, and nothing of them reaches a gradient."""
    x, w, b, cu, dy = product_case([50, 0, 77], 40, 72, dtype, True, seed=2, before=13, after=200)
    x[:13], x[140:], dy[:13], dy[140:] = math.nan, math.inf, math.inf, math.nan
    check_product(x, w, b, cu, dy, dtype)


@BOTH
def test_expert_linear_keeps_experts_apart(dtype):
    """Values that are not finite reach their expert's results alone, also where a tile's last rows or terms end."""
    counts, K, N = [70, 45, 61], 40, 56
    x, w, b, cu, dy = product_case(counts, K, N, dtype, True, seed=3)

    def run(x, w, dy):
        leaves = [t.detach().clone().requires_grad_() for t in (x, w, b)]
        y = tokens.expert_linear(leaves[0], leaves[1], cu, leaves[2])
        return (y,) + torch.autograd.grad(y, leaves, dy)
    clean = run(x, w, dy)
    for which in range(3):
        args = [t.clone() for t in (x, w, dy)]
        args[which][1 if which == 1 else slice(70, 115)] = math.nan
        got = run(*args)
        for a, c in zip(got[:2], clean[:2]):
            assert torch.equal(a[:70], c[:70]) and torch.equal(a[115:], c[115:])
        for a, c in zip(got[2:], clean[2:]):
            assert torch.equal(a[0], c[0]) and torch.equal(a[2], c[2])


def test_expert_linear_float32_is_float32():
    """The products of three parts against float32's own: 24 bits of each factor.  One term of K = 8 is not zero, so the
    result is one product; the parts that are left out are below 3 2^-24 of it, and it is rounded once."""
    g = gen(5)
    x, w = torch.zeros(64, 8, device=DEV), torch.zeros(1, 64, 8, device=DEV)
    x[:, 3], w[0, :, 3] = normal(g, 64, scale=3.0), normal(g, 64)
    y = tokens.expert_linear(x, w, torch.tensor([0, 64], dtype=torch.int32, device=DEV))
    want = x[:, 3].double()[:, None] * w[0, :, 3].double()
    within(y, want, 4 * 2.0 ** -24 * want.abs(), "y")


def test_expert_linear_layouts():
    g = gen(6)
    cu = torch.tensor([0, 20, 33], dtype=torch.int32, device=DEV)
    w, b = normal(g, 2, 24, 16, dtype=torch.bfloat16), normal(g, 2, 24, dtype=torch.bfloat16)
    big = normal(g, 33, 64, dtype=torch.bfloat16)
    want = tokens.expert_linear(big[:, 8:24].contiguous(), w, cu, b)
    assert torch.equal(tokens.expert_linear(big[:, 8:24], w, cu, b), want)           # strided rows, aligned
    odd = torch.empty(33 * 64 + 1, device=DEV, dtype=torch.bfloat16)[1:].view(33, 64).copy_(big)
    assert torch.equal(tokens.expert_linear(odd[:, 8:24], w, cu, b), want)           # not aligned
    assert torch.equal(tokens.expert_linear(big[:, 8:24].t().contiguous().t(), w, cu, b), want)
    wide = torch.empty(2 * 24 * 16 + 1, device=DEV, dtype=torch.bfloat16)[1:].view(2, 24, 16).copy_(w)
    assert torch.equal(tokens.expert_linear(big[:, 8:24], wide, cu, b), want)
    x = big[:, 8:24].detach().requires_grad_()
    wr = w.clone().requires_grad_()
    y = tokens.expert_linear(x, wr, cu)
    y.float().sum().backward()                                                       # a gradient without strides
    assert torch.allclose(x.grad[:20].float(), w[0].float().sum(0).expand(20, 16), rtol=2.0 ** -7, atol=1e-3)
    only = torch.autograd.grad(tokens.expert_linear(x, w, cu, b), x, torch.ones(33, 24, device=DEV, dtype=torch.bfloat16))
    assert torch.equal(only[0], x.grad)
    empty = tokens.expert_linear(torch.zeros(0, 16, device=DEV, dtype=torch.bfloat16), wr, torch.zeros(3, dtype=torch.int32, device=DEV))
    dw, = torch.autograd.grad(empty, wr, torch.zeros(0, 24, device=DEV, dtype=torch.bfloat16))
    assert empty.shape == (0, 24) and not dw.any()


def test_expert_linear_bounds_outside_of_the_rows():
    x, w, b, cu, dy = product_case([30, 34], 16, 16, "fp32", False, seed=7)
    got = tokens.expert_linear(x, w, torch.tensor([-7, 30, 1 << 30], dtype=torch.int32, device=DEV))
    assert torch.equal(got, tokens.expert_linear(x, w, cu))
    x.requires_grad_(), w.requires_grad_()
    y = tokens.expert_linear(x, w, torch.tensor([40, 10, 64], dtype=torch.int32, device=DEV))   # decreasing: nothing out of range
    torch.autograd.grad(y, (x, w), dy)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ by differences
def by_differences(f, args, seed):
    """The gradient along a direction against differences of f's values.  A difference over 2 e is off by its third
    derivative, which is a third of how far the one over 4 e is off from it, and by the float32 noise of f over e."""
    args = [a.detach().clone().requires_grad_() for a in args]
    g = gen(seed)
    out = [o for o in f(*args) if o is not None]
    weights = [normal(g, *o.shape) for o in out]
    grads = torch.autograd.grad(out, args, weights)
    way = [normal(g, *a.shape) for a in args]
    got = sum((d.double() * v.double()).sum() for d, v in zip(grads, way))

    def loss(e):
        with torch.no_grad():
            o = [t for t in f(*(a + e * v for a, v in zip(args, way))) if t is not None]
            return sum((t.double() * w.double()).sum() for t, w in zip(o, weights)), \
                sum((t.double() * w.double()).abs().sum() for t, w in zip(o, weights))
    e = 2.0 ** -7
    (p1, m), (n1, _), (p2, _), (n2, _) = loss(e), loss(-e), loss(2 * e), loss(-2 * e)
    near, far = (p1 - n1) / (2 * e), (p2 - n2) / (4 * e)
    assert abs(got - near) <= abs(far - near) + 64 * F32 * m / e, (float(got), float(near), float(far))


def test_gradients_by_differences():
    g = gen(9)
    cu = torch.tensor([0, 9, 9, 30, 70], dtype=torch.int32, device=DEV)
    by_differences(lambda x, w, b, r: tokens.layer_norm(x, w, b, r), (normal(g, 9, 40), 1 + normal(g, 40, scale=0.1), normal(g, 40), normal(g, 9, 40)), 1)
    for reverse in (False, True):
        by_differences(lambda x, f, s: tokens.gated_scan(x, f, cu, s, reverse), (normal(g, 70, 12), normal(g, 70, 12), normal(g, 4, 12)), 2)
    order = tokens.expert_order(torch.randint(-1, 4, (30, 2), generator=g, device=DEV).int(), 4)
    by_differences(lambda x: (tokens.expert_gather(x, order),), (normal(g, 30, 20),), 3)
    by_differences(lambda r, w: (tokens.expert_combine(r, w, order),), (normal(g, 60, 20), normal(g, 30, 2)), 4)
    by_differences(lambda x, w, b: (tokens.expert_linear(x, w, order.cu_experts, b),),
                   (normal(g, 60, 24), normal(g, 4, 32, 24, scale=0.2), normal(g, 4, 32)), 5)


# ------------------------------------------------------------------ together
def test_experts_are_the_sum_of_dense_branches():
    """The module against each expert's branch on all tokens, weighted: float32, so both round K terms a layer."""
    torch.manual_seed(0)
    m = tokens.Experts(24, 40, 5, k=2, device=DEV, dtype=torch.float32)
    x = torch.randn(50, 24, device=DEV)
    top, chosen = m.router(x).topk(2, 1)
    w = torch.zeros(50, 5, device=DEV, dtype=torch.float64).scatter_(1, chosen, torch.softmax(top, 1).double())
    d = lambda p: p.detach().double()
    dense = torch.stack([torch.nn.functional.gelu(d(x) @ d(m.up[e]).T + d(m.up_bias[e])) @ d(m.down[e]).T + d(m.down_bias[e])
                         for e in range(5)], 1)
    want = (w[..., None] * dense).sum(1)
    assert torch.allclose(m(x).double(), want.detach(), rtol=0, atol=200 * F32 * float(dense.abs().max()))


@pytest.mark.parametrize("causal", [False, True])
def test_scan_block_is_its_parts(causal):
    torch.manual_seed(1)
    m = tokens.ScanBlock(32, hidden=48, experts=4, causal=causal, device=DEV, dtype=torch.bfloat16)
    cu = torch.tensor([0, 20, 55], dtype=torch.int32, device=DEV)
    x = torch.randn(55, 32, device=DEV, dtype=torch.bfloat16)
    p = m.values(m.norm1(x))
    if causal:
        mixed = tokens.gated_scan(p[:, :32].contiguous(), p[:, 32:].contiguous(), cu)[0]
    else:
        a = tokens.gated_scan(p[:, :16].contiguous(), p[:, 32:48].contiguous(), cu)[0]
        b = tokens.gated_scan(p[:, 16:32].contiguous(), p[:, 48:].contiguous(), cu, reverse=True)[0]
        mixed = torch.cat([a, b], 1)
    h = x + m.proj(mixed)
    assert torch.equal(m(x, cu), h + m.experts(m.norm2(h)))
    y = m(x.requires_grad_(), cu)
    y.float().square().mean().backward()
    assert all(t.grad is not None and t.grad.isfinite().all() for t in m.parameters())


def test_scan_block_token_after_token():
    """A causal block's steps give what it gives on whole sequences: float32, 30 tokens of sums of at most 64 terms."""
    torch.manual_seed(2)
    m = tokens.ScanBlock(32, experts=4, causal=True, device=DEV, dtype=torch.float32)
    x = torch.randn(3, 30, 32, device=DEV)
    whole = m(x.reshape(90, 32), torch.tensor([0, 30, 60, 90], dtype=torch.int32, device=DEV)).view(3, 30, 32)
    state = torch.zeros(3, 32, device=DEV)
    for t in range(30):
        out, same = m.step(x[:, t], state)
        assert same is state
        assert torch.allclose(out, whole[:, t], rtol=0, atol=4000 * F32 * float(whole.abs().max()))
    with pytest.raises(ValueError, match="causal"):
        tokens.ScanBlock(32, device=DEV).step(x[:, 0], state)


def test_hybrid_network_of_scans_runs():
    from memory_bound_cnn_amd import hybrid
    assert all(math.isfinite(v) for v in hybrid.train(steps=3, log=None, scan=True))


# ------------------------------------------------------------------ the C functions
def test_c_functions_agree_with_the_operators():
    g = gen(11)
    cu = torch.tensor([0, 100, 260], dtype=torch.int32, device=DEV)
    x, gate, r, state = normal(g, 260, 24), normal(g, 260, 24), normal(g, 260, 24), normal(g, 2, 24)
    w, b = 1 + normal(g, 24, scale=0.1), normal(g, 24)
    leaves = [t.requires_grad_() for t in (x, w, b, r)]
    y, h = tokens.layer_norm(x, w, b, r)
    dy, dh = normal(g, 260, 24), normal(g, 260, 24)
    want = torch.autograd.grad((y, h), leaves, (dy, dh))
    with torch.no_grad():
        yc, hc, stats = tb.wtconv_layer_norm_forward(x, w, b, r, want_stats=True)
        dx, dw, db = tb.wtconv_layer_norm_backward(dy, dh, hc, w, stats)
    for a, c in zip((y, h) + want[:3], (yc, hc, dx, dw, db)):
        assert torch.equal(a, c)
    x, gate, state = (t.detach().requires_grad_() for t in (x, gate, state))
    for reverse in (False, True):
        y, last = tokens.gated_scan(x, gate, cu, state, reverse)
        dl = normal(g, 2, 24)
        want = torch.autograd.grad((y, last), (x, gate, state), (dy, dl))
        with torch.no_grad():
            yc, lc, kept = tb.wtconv_gated_scan_forward(x, gate, cu, state, reverse, want_kept=True)
            got = tb.wtconv_gated_scan_backward(dy, dl, x, gate, cu, state, kept, reverse)
        for a, c in zip((y, last) + want, (yc, lc) + got):
            assert torch.equal(a, c)
    with torch.no_grad():
        for a, c in zip(tokens.gated_scan_step(x[:2], gate[:2], state), tb.wtconv_gated_scan_step(x[:2], gate[:2], state)):
            assert torch.equal(a, c)
    experts = torch.randint(-1, 3, (130, 2), generator=g, device=DEV).int()
    order = tokens.expert_order(experts, 3)
    for a, c in zip(order, tb.wtconv_expert_order(experts, 3)):
        assert torch.equal(a, c)
    t, rows, wt = (v.requires_grad_() for v in (normal(g, 130, 24), normal(g, 260, 24), normal(g, 130, 2)))
    xs, y = tokens.expert_gather(t, order), tokens.expert_combine(rows, wt, order)
    dt, = torch.autograd.grad(xs, t, dy)
    dyt = normal(g, 130, 24)
    dr, dwt = torch.autograd.grad(y, (rows, wt), dyt)
    with torch.no_grad():
        assert torch.equal(xs, tb.wtconv_expert_gather(t, order.slot, order.cu_experts))
        assert torch.equal(y, tb.wtconv_expert_combine(rows, wt, order.slot))
        assert torch.equal(dt, tb.wtconv_expert_combine(dy, None, order.slot))
        for a, c in zip((dr, dwt), tb.wtconv_expert_combine_backward(dyt, rows, wt, order.slot, order.cu_experts)):
            assert torch.equal(a, c)
    W, B, dN = normal(g, 3, 40, 24).requires_grad_(), normal(g, 3, 40).requires_grad_(), normal(g, 260, 40)
    y = tokens.expert_linear(rows, W, order.cu_experts, B)
    want = torch.autograd.grad(y, (rows, W, B), dN)
    with torch.no_grad():
        assert torch.equal(y, tb.wtconv_expert_linear_forward(rows, W, order.cu_experts, B))
        assert torch.equal(want[0], tb.wtconv_expert_linear_input_grad(dN, W, order.cu_experts))
        for a, c in zip(want[1:], tb.wtconv_expert_linear_weight_grad(dN, rows, order.cu_experts)):
            assert torch.equal(a, c)
