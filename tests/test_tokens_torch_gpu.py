"""The token operators inside PyTorch's own machinery: activation checkpointing,
captured graphs, forward-mode derivatives, traces."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from memory_bound_cnn_amd import tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


def block_and_input(**kw):
    torch.manual_seed(0)
    m = tokens.TokenBlock(64, 2, kv_heads=1, p=0.3, device=DEV, dtype=torch.float32, **kw)
    pos, cu = tokens.image_positions([(5, 7), (4, 9)], device=DEV)
    return m, torch.randn(71, 64, device=DEV), pos, cu


# ------------------------------------------------------------------ the block's dropout
@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpointed_block_has_the_blocks_gradients(reentrant):
    m, x, pos, cu = block_and_input()

    def gradients(call):
        torch.manual_seed(1)
        m.zero_grad()
        t = x.clone().requires_grad_()
        y = call(t)
        y.square().sum().backward()
        return [y.detach(), t.grad] + [p.grad.clone() for p in m.parameters()]

    want = gradients(lambda t: m(t, pos, cu))
    got = gradients(lambda t: checkpoint(m, t, pos, cu, use_reentrant=reentrant))
    assert not torch.equal(want[0], m.eval()(x, pos, cu))
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_block_in_a_graph_drops_other_elements_each_replay():
    """Dropout's words come from the generator in every replay; what is not
    dropped is the eager result of the same words."""
    m, x, pos, cu = block_and_input()
    seen = []
    call = tokens.dropout

    def watched(t, p, rng, residual=None):
        seen.append(rng)
        return call(t, p, rng, residual)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.no_grad():
        m(x, pos, cu)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    tokens.dropout = watched
    try:
        with torch.no_grad(), torch.cuda.graph(graph):
            out = m(x, pos, cu)
    finally:
        tokens.dropout = call
    assert len(seen) == 2
    keys = set()
    for i in range(3):
        x.copy_(torch.randn(71, 64, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        keys.add(int(seen[0][0]))
        words = iter(w.clone() for w in seen)
        try:
            tokens.dropout = lambda t, p, rng, residual=None: call(t, p, next(words), residual)
            with torch.no_grad():
                want = m(x, pos, cu)
        finally:
            tokens.dropout = call
        assert torch.equal(out, want)
    assert len(keys) == 3


# ------------------------------------------------------------------ forward-mode derivatives
def operator_calls():
    """{name: (call, its activations)}"""
    g = torch.Generator(device=DEV).manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    w, rng = 1 + 0.1 * n(32), torch.tensor([3, 4], device=DEV)
    pos, cu = tokens.image_positions([(3, 5), (4, 4)], device=DEV)
    f = tokens.rotary_frequencies((8, 8), device=DEV)
    return {
        "rms_norm": (lambda x, w: tokens.rms_norm(x, w), (n(31, 32), w)),
        "rms_norm residual": (lambda x, w, r: tokens.rms_norm(x, w, r), (n(31, 32), w, n(31, 32))),
        "rms_norm_fp8": (lambda x, w, r: tokens.rms_norm_fp8(x, w, r)[:2], (n(31, 32), w, n(31, 32))),
        "rotary": (lambda x: tokens.rotary(x, pos, f, (8, 8)), (n(31, 2, 32),)),
        "attention": (lambda q, k, v: tokens.attention(q, k, v, cu), (n(31, 4, 32), n(31, 2, 32), n(31, 2, 32))),
        "rotary_attention": (lambda x: tokens.rotary_attention(x, 4, 2, pos, f, (8, 8), cu), (n(31, 8, 32),)),
        "dropout": (lambda x: tokens.dropout(x, 0.5, rng), (n(31, 32),)),
        "dropout residual": (lambda x, r: tokens.dropout(x, 0.5, rng, r), (n(31, 32), n(31, 32))),
    }


CALLS = ["rms_norm", "rms_norm residual", "rms_norm_fp8", "rotary", "attention", "rotary_attention", "dropout",
         "dropout residual"]


@pytest.mark.parametrize("name", CALLS)
def test_forward_mode_derivatives_are_refused(name):
    """By every activation alone, whether it requires a gradient or not."""
    import torch.autograd.forward_ad as fwd
    call, args = operator_calls()[name]
    for i in range(len(args)):
        for requires in (False, True):
            with fwd.dual_level():
                a = [t.clone() for t in args]
                if requires and name != "rms_norm_fp8":
                    a[i].requires_grad_()
                a[i] = fwd.make_dual(a[i], torch.ones_like(a[i]))
                with pytest.raises(RuntimeError, match="forward-mode"):
                    call(*a)
    call(*args)


# ------------------------------------------------------------------ sizes
def test_sizes_beyond_32_bits_are_refused():
    """Not taken modulo 2^32: each of these would pass as a small one."""
    from memory_bound_cnn_amd import token_binding as tb
    big = (1 << 32) + 8
    x = torch.zeros(1, device=DEV, dtype=torch.bfloat16)
    w, f, cu = torch.ones(8, device=DEV), torch.ones(2, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    pos, cus = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV).expand(big)
    small = x.expand(1, 8, 8)
    for call in (lambda: tokens.rms_norm(x.expand(1, big), w), lambda: tokens.rms_norm_fp8(x.expand(1, big), w),
                 lambda: tokens.rotary(x.expand(1, big, 8), pos, f, (2,)),
                 lambda: tokens.rotary(x.expand(1, 8, big), pos, f, (2,)),
                 lambda: tokens.attention(x.expand(1, big, 8), small, small, cu),
                 lambda: tokens.attention(x.expand(1, 8, big), x.expand(1, 8, big), x.expand(1, 8, big), cu),
                 lambda: tokens.attention(small, small, small, cus),
                 lambda: tokens.rotary_attention(x.expand(1, big, 8), big - 4, 2, pos, f, (2,), cu),
                 lambda: tb.wtconv_rms_norm_forward(x.expand(1, big), w),
                 lambda: tb.wtconv_rotary(x.expand(1, big, 1), pos, f[:0], (0,)),
                 lambda: tb.wtconv_attention_forward(x.expand(1, big, 1), x.expand(1, 8, 1), x.expand(1, 8, 1), cu),
                 lambda: tb.wtconv_attention_forward(x.expand(1, 8, 1), x.expand(1, 8, 1), x.expand(1, 8, 1), cus)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


# ------------------------------------------------------------------ traces
def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def compare(got, want):
    assert len(flat(got)) == len(flat(want))
    for a, b in zip(flat(got), flat(want)):
        assert a.dtype == b.dtype and torch.equal(a.float(), b.float())


@pytest.mark.parametrize("name", CALLS)
def test_traced_functions_compute(name):
    """A TorchScript trace and a make_fx graph hold the operator: on other
    inputs they give what a call gives."""
    from torch.fx.experimental.proxy_tensor import make_fx
    call, args = operator_calls()[name]
    others = [t.flip(0) * 2 for t in args]
    want = call(*others)
    for traced in (torch.jit.trace(lambda *a: tuple(flat(call(*a))), args, check_trace=False),
                   make_fx(lambda *a: tuple(flat(call(*a))))(*args)):
        compare(call(*args), call(*args))     # memory that a trace must not find its answer in
        compare(traced(*others), want)


@pytest.mark.parametrize("name", [n for n in CALLS if n != "rms_norm_fp8"])
def test_traced_gradients_compute(name):
    """The gradient of a traced function, and a graph of a function that takes gradients."""
    from torch.fx.experimental.proxy_tensor import make_fx
    call, args = operator_calls()[name]
    others = [t.flip(0) * 2 for t in args]

    def gradients(f, a):
        a = [t.detach().requires_grad_() for t in a]
        return torch.autograd.grad(sum(t.float().square().sum() for t in flat(f(*a))), a)

    want = gradients(call, others)
    traced = torch.jit.trace(lambda *a: tuple(flat(call(*a))), args, check_trace=False)
    compare(gradients(traced, others), want)
    compare(make_fx(lambda *a: gradients(call, a))(*args)(*others), want)


def test_parts_of_a_gradient_check_their_arguments():
    """A graph may call them with any tensors."""
    tokens._load()
    o = torch.ops.wtconv_tokens
    x, w, s = torch.randn(5, 32, device=DEV), torch.ones(32, device=DEV), torch.ones(5, device=DEV)
    x3, cu, pos = x.view(5, 1, 32), torch.tensor([0, 5], dtype=torch.int32, device=DEV), torch.zeros(5, 1, dtype=torch.int32, device=DEV)
    f = tokens.rotary_frequencies((4,), device=DEV)
    kept = o._attention_forward(x3, x3, x3, cu, False, None)
    qkv, qk = x3.expand(5, 3, 32).contiguous(), x3.expand(5, 2, 32).contiguous()
    for call in (lambda: o._rms_norm_backward(x, None, x, w, s[:4]), lambda: o._rms_norm_backward(x[:4], None, x, w, s),
                 lambda: o._rms_norm_backward(x, x[:4], x, w, s), lambda: o._rms_norm_backward(x, None, x, w[:31], s),
                 lambda: o._rms_norm_backward(x.bfloat16(), None, x, w, s), lambda: o._rms_norm_backward(x.cpu(), None, x.cpu(), w, s),
                 lambda: o._rotary_backward(x3, pos[:4], f, (4,), False), lambda: o._rotary_backward(x3, pos, f, (17,), False),
                 lambda: o._attention_backward(x3, x3, x3, x3[:4], kept, cu, False, None),
                 lambda: o._attention_backward(x3[:4], x3, x3, x3, kept, cu, False, None),
                 lambda: o._attention_backward(x3, x3, x3, x3, [kept[0]], cu, False, None),
                 lambda: o._attention_backward(x3, x3, x3, x3, [kept[0][:4], kept[1]], cu, False, None),
                 lambda: o._attention_backward(x3, x3, x3, x3, [kept[0], kept[1][:, :4]], cu, False, None),
                 lambda: o._attention_backward(x3, x3, x3, x3, [*kept, x3], cu, False, None),
                 lambda: o._rotary_attention_backward(x3, qkv, qk[:, :1], kept, 1, 1, pos, f, (4,), cu, False, False, None),
                 lambda: o._rotary_attention_backward(x3, qkv[:, :2], qk, kept, 1, 1, pos, f, (4,), cu, False, False, None)):
        with pytest.raises(ValueError):
            call()
    dy = x.clone().requires_grad_()
    dx, _ = o._rms_norm_backward(dy, None, x, w, s)
    with pytest.raises(RuntimeError, match="not implemented"):
        dx.sum().backward()


def test_lazily_negated_inputs():
    """Memory that stands for its negative (as the imaginary part of a conjugate does)."""
    x, w = torch.randn(5, 32, device=DEV), torch.ones(32, device=DEV)
    assert torch.equal(tokens.rms_norm(torch._neg_view(x), w), tokens.rms_norm(-x, w))
    assert torch.equal(tokens.dropout(torch._neg_view(x), 0.0, torch.zeros(2, dtype=torch.int64, device=DEV)), -x)


@pytest.mark.parametrize("name", CALLS)
def test_function_transforms_compute_or_refuse(name):
    """vmap gives what a loop gives where it gives anything; grad and jvp of
    torch.func, which the gradients are not written for, raise."""
    call, args = operator_calls()[name]
    first = lambda *a: flat(call(*a))[0].float()
    try:
        got = torch.func.vmap(first)(*(torch.stack([a, a * 2]) for a in args))
    except RuntimeError:
        got = None
    for i in range(2 if got is not None else 0):
        assert torch.equal(got[i], first(*(a * (i + 1) for a in args)))
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.grad(lambda *a: first(*a).sum())(*args)
    with pytest.raises(RuntimeError, match="forward-mode"):
        torch.func.jvp(first, args, tuple(torch.ones_like(a) for a in args))


def test_float32_block_trains_under_autocast_and_a_converted_one_in_bfloat16():
    for convert, autocast, dtype in ((False, True, torch.float32), (True, False, torch.bfloat16)):
        m, x, pos, cu = block_and_input()
        if convert:
            m, x = m.to(torch.bfloat16), x.bfloat16()
        with torch.autocast("cuda", torch.bfloat16, enabled=autocast):
            y = m(x, pos, cu)
        assert y.dtype == dtype
        y.float().square().mean().backward()
        assert all(p.grad is not None and p.grad.dtype == p.dtype and torch.isfinite(p.grad).all() for p in m.parameters())
