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
