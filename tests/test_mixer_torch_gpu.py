"""Layer norm, gated scan and experts inside PyTorch's own machinery: captured
graphs, checkpointing, traces, function transforms, derivatives that are refused,
sizes beyond 32 bits, and refusals of tensors."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from memory_bound_cnn_amd import token_binding as tb, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed=0):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def operator_calls():
    """{name: (call, its activations)}"""
    g = gen()
    n = lambda *s: normal(g, *s)
    cu = torch.tensor([0, 12, 12, 31], dtype=torch.int32, device=DEV)
    order = tokens.expert_order(torch.randint(-1, 4, (31, 2), generator=g, device=DEV).int(), 4)
    w = 1 + 0.1 * n(32)
    return {
        "layer_norm": (lambda x, w, b: tokens.layer_norm(x, w, b), (n(31, 32), w, n(32))),
        "layer_norm residual": (lambda x, w, r: tokens.layer_norm(x, w, None, r), (n(31, 32), w, n(31, 32))),
        "gated_scan": (lambda x, f: tokens.gated_scan(x, f, cu), (n(31, 32), n(31, 32))),
        "gated_scan state": (lambda x, f, s: tokens.gated_scan(x, f, cu, s, True), (n(31, 32), n(31, 32), n(3, 32))),
        "gated_scan_step": (lambda x, f, s: tokens.gated_scan_step(x, f, s), (n(31, 32), n(31, 32), n(31, 32))),
        "expert_gather": (lambda x: tokens.expert_gather(x, order), (n(31, 32),)),
        "expert_combine": (lambda r, w: tokens.expert_combine(r, w, order), (n(62, 32), n(31, 2))),
        "expert_linear": (lambda x, w, b: tokens.expert_linear(x, w, order.cu_experts, b), (n(62, 32), n(4, 40, 32), n(4, 40))),
    }


CALLS = ["layer_norm", "layer_norm residual", "gated_scan", "gated_scan state", "gated_scan_step", "expert_gather",
         "expert_combine", "expert_linear"]
WITH_GRADIENT = [n for n in CALLS if n != "gated_scan_step"]


def flat(r):
    return [t for t in (r if isinstance(r, (tuple, list)) else (r,)) if t is not None]


def compare(got, want):
    assert len(flat(got)) == len(flat(want))
    for a, b in zip(flat(got), flat(want)):
        assert a.dtype == b.dtype and torch.equal(a, b)


def gradients(call, args):
    a = [t.detach().requires_grad_() for t in args]
    return torch.autograd.grad(sum(t.float().square().sum() for t in flat(call(*a))), a)


# ------------------------------------------------------------------ graphs
def captured(step):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    return graph, out


@pytest.mark.parametrize("name", CALLS)
def test_operators_replay_in_a_graph(name):
    """Captured once, replayed with eager work and synchronizations between: each replay is the eager result, the
    gradients too."""
    call, args = operator_calls()[name]

    def step():
        if name == "gated_scan_step":
            return flat(call(*args))
        # leaves of the step's own: none of them lives on from an eager pass
        return flat(call(*args)) + list(gradients(call, args))
    graph, out = captured(step)
    for i in range(3):
        for t in args:
            t.copy_(normal(gen(10 + i), *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        compare(got, step())


@pytest.mark.parametrize("name", ["layer_norm", "gated_scan", "expert_linear"])
def test_a_backward_pass_is_not_captured_beside_an_eager_one(name):
    """Its leaves' gradients would belong to the default stream: refused, and captured once the eager pass is gone."""
    call, args = operator_calls()[name]
    leaves = [t.detach().requires_grad_() for t in args]

    def step():
        return torch.autograd.grad(sum(t.float().square().sum() for t in flat(call(*leaves))), leaves)
    want = [t.clone() for t in step()]
    eager = call(*leaves)
    with pytest.raises(RuntimeError, match="cannot be captured while an eager pass"):
        captured(step)
    torch.cuda.synchronize()
    del eager
    graph, out = captured(step)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        compare(out, want)


def behind_other_operators(name):
    """(module, call): leaves that reach the operators through others: a linear layer, casts, splits of a projection."""
    torch.manual_seed(0)
    x, cu = normal(gen(), 71, 64), torch.tensor([0, 35, 71], dtype=torch.int32, device=DEV)
    if name == "linear":
        m = torch.nn.Linear(64, 32, device=DEV)
        w = torch.ones(32, device=DEV)
        return m, lambda: tokens.layer_norm(m(x), w)
    m = tokens.ScanBlock(64, experts=4, device=DEV, dtype=torch.float32)

    def call():
        with torch.autocast("cuda", torch.bfloat16, enabled=name == "autocast block", cache_enabled=False):
            return m(x, cu)
    return m, call


BEHIND = pytest.mark.parametrize("name", ["linear", "block", "autocast block"])


@BEHIND
def test_leaves_of_the_default_stream_are_found(name):
    m, call = behind_other_operators(name)
    meets, s = tokens._load()._meets_default_stream, torch.cuda.Stream()

    def aside():
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = call()
        torch.cuda.current_stream().wait_stream(s)
        return y
    assert not meets(aside())
    eager = call()
    assert meets(eager) and meets(aside())      # the leaves are the eager pass's as long as that lives
    del eager
    assert not meets(aside())
    with torch.no_grad():
        assert not meets(call())


@BEHIND
def test_a_backward_pass_behind_others_is_not_captured_beside_an_eager_one(name):
    m, call = behind_other_operators(name)
    leaves = list(m.parameters())

    def step():
        return torch.autograd.grad(call().float().square().sum(), leaves)
    want = [t.clone() for t in step()]
    eager = call()
    assert tokens._load()._meets_default_stream(eager)
    with pytest.raises(RuntimeError, match="cannot be captured while an eager pass"):
        captured(step)
    torch.cuda.synchronize()
    del eager
    graph, out = captured(step)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        compare(out, want)


def test_a_captured_pass_is_refused_for_what_it_runs_through_alone():
    """An eager pass of leaves whose gradients are not asked for does not matter."""
    m, call = behind_other_operators("linear")
    b = torch.zeros(32, device=DEV)

    def step():
        mine = b.detach().requires_grad_()
        y = tokens.layer_norm(call(), torch.ones(32, device=DEV), mine)
        return torch.autograd.grad(y.square().sum(), (mine,))
    want = [t.clone() for t in step()]
    eager = call()
    graph, out = captured(step)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        compare(out, want)
    assert eager.isfinite().all()


def test_larger_packs_replay_in_a_graph():
    """What has workspaces: scans of several parts, orders of several workgroups, weights' gradients of several splits;
    two graphs of the same work replayed in turn."""
    g = gen(3)
    cu = torch.tensor([0, 1500, 1500, 4000], dtype=torch.int32, device=DEV)
    x, f = normal(g, 4000, 40), normal(g, 4000, 40)
    experts = torch.randint(-1, 6, (9000, 1), generator=g, device=DEV).int()
    rows, W = normal(g, 9000, 64, dtype=torch.bfloat16), normal(g, 6, 64, 64, dtype=torch.bfloat16)

    def step():
        order = tokens.expert_order(experts, 6)
        call = lambda r, w: tokens.expert_linear(r, w, order.cu_experts)
        scan = lambda a, b: tokens.gated_scan(a, b, cu)
        return list(order) + flat(call(rows, W)) + list(gradients(call, (rows, W))) + flat(scan(x, f)) + list(gradients(scan, (x, f)))
    one, a = captured(step)
    two, b = captured(step)
    for i in range(3):
        x.copy_(normal(gen(20 + i), 4000, 40))
        experts.copy_(torch.randint(-1, 6, (9000, 1), generator=gen(i), device=DEV).int())
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        want = step()
        compare(a, want)
        compare(b, want)


def test_steps_in_a_graph_go_on():
    """The state updated in place by every replay."""
    g = gen(5)
    m = tokens.ScanBlock(32, experts=4, causal=True, device=DEV, dtype=torch.float32)
    x, state = normal(g, 6, 32), torch.zeros(6, 32, device=DEV)
    with torch.no_grad():
        graph, out = captured(lambda: m.step(x, state)[0])
    state.zero_()
    mine = torch.zeros(6, 32, device=DEV)
    for i in range(4):
        x.copy_(normal(gen(30 + i), 6, 32))
        graph.replay()
        torch.cuda.synchronize()
        want, mine = m.step(x, mine)
        assert torch.equal(out, want) and torch.equal(state, mine)


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpointed_block_has_the_blocks_gradients(reentrant):
    torch.manual_seed(0)
    m = tokens.ScanBlock(64, experts=4, device=DEV, dtype=torch.float32)
    cu = torch.tensor([0, 35, 71], dtype=torch.int32, device=DEV)
    x = torch.randn(71, 64, device=DEV)

    def run(call):
        m.zero_grad()
        t = x.clone().requires_grad_()
        y = call(t)
        y.square().sum().backward()
        return [y.detach(), t.grad] + [p.grad.clone() for p in m.parameters()]
    compare(run(lambda t: checkpoint(m, t, cu, use_reentrant=reentrant)), run(lambda t: m(t, cu)))


# ------------------------------------------------------------------ derivatives that are not there
@pytest.mark.parametrize("name", CALLS)
def test_forward_mode_derivatives_are_refused(name):
    import torch.autograd.forward_ad as fwd
    call, args = operator_calls()[name]
    for i in range(len(args)):
        with fwd.dual_level():
            a = [t.clone() for t in args]
            a[i] = fwd.make_dual(a[i], torch.ones_like(a[i]))
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(*a)
    call(*args)


@pytest.mark.parametrize("name", WITH_GRADIENT)
def test_second_derivatives_are_refused(name):
    call, args = operator_calls()[name]
    a = [t.detach().requires_grad_() for t in args]
    out = [t for t in flat(call(*a))]
    g = [torch.ones_like(t).requires_grad_() for t in out]
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(out, a, g, create_graph=True)


def test_step_refuses_gradients_and_overlaps():
    x, s = normal(gen(), 4, 8), normal(gen(1), 4, 8)
    with pytest.raises(ValueError, match="no gradient"):
        tokens.gated_scan_step(x.requires_grad_(), x, s)
    x = x.detach()
    long = torch.zeros(40, device=DEV)
    with pytest.raises(RuntimeError, match="memory"):
        tokens.gated_scan_step(x, x, long[:32].view(4, 8), out=long[8:].view(4, 8))


def test_step_into_its_inputs():
    """The new state may replace an input of its type as a whole, not a part of one."""
    x, gate, state = normal(gen(), 4, 8), normal(gen(1), 4, 8), normal(gen(2), 4, 8)
    y, new = tokens.gated_scan_step(x, gate, state)
    for i in range(3):
        args = [x.clone(), gate.clone(), state.clone()]
        again, out = tokens.gated_scan_step(*args, out=args[i])
        assert torch.equal(again, y) and torch.equal(out, new) and out.data_ptr() == args[i].data_ptr()
    long = torch.zeros(40, device=DEV)
    for args in ((long[:32].view(4, 8), gate), (x, long[:32].view(4, 8))):
        with pytest.raises(RuntimeError, match="memory"):
            tokens.gated_scan_step(*args, state, out=long[8:].view(4, 8))


def test_step_into_memory_between_rows():
    """The new state may lie before, behind or between the rows of an input, which are apart, but not in one of them."""
    n, C, apart = 4, 8, 40                                     # a state is 32 long, as are the gaps between rows
    want = tokens.gated_scan_step(normal(gen(), n, C), normal(gen(1), n, C), normal(gen(2), n, C))
    for at in range(0, 32 + 4 * apart):
        long = torch.zeros(32 + 4 * apart + 32, device=DEV)
        x = long[32:32 + 4 * apart].view(n, apart)[:, :C]      # rows at 32, 72, 112, 152
        x.copy_(normal(gen(), n, C))
        out = long[at:at + 32].view(n, C)
        meets = any(at < r + C and r < at + 32 for r in (32, 72, 112, 152))
        for args in ((x, normal(gen(1), n, C)), (normal(gen(), n, C), x)):
            if meets:
                with pytest.raises(RuntimeError, match="memory"):
                    tokens.gated_scan_step(*args, normal(gen(2), n, C), out=out)
        if not meets:
            y, new = tokens.gated_scan_step(x, normal(gen(1), n, C), normal(gen(2), n, C), out=out)
            assert torch.equal(y, want[0]) and torch.equal(out, want[1]) and torch.equal(x, normal(gen(), n, C))
    row = torch.zeros(64, device=DEV)
    with pytest.raises(RuntimeError, match="memory"):          # one row for all
        tokens.gated_scan_step(row[20:28].expand(n, C), row[:8].expand(n, C), normal(gen(2), n, C), out=row[:32].view(n, C))


def test_step_in_place_is_seen_by_autograd():
    """A state that is saved for a gradient and then overwritten is an error, not a wrong gradient."""
    s = normal(gen(), 4, 8)
    w = torch.ones(4, 8, device=DEV, requires_grad=True)
    y = w * s
    with torch.no_grad():
        tokens.gated_scan_step(s.clone(), s.clone(), s, out=s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


# ------------------------------------------------------------------ traces
@pytest.mark.parametrize("name", CALLS)
def test_traced_functions_compute(name):
    from torch.fx.experimental.proxy_tensor import make_fx
    call, args = operator_calls()[name]
    others = [t.flip(0) * 2 for t in args]
    want = call(*others)
    for traced in (torch.jit.trace(lambda *a: tuple(flat(call(*a))), args, check_trace=False),
                   make_fx(lambda *a: tuple(flat(call(*a))))(*args)):
        compare(call(*args), call(*args))     # memory that a trace must not find its answer in
        compare(traced(*others), want)


def test_traced_order_computes():
    from torch.fx.experimental.proxy_tensor import make_fx
    a, b = (torch.randint(-1, 4, (50, 2), generator=gen(i), device=DEV).int() for i in range(2))
    for traced in (torch.jit.trace(lambda e: tuple(tokens.expert_order(e, 4)), (a,), check_trace=False),
                   make_fx(lambda e: tuple(tokens.expert_order(e, 4)))(a)):
        compare(traced(b), tuple(tokens.expert_order(b, 4)))


@pytest.mark.parametrize("name", WITH_GRADIENT)
def test_traced_gradients_compute(name):
    from torch.fx.experimental.proxy_tensor import make_fx
    call, args = operator_calls()[name]
    others = [t.flip(0) * 2 for t in args]
    want = gradients(call, others)
    traced = torch.jit.trace(lambda *a: tuple(flat(call(*a))), args, check_trace=False)
    compare(gradients(traced, others), want)
    compare(make_fx(lambda *a: gradients(call, a))(*args)(*others), want)


@pytest.mark.parametrize("name", CALLS)
def test_function_transforms_compute_or_refuse(name):
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


# ------------------------------------------------------------------ refusals
def test_sizes_beyond_32_bits_are_refused():
    big = (1 << 32) + 8
    x, w = torch.zeros(1, device=DEV, dtype=torch.bfloat16), torch.ones(8, device=DEV)
    one = torch.zeros(1, device=DEV, dtype=torch.int32)
    cus = one.expand(big)
    for call in (lambda: tokens.layer_norm(x.expand(1, big), w), lambda: tokens.gated_scan(x.expand(1, big), x.expand(1, big), cus[:2]),
                 lambda: tokens.gated_scan(x.expand(1, 8), x.expand(1, 8), cus),
                 lambda: tokens.gated_scan_step(x.expand(1, big), x.expand(1, big), w[:1].expand(1, big), out=w[:1].expand(1, big)),
                 lambda: tokens.expert_order(one.view(1, 1), big), lambda: tb.wtconv_expert_order(one.view(1, 1), big),
                 lambda: tb.wtconv_layer_norm_forward(x.expand(1, big), w),
                 lambda: tb.wtconv_gated_scan_forward(x.expand(1, 8), x.expand(1, 8), cus)):
        with pytest.raises((ValueError, RuntimeError), match="32 bits|contiguous|overlap|memory"):
            call()


def test_entry_points_refuse():
    x, w, cu = torch.zeros(6, 16, device=DEV), torch.ones(16, device=DEV), torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    half, host = x.half(), torch.zeros(6, 16)
    order = tokens.expert_order(torch.zeros(3, 2, dtype=torch.int32, device=DEV), 4)
    W = torch.zeros(4, 24, 16, device=DEV)
    for call in (lambda: tokens.layer_norm(half, w), lambda: tokens.layer_norm(x, w[:8]), lambda: tokens.layer_norm(x, w.bfloat16()),
                 lambda: tokens.layer_norm(x, w, w[:8]), lambda: tokens.layer_norm(x, w, residual=x[:3]),
                 lambda: tokens.layer_norm(x, w, residual=x.bfloat16()), lambda: tokens.layer_norm(x, host[0]),
                 lambda: tokens.gated_scan(half, half, cu), lambda: tokens.gated_scan(x, x[:, :8], cu), lambda: tokens.gated_scan(x, x.bfloat16(), cu),
                 lambda: tokens.gated_scan(x, x, cu.long()), lambda: tokens.gated_scan(x, x, cu.cpu()), lambda: tokens.gated_scan(x, x, cu[:0]),
                 lambda: tokens.gated_scan(x, x, cu, x), lambda: tokens.gated_scan(x, x, cu, x[:1].bfloat16()),
                 lambda: tokens.gated_scan(x[0], x[0], cu),
                 lambda: tokens.gated_scan_step(x, x, x[:3]), lambda: tokens.gated_scan_step(x, x, x, out=x.bfloat16()),
                 lambda: tokens.expert_order(order.slot.long(), 4), lambda: tokens.expert_order(order.pair, 4),
                 lambda: tokens.expert_order(order.slot[:, :0], 4),
                 lambda: tokens.expert_gather(x, order), lambda: tokens.expert_gather(x[:3].half(), order),
                 lambda: tokens.expert_gather(x[:3], order._replace(cu_experts=order.cu_experts.long())),
                 lambda: tokens.expert_gather(x[:3], order._replace(slot=order.slot.cpu())),
                 lambda: tokens.expert_combine(x[:5], torch.ones(3, 2, device=DEV), order),
                 lambda: tokens.expert_combine(x, torch.ones(2, 3, device=DEV), order),
                 lambda: tokens.expert_combine(x, torch.ones(3, 2, device=DEV).bfloat16(), order),
                 lambda: tokens.expert_linear(x, W[:3], order.cu_experts), lambda: tokens.expert_linear(x, W[..., :8], order.cu_experts),
                 lambda: tokens.expert_linear(x, W.bfloat16(), order.cu_experts), lambda: tokens.expert_linear(x, W[0], order.cu_experts),
                 lambda: tokens.expert_linear(x, W, order.cu_experts, w), lambda: tokens.expert_linear(x, W, order.cu_experts.long()),
                 lambda: tokens.expert_linear(x, W.transpose(1, 2).contiguous().transpose(1, 2), order.cu_experts)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tokens.expert_order(order.slot, 0), lambda: tokens.expert_order(order.slot, 513),
                 lambda: tokens.layer_norm(x, w, eps=-1.0),
                 lambda: tokens.expert_linear(x[:, :12].contiguous(), W[..., :12].contiguous(), order.cu_experts)):
        with pytest.raises(RuntimeError, match="status"):
            call()


def test_parts_of_a_gradient_check_their_arguments():
    """A graph may call them with any tensors."""
    tokens._load()
    o = torch.ops.wtconv_tokens
    g = gen()
    x, w, cu = normal(g, 6, 16), torch.ones(16, device=DEV), torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    stats = torch.ones(6, 2, device=DEV)
    kept = o._gated_scan_forward(x, x, cu, None, False)[2]
    order = tokens.expert_order(torch.zeros(3, 2, dtype=torch.int32, device=DEV), 2)
    wt, W = torch.ones(3, 2, device=DEV), torch.zeros(2, 24, 16, device=DEV)
    for call in (lambda: o._layer_norm_backward(x, None, x, w, stats[:5], True), lambda: o._layer_norm_backward(x[:5], None, x, w, stats, True),
                 lambda: o._layer_norm_backward(x, x[:5], x, w, stats, True), lambda: o._layer_norm_backward(x, None, x, w[:8], stats, True),
                 lambda: o._gated_scan_backward(x[:5], None, x, x, cu, None, kept, False),
                 lambda: o._gated_scan_backward(x, x, x, x, cu, None, kept, False),
                 lambda: o._gated_scan_backward(x, None, x, x, cu, None, kept[:8], False),
                 lambda: o._gated_scan_backward(x, None, x, x, cu, x, kept, False),
                 lambda: o._expert_sum(x[:5], None, order.slot), lambda: o._expert_sum(x, wt[:2], order.slot),
                 lambda: o._expert_combine_backward(x, x, wt, order.slot, order.cu_experts),
                 lambda: o._expert_combine_backward(x[:3], x[:5], wt, order.slot, order.cu_experts),
                 lambda: o._expert_combine_backward(x[:3], x, wt.t(), order.slot, order.cu_experts),
                 lambda: o._expert_linear_input_grad(x, W, order.cu_experts), lambda: o._expert_linear_input_grad(x, W[:1], order.cu_experts),
                 lambda: o._expert_linear_weight_grad(x[:5], x, order.cu_experts, True),
                 lambda: o._expert_linear_weight_grad(x.bfloat16(), x, order.cu_experts, True)):
        with pytest.raises(ValueError):
            call()
    dy = x.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="not implemented"):
        o._layer_norm_backward(dy, None, x, w, stats, True)[0].sum().backward()


def test_lazily_negated_inputs():
    """Memory that stands for its negative (as the imaginary part of a conjugate does)."""
    g = gen()
    x, w, cu = normal(g, 5, 32), torch.ones(32, device=DEV), torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    assert torch.equal(tokens.layer_norm(torch._neg_view(x), w), tokens.layer_norm(-x, w))
    assert torch.equal(tokens.gated_scan(torch._neg_view(x), x, cu)[0], tokens.gated_scan(-x, x, cu)[0])
    W = normal(g, 1, 8, 32)
    assert torch.equal(tokens.expert_linear(torch._neg_view(x), W, cu), tokens.expert_linear(-x, W, cu))


def test_unwanted_gradients_are_not_computed_and_inference_mode_runs():
    g = gen()
    x, W, b = normal(g, 9, 16), normal(g, 1, 8, 16), normal(g, 1, 8)
    cu = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    full = gradients(lambda x, W, b: tokens.expert_linear(x, W, cu, b), (x, W, b))
    for which in range(3):
        a = [t.clone().requires_grad_(i == which) for i, t in enumerate((x, W, b))]
        got, = torch.autograd.grad(tokens.expert_linear(a[0], a[1], cu, a[2]).square().sum(), a[which])
        assert torch.equal(got, full[which])
    with torch.inference_mode():
        s = torch.zeros(9, 16, device=DEV)
        y, out = tokens.gated_scan_step(x, x, s, out=s)
        assert torch.equal(out, tokens.gated_scan_step(x, x, torch.zeros(9, 16, device=DEV))[1])
        assert tokens.expert_linear(x, W, cu, b).shape == (9, 8)


def test_float32_block_trains_under_autocast_and_a_converted_one_in_bfloat16():
    cu = torch.tensor([0, 35, 71], dtype=torch.int32, device=DEV)
    for convert, autocast, dtype in ((False, True, torch.float32), (True, False, torch.bfloat16)):
        torch.manual_seed(0)
        m, x = tokens.ScanBlock(64, experts=4, device=DEV, dtype=torch.float32), torch.randn(71, 64, device=DEV)
        if convert:
            m, x = m.to(torch.bfloat16), x.bfloat16()
        with torch.autocast("cuda", torch.bfloat16, enabled=autocast):
            y = m(x, cu)
        assert y.dtype == dtype
        y.float().square().mean().backward()
        assert all(p.grad is not None and p.grad.dtype == p.dtype and torch.isfinite(p.grad).all() for p in m.parameters())
