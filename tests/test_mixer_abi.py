"""Layer norm, gated scan and experts without a GPU: bad arguments are refused
before any HIP call, and the Python entry points refuse tensors they cannot take."""

import ctypes

import pytest
import torch

from memory_bound_cnn_amd import binding, token_binding as tb, tokens

P = ctypes.c_void_p(4096)    # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(4100)  # 4-byte aligned alone
EINVAL, ESHAPE, EDTYPE, EWORKSPACE = binding.WTC_EINVAL, binding.WTC_ESHAPE, binding.WTC_EDTYPE, binding.WTC_EWORKSPACE
OK = binding.WTC_OK


def ref(d):
    return ctypes.addressof(d)


def desc(cls, defaults, **kw):
    assert set(kw) <= set(defaults)
    return cls(*{**defaults, **kw}.values())


def layer(**kw):
    return desc(tb.wtc_layer_desc, dict(rows=3, x_stride=8, r_stride=8, g_stride=8, C=8, dtype=0, eps=1e-6), **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(C=0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(x_stride=-8), EINVAL), (dict(g_stride=-1), EINVAL), (dict(dtype=2), EDTYPE),
    (dict(C=tb.RMS_MAX_C + 1), ESHAPE), (dict(rows=1 << 31), ESHAPE),
])
def test_layer_norm_rejects_descriptors(kw, status):
    lib, d = tb._load(), layer(**kw)
    assert lib.wtconv_layer_norm_forward(ref(d), P, P, P, P, P, P, P, None) == status
    assert lib.wtconv_layer_norm_backward(ref(d), P, P, P, P, P, P, P, P, P, 1 << 40, None) == status
    assert lib.wtconv_layer_norm_backward_workspace(ref(d)) == 0


def test_layer_norm_rejects_pointers():
    lib, d = tb._load(), layer()
    f, b = lib.wtconv_layer_norm_forward, lib.wtconv_layer_norm_backward
    assert f(None, P, None, P, P, P, None, None, None) == EINVAL
    for at in (0, 2, 4):
        args = [P, None, P, P, P, None, None]
        args[at] = None
        assert f(ref(d), *args, None) == EINVAL
    assert f(ref(d), P, P, P, P, P, None, None, None) == EINVAL        # a residual without h
    assert f(ref(d), P, None, P, P, P, P, None, None) == EINVAL        # h without a residual
    assert f(ref(d), P, None, P, P, P, None, ODD, None) == EINVAL      # stats are pairs
    need = lib.wtconv_layer_norm_backward_workspace(ref(d))
    assert need == 2 * 4 * d.C
    for at in (0, 2, 3, 4, 5, 6):
        args = [P] * 8
        args[at] = None
        assert b(ref(d), *args, P, need, None) == EINVAL
    assert b(ref(d), *[P] * 8, P, need - 1, None) == EWORKSPACE
    assert b(ref(d), *[P] * 8, None, need, None) == EWORKSPACE
    assert f(ref(layer(rows=0)), *[None] * 8) == OK


def scan(**kw):
    return desc(tb.wtc_scan_desc, dict(T=200, x_stride=8, f_stride=8, g_stride=8, n_seq=2, C=8, dtype=1, reverse=0), **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), EINVAL), (dict(n_seq=-1), EINVAL), (dict(C=0), EINVAL), (dict(reverse=2), EINVAL), (dict(f_stride=-8), EINVAL),
    (dict(dtype=3), EDTYPE), (dict(C=(1 << 20) + 1), ESHAPE), (dict(T=(1 << 31) - (1 << 10)), ESHAPE), (dict(n_seq=(1 << 24) + 1), ESHAPE),
])
def test_gated_scan_rejects_descriptors(kw, status):
    lib, d = tb._load(), scan(**kw)
    assert lib.wtconv_gated_scan_forward(ref(d), *[P] * 8, 1 << 40, None) == status
    assert lib.wtconv_gated_scan_backward(ref(d), *[P] * 11, 1 << 40, None) == status
    assert lib.wtconv_gated_scan_step(ref(d), *[P] * 5, None) == status
    assert lib.wtconv_gated_scan_workspace(ref(d)) == lib.wtconv_gated_scan_kept(ref(d)) == 0


def test_gated_scan_rejects_pointers_and_workspaces():
    lib, d = tb._load(), scan()
    f, b, s = lib.wtconv_gated_scan_forward, lib.wtconv_gated_scan_backward, lib.wtconv_gated_scan_step
    need = lib.wtconv_gated_scan_workspace(ref(d))
    assert need > 0 and lib.wtconv_gated_scan_kept(ref(d)) == 25 * 8 * 4        # the state of every 8th token
    assert lib.wtconv_gated_scan_workspace(ref(scan(T=64))) == 0
    assert f(None, *[P] * 8, need, None) == EINVAL
    for at in (0, 1, 2, 4):
        args = [P] * 7
        args[at] = None
        assert f(ref(d), *args, P, need, None) == EINVAL
    assert f(ref(d), *[P] * 7, P, need - 1, None) == EWORKSPACE and f(ref(d), *[P] * 7, None, need, None) == EWORKSPACE
    assert f(ref(d), *[P] * 7, ODD, need, None) == EINVAL
    for at in (0, 1, 2, 4, 5, 7, 8):
        args = [P] * 10
        args[at] = None
        assert b(ref(d), *args, P, need, None) == EINVAL
    assert b(ref(d), *[P] * 10, P, need - 1, None) == EWORKSPACE
    for at in range(5):
        args = [P] * 5
        args[at] = None
        assert s(ref(d), *args, None) == EINVAL
    assert f(ref(scan(T=0, n_seq=0)), *[None] * 8, 0, None) == OK and s(ref(scan(T=0)), *[None] * 6) == OK


def test_expert_order_rejects():
    lib = tb._load()
    f, need = lib.wtconv_expert_order, lib.wtconv_expert_order_workspace(20000, 8)
    assert need > 0 and lib.wtconv_expert_order_workspace(100, 8) == 0
    for n, E, status in ((-1, 8, EINVAL), (10, 0, EINVAL), (10, -1, EINVAL), (10, tb.EXPERTS_MAX + 1, ESHAPE),
                         ((1 << 31) - (1 << 16), 8, ESHAPE)):
        assert f(n, E, P, P, P, P, P, 1 << 40, None) == status and lib.wtconv_expert_order_workspace(n, E) == 0
    for at in range(4):
        args = [P] * 4
        args[at] = None
        assert f(10, 8, *args, None, 0, None) == EINVAL
    assert f(20000, 8, P, P, P, P, P, need - 1, None) == EWORKSPACE and f(20000, 8, P, P, P, P, None, need, None) == EWORKSPACE
    assert f(20000, 8, P, P, P, P, ODD, need, None) == EINVAL


def rows(**kw):
    return desc(tb.wtc_rows_desc, dict(T=10, x_stride=8, r_stride=8, k=2, E=4, C=8, dtype=0), **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(C=0), EINVAL), (dict(E=0), EINVAL), (dict(x_stride=-1), EINVAL),
    (dict(r_stride=-1), EINVAL), (dict(dtype=7), EDTYPE), (dict(C=65537), ESHAPE), (dict(E=tb.EXPERTS_MAX + 1), ESHAPE),
    (dict(T=1 << 30), ESHAPE), (dict(T=1 << 31, k=1), ESHAPE), (dict(T=1 << 30, k=1, C=64), ESHAPE),
])
def test_expert_rows_reject_descriptors(kw, status):
    lib, d = tb._load(), rows(**kw)
    assert lib.wtconv_expert_gather(ref(d), P, P, P, P, None) == status
    assert lib.wtconv_expert_combine(ref(d), P, P, P, P, None) == status
    assert lib.wtconv_expert_combine_backward(ref(d), *[P] * 7, None) == status


def test_expert_rows_reject_pointers():
    lib, d = tb._load(), rows()
    for f, args, needed in ((lib.wtconv_expert_gather, 4, range(4)), (lib.wtconv_expert_combine, 4, (0, 2, 3)),
                            (lib.wtconv_expert_combine_backward, 7, range(7))):
        for at in needed:
            a = [P] * args
            a[at] = None
            assert f(ref(d), *a, None) == EINVAL
        assert f(None, *[P] * args, None) == EINVAL
        assert f(ref(rows(T=0)), *[None] * args, None) == OK


def expert(**kw):
    return desc(tb.wtc_expert_desc, dict(R=10, x_stride=16, g_stride=24, E=2, K=16, N=24, dtype=1), **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), EINVAL), (dict(E=0), EINVAL), (dict(K=0), EINVAL), (dict(N=-8), EINVAL), (dict(dtype=4), EDTYPE),
    (dict(K=12), ESHAPE), (dict(N=20), ESHAPE), (dict(K=65544), ESHAPE), (dict(N=65544), ESHAPE),
    (dict(E=tb.EXPERTS_MAX + 1), ESHAPE), (dict(R=1 << 31), ESHAPE), (dict(x_stride=20, g_stride=20), EINVAL),
    (dict(x_stride=-16, g_stride=-16), EINVAL), (dict(x_stride=(1 << 22) + 8, g_stride=(1 << 22) + 8), ESHAPE),
])
def test_expert_linear_rejects_descriptors(kw, status):
    lib, d = tb._load(), expert(**kw)
    assert lib.wtconv_expert_linear_forward(ref(d), P, P, P, P, P, None) == status
    assert lib.wtconv_expert_linear_input_grad(ref(d), P, P, P, P, None) == status
    assert lib.wtconv_expert_linear_weight_grad(ref(d), *[P] * 6, 1 << 40, None) == status


def test_expert_linear_rejects_pointers_and_workspaces():
    lib, d = tb._load(), expert()
    for f, args, needed, wide in ((lib.wtconv_expert_linear_forward, 5, (0, 1, 3, 4), (0, 1, 2, 4)),
                                  (lib.wtconv_expert_linear_input_grad, 4, range(4), (0, 1, 3))):
        for at in needed:
            a = [P] * args
            a[at] = None
            assert f(ref(d), *a, None) == EINVAL
        for at in wide:      # 16-byte aligned; cu_experts is int32
            a = [P] * args
            a[at] = ODD
            assert f(ref(d), *a, None) == EINVAL
        assert f(None, *[P] * args, None) == EINVAL
        assert f(ref(expert(R=0)), *[None] * args, None) == OK
    f = lib.wtconv_expert_linear_weight_grad
    for at in (0, 1, 2, 3):
        a = [P] * 5
        a[at] = None
        assert f(ref(d), *a, None, 0, None) == EINVAL
    for at in (0, 1, 3, 4):
        a = [P] * 5
        a[at] = ODD
        assert f(ref(d), *a, None, 0, None) == EINVAL
    many = expert(R=100000, E=1)       # few tiles of dW, many rows: shared by workgroups, whose sums need a place
    need = lib.wtconv_expert_linear_weight_grad_workspace(ref(many))
    assert need > 0 and lib.wtconv_expert_linear_weight_grad_workspace(ref(d)) == 0
    assert f(ref(many), *[P] * 5, P, need - 1, None) == EWORKSPACE and f(ref(many), *[P] * 5, None, need, None) == EWORKSPACE
    assert f(ref(many), *[P] * 5, ODD, need, None) == EINVAL


def test_python_entry_points_refuse_host_tensors():
    x, w, cu = torch.zeros(4, 16), torch.ones(16), torch.tensor([0, 4], dtype=torch.int32)
    order = tokens.ExpertOrder(torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), cu)
    for call in (lambda: tokens.layer_norm(x, w), lambda: tokens.gated_scan(x, x, cu), lambda: tokens.gated_scan_step(x, x, x),
                 lambda: tokens.expert_order(order.slot, 1), lambda: tokens.expert_gather(x, order),
                 lambda: tokens.expert_combine(x, torch.ones(4, 1), order), lambda: tokens.expert_linear(x, w.view(1, 1, 16), cu),
                 lambda: tb.wtconv_layer_norm_forward(x, w), lambda: tb.wtconv_gated_scan_forward(x, x, cu),
                 lambda: tb.wtconv_gated_scan_step(x, x, x), lambda: tb.wtconv_expert_order(order.slot, 1),
                 lambda: tb.wtconv_expert_gather(x, order.slot, cu), lambda: tb.wtconv_expert_combine(x, None, order.slot),
                 lambda: tb.wtconv_expert_linear_forward(x, w.view(1, 1, 16), cu),
                 lambda: tb.wtconv_expert_linear_weight_grad(x, x, cu)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="residual has shape"):
        tokens.layer_norm(x, w, residual=x[:3])


def test_modules_refuse_and_keep_their_norms():
    with pytest.raises(ValueError, match="experts a token"):
        tokens.Experts(8, 16, 2, k=3)
    with pytest.raises(ValueError, match="directions"):
        tokens.ScanBlock(9)
    m = tokens.ScanBlock(8, experts=2, dtype=torch.float32)
    with torch.no_grad():
        m.norm1.bias.add_(0.1)
    m.to(torch.bfloat16)
    assert m.norm1.weight.dtype == m.norm1.bias.dtype == torch.float32 and m.experts.up.dtype == m.values.weight.dtype == torch.bfloat16
    assert torch.equal(m.norm1.bias, torch.full((8,), 0.1))
    assert tokens.LayerNorm(8, bias=False).bias is None


@pytest.mark.parametrize("make", [lambda: tokens.Experts(100, 64, 2), lambda: tokens.Experts(64, 100, 2), lambda: tokens.ScanBlock(100),
                                  lambda: tokens.ScanBlock(9, causal=True), lambda: tokens.ScanBlock(64, hidden=36)])
def test_modules_refuse_sizes_that_their_products_do_not_take(make):
    with pytest.raises(ValueError, match="multiples of 8"):
        make()
    with pytest.raises(ValueError, match="up to 512"):
        tokens.Experts(8, 8, tb.EXPERTS_MAX + 1)


@pytest.fixture
def plain(monkeypatch):
    """The operators that the modules call, in plain PyTorch."""
    def layer_norm(x, weight, bias=None, residual=None, eps=1e-6):
        assert weight.dtype == torch.float32 and (residual is None or residual.dtype == x.dtype)
        h = x if residual is None else x + residual
        y = torch.nn.functional.layer_norm(h.float(), h.shape[-1:], weight, bias, eps).to(h.dtype)
        return y if residual is None else (y, h)

    def gated_scan(x, gate, cu, state=None, reverse=False):
        a, out = torch.sigmoid(gate.float()), []
        for s, e in zip(cu[:-1].tolist(), cu[1:].tolist()):
            h, part = torch.zeros(x.shape[1]), []
            for t in reversed(range(s, e)) if reverse else range(s, e):
                h = a[t] * h + (1 - a[t]) * x[t].float()
                part.append(h)
            out += reversed(part) if reverse else part
        return torch.stack(out).to(x.dtype), None

    def expert_order(experts, n):
        e = experts.reshape(-1)
        pair = torch.argsort(e, stable=True)
        slot = torch.empty_like(pair)
        slot[pair] = torch.arange(e.numel())
        return tokens.ExpertOrder(slot.view(experts.shape), pair, torch.bincount(e, minlength=n).cumsum(0))

    def expert_linear(x, w, cu, bias=None):
        assert x.dtype == w.dtype
        at = [0] + cu.tolist()
        return torch.cat([x[at[e]:at[e + 1]] @ w[e].T + bias[e] for e in range(len(w))])

    plain = dict(layer_norm=layer_norm, gated_scan=gated_scan, expert_order=expert_order, expert_linear=expert_linear,
                 expert_gather=lambda x, o: x[o.pair // o.slot.shape[1]],
                 expert_combine=lambda r, w, o: (r[o.slot].float() * w[..., None]).sum(1).to(r.dtype))
    for name, f in plain.items():
        monkeypatch.setattr(tokens, name, f)


@pytest.mark.parametrize("autocast", [False, True])
def test_scan_block_with_plain_operators(plain, autocast):
    """Types under autocast, and a gradient for every parameter."""
    torch.manual_seed(0)
    m, x = tokens.ScanBlock(16, experts=3, dtype=torch.float32), torch.randn(12, 16, requires_grad=True)
    cu = torch.tensor([0, 5, 12])
    with torch.autocast("cpu", torch.bfloat16, enabled=autocast):
        y = m(x, cu)
    assert y.dtype == torch.float32
    y.square().mean().backward()
    assert all(p.grad is not None and p.grad.isfinite().all() and p.grad.dtype == p.dtype for p in m.parameters())
    # half of the channels see the tokens before, half those after, and none another sequence
    z = x.detach().clone()
    z[6, 3] += 1.0     # not of all channels: the norm takes that away
    with torch.autocast("cpu", torch.bfloat16, enabled=autocast):
        changed = (m(z, cu) != m(x.detach(), cu)).any(1)
    assert not changed[:5].any() and changed[5:].all()
