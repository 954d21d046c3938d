"""TokenBlock's use of its operators, with plain PyTorch in their place: which
generator words its dropouts get, and what type conversions leave of it."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from memory_bound_cnn_amd import tokens

T, C = 24, 32


@pytest.fixture
def plain(monkeypatch):
    """The operators the block calls, in plain PyTorch; records dropout's words."""
    words = []

    def dropout(x, p, rng, residual=None):
        assert residual is None or residual.dtype == x.dtype
        words.append(tuple(rng.tolist()))
        g = torch.Generator().manual_seed(hash(words[-1]) % (1 << 62))
        kept = x * (torch.rand(x.shape, generator=g) >= p) / (1 - p)
        return kept if residual is None else kept + residual

    def rotary_attention(qkv, Hq, Hk, *a, **k):
        return qkv[:, :Hq] * qkv[:, Hq:Hq + Hk].mean(1, keepdim=True) + qkv[:, Hq + Hk:].mean(1, keepdim=True)

    def rms_norm(x, weight, residual=None, eps=1e-6):
        assert residual is None and weight.dtype == torch.float32
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + eps) * weight).to(x.dtype)

    for f in (dropout, rotary_attention, rms_norm):
        monkeypatch.setattr(tokens, f.__name__, f)
    return words


def block(**kw):
    return tokens.TokenBlock(C, 2, kv_heads=1, p=0.5, dtype=torch.float32, **kw)


def gradients(m, x, call):
    m.zero_grad()
    x = x.clone().requires_grad_()
    y = call(x)
    y.square().sum().backward()
    return [y.detach(), x.grad] + [p.grad.clone() for p in m.parameters()]


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpointed_block_has_the_blocks_gradients(plain, reentrant):
    """A forward pass that is computed again in the backward pass drops what it dropped."""
    torch.manual_seed(0)
    m, x = block(), torch.randn(T, C)
    torch.manual_seed(1)
    want = gradients(m, x, lambda t: m(t, None, None))
    n = len(plain)
    torch.manual_seed(1)
    got = gradients(m, x, lambda t: checkpoint(m, t, None, None, use_reentrant=reentrant))
    assert plain[:n] == plain[n:2 * n] == plain[2 * n:]
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_blocks_without_seeds_drop_different_elements(plain):
    torch.manual_seed(0)
    net = torch.nn.ModuleList(block() for _ in range(3))
    x = torch.randn(T, C)
    for _ in range(2):
        for m in net:
            x = m(x, None, None)
    assert len(set(plain)) == 2 * 2 * 3


def test_seeds_tell_blocks_of_one_generator_state_apart(plain):
    """As on the ranks of a data-parallel run that all started from one seed."""
    x = torch.randn(T, C)
    for seed in (0, 1, -1, 2 ** 63 - 1):
        m = block(seed=seed)
        torch.manual_seed(5)
        m(x, None, None)
    assert len(set(plain)) == 8


def test_the_generator_decides(plain):
    m, x = block(), torch.randn(T, C)
    out = []
    for seed in (3, 3, 4):
        torch.manual_seed(seed)
        out.append(m(x, None, None))
    assert torch.equal(out[0], out[1]) and not torch.equal(out[0], out[2])


def test_norms_and_frequencies_stay_float32(plain):
    """The operators take float32 parameters whatever the activations' type; a
    conversion of the module must not round them either."""
    torch.manual_seed(0)
    m = block()
    with torch.no_grad():
        m.norm1.weight.add_(torch.randn(C) * 0.1)
    weight, f = m.norm1.weight.clone(), m.inv_freq.clone()
    for convert in (lambda: m.to(torch.bfloat16), lambda: m.bfloat16(), lambda: m.double(), lambda: m.to(torch.bfloat16)):
        assert convert() is m
        assert m.norm1.weight.dtype == m.inv_freq.dtype == torch.float32 and isinstance(m.norm1.weight, torch.nn.Parameter)
        assert torch.equal(m.norm1.weight, weight) and torch.equal(m.inv_freq, f)
        assert "inv_freq" in m.state_dict()
    assert m.qkv.weight.dtype == torch.bfloat16 and m.rng.dtype == torch.int64
    assert m(torch.randn(T, C, dtype=torch.bfloat16), None, None).dtype == torch.bfloat16
    n = tokens.RMSNorm(C).to("meta", torch.bfloat16)
    assert n.weight.dtype == torch.float32 and n.weight.is_meta


@pytest.mark.parametrize("train", [False, True])
def test_block_under_autocast(plain, train):
    m, x = block().train(train), torch.randn(T, C)
    with torch.autocast("cpu", torch.bfloat16):
        y = m(x, None, None)
    assert y.dtype == torch.float32
    y.sum().backward()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in m.parameters())
