"""Token operators without a GPU: the library exports what
include/wtconv_tokens.h declares and refuses bad arguments before any HIP call;
the Python entry points refuse tensors they cannot take."""

import ctypes
import os
import re

import pytest
import torch

from memory_bound_cnn_amd import binding, token_binding as tb, tokens

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(4096)    # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(4100)  # not 16-byte aligned
EINVAL, ESHAPE, EDTYPE, EWORKSPACE = binding.WTC_EINVAL, binding.WTC_ESHAPE, binding.WTC_EDTYPE, binding.WTC_EWORKSPACE


def ref(d):
    return ctypes.addressof(d)


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "wtconv_tokens.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(wtconv_\w+)\s*\(", src)))
    assert "wtconv_attention_forward" in names and "wtconv_dropout" in names
    lib = tb._load()
    for n in names:
        assert hasattr(lib, n), n


def rms(**kw):
    a = dict(rows=3, x_stride=8, r_stride=8, g_stride=8, C=8, dtype=0, fp8=0, eps=1e-6)
    a.update(kw)
    return tb.wtc_rms_desc(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(C=0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(x_stride=-8), EINVAL), (dict(dtype=2), EDTYPE), (dict(fp8=2), EDTYPE),
    (dict(C=tb.RMS_MAX_C + 1), ESHAPE), (dict(rows=1 << 31), ESHAPE),
])
def test_rms_norm_rejects_descriptors(kw, status):
    lib, d = tb._load(), rms(**kw)
    scale = P if kw.get("fp8") else None
    assert lib.wtconv_rms_norm_forward(ref(d), P, P, P, P, P, None, scale, None) == status
    assert lib.wtconv_rms_norm_backward_workspace(ref(d)) == 0


def test_rms_norm_rejects_pointers():
    lib, d = tb._load(), rms()
    f = lib.wtconv_rms_norm_forward
    assert f(None, P, P, P, P, P, None, None, None) == EINVAL
    assert f(ref(d), None, None, P, P, None, None, None, None) == EINVAL
    assert f(ref(d), P, None, None, P, None, None, None, None) == EINVAL
    assert f(ref(d), P, None, P, None, None, None, None, None) == EINVAL
    assert f(ref(d), P, P, P, P, None, None, None, None) == EINVAL      # a residual without h
    assert f(ref(d), P, None, P, P, P, None, None, None) == EINVAL      # h without a residual
    assert f(ref(d), P, None, P, P, None, None, P, None) == EINVAL      # a scale without fp8
    assert f(ref(rms(fp8=1)), P, None, P, P, None, None, None, None) == EINVAL
    b = lib.wtconv_rms_norm_backward
    need = lib.wtconv_rms_norm_backward_workspace(ref(d))
    assert need == 4 * d.C    # three rows of 8 channels: one workgroup, one record
    assert b(ref(d), P, P, P, P, P, P, P, P, need - 1, None) == EWORKSPACE
    assert b(ref(d), P, P, P, P, P, P, P, None, need, None) == EWORKSPACE
    assert b(ref(d), P, P, P, P, P, P, None, P, need, None) == EINVAL
    assert b(ref(d), None, P, P, P, P, P, P, P, need, None) == EINVAL
    assert b(ref(rms(fp8=1)), P, P, P, P, P, P, P, P, need, None) == EDTYPE
    assert f(ref(rms(rows=0)), None, None, None, None, None, None, None, None) == binding.WTC_OK


def rot(**kw):
    a = dict(T=2, x_token=64, x_head=16, y_token=64, y_head=16, heads=4, D=16, dtype=0, axes=2, pairs=(4, 4),
             interleaved=0, inverse=0)
    a.update(kw)
    return tb.wtc_rotary_desc(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), EINVAL), (dict(heads=0), EINVAL), (dict(D=0), EINVAL), (dict(axes=0), EINVAL),
    (dict(axes=5), EINVAL), (dict(pairs=(-1, 4)), EINVAL), (dict(pairs=(5, 4)), ESHAPE), (dict(dtype=9), EDTYPE),
    (dict(interleaved=2), EINVAL), (dict(inverse=-1), EINVAL), (dict(x_head=-16), EINVAL), (dict(T=1 << 31), ESHAPE),
])
def test_rotary_rejects(kw, status):
    assert tb._load().wtconv_rotary(ref(rot(**kw)), P, P, P, P, None) == status


def test_rotary_rejects_pointers():
    f = tb._load().wtconv_rotary
    for at in range(4):
        args = [P, P, P, P]
        args[at] = None
        assert f(ref(rot()), *args, None) == EINVAL
    assert f(None, P, P, P, P, None) == EINVAL
    assert f(ref(rot(T=0)), None, None, None, None, None) == binding.WTC_OK


def test_dropout_rejects():
    f = tb._load().wtconv_dropout
    assert f(-1, 0, 0.1, P, P, P, P, None) == EINVAL
    for p in (-0.1, 1.1, float("nan")):
        assert f(8, 0, p, P, P, P, P, None) == EINVAL
    assert f(8, 5, 0.1, P, P, P, P, None) == EDTYPE
    assert f(8, 0, 0.1, None, P, P, P, None) == EINVAL
    assert f(8, 0, 0.1, P, P, None, P, None) == EINVAL
    assert f(8, 0, 0.1, P, P, P, None, None) == EINVAL
    assert f(0, 0, 0.1, None, None, None, None, None) == binding.WTC_OK


def attn(**kw):
    strides = {n: (256, 64) for n in ("q", "k", "v", "o", "g", "dq", "dk", "dv")}
    a = dict(T=5, n_seq=1, Hq=4, Hk=2, D=64, dtype=1, causal=0, scale=0.125)
    a.update({k: v for k, v in kw.items() if k not in strides})
    strides.update({k: v for k, v in kw.items() if k in strides})
    return tb.wtc_attn_desc(*a.values(), *strides.values())


ATTN_BAD = [
    (dict(T=-1), EINVAL), (dict(n_seq=-1), EINVAL), (dict(Hq=0), EINVAL), (dict(Hk=0), EINVAL), (dict(Hk=3), EINVAL),
    (dict(D=0), EINVAL), (dict(D=60), ESHAPE), (dict(D=136), ESHAPE), (dict(causal=2), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(dtype=3), EDTYPE),
    (dict(T=1 << 31), ESHAPE), (dict(q=(257, 64)), EINVAL), (dict(k=(256, 68)), EINVAL), (dict(v=(-256, 64)), EINVAL),
    (dict(o=(256, 4)), EINVAL), (dict(q=((1 << 22) + 8, 64)), ESHAPE), (dict(T=1 << 30), ESHAPE),
]


@pytest.mark.parametrize("kw,status", ATTN_BAD)
def test_attention_rejects(kw, status):
    lib, d = tb._load(), attn(**kw)
    assert lib.wtconv_attention_forward(ref(d), P, P, P, P, P, P, None, P, 1 << 62, None) == status
    assert lib.wtconv_attention_backward(ref(d), P, P, P, P, P, None, P, P, P, P, P, P, 1 << 62, None) == status


def test_attention_rejects_pointers_and_workspaces():
    lib, d = tb._load(), attn()
    for at in range(5):
        args = [P] * 6
        args[at] = None
        assert lib.wtconv_attention_forward(ref(d), *args, None, None, 0, None) == EINVAL
        if at != 3:    # cu_seqlens is int32
            args[at] = ODD
            assert lib.wtconv_attention_forward(ref(d), *args, None, None, 0, None) == EINVAL
    assert lib.wtconv_attention_forward(ref(d), *[P] * 6, ODD, None, 0, None) == EINVAL
    assert lib.wtconv_attention_forward(ref(attn(dtype=0)), *[P] * 6, P, None, 0, None) == EDTYPE   # nothing is rounded off
    need = lib.wtconv_attention_backward_workspace(ref(d))
    assert need == 256    # 4 heads x 5 tokens x 4 bytes, to the next 256
    for at in range(11):
        if at == 5:    # out_low may be NULL
            continue
        args = [P] * 11
        args[at] = None
        assert lib.wtconv_attention_backward(ref(d), *args, P, need, None) == EINVAL
    assert lib.wtconv_attention_backward(ref(d), *[P] * 11, P, need - 1, None) == EWORKSPACE
    assert lib.wtconv_attention_backward(ref(d), *[P] * 11, None, need, None) == EWORKSPACE
    for name in ("g", "dq", "dk", "dv"):
        bad = attn(**{name: (256, 63)})
        assert lib.wtconv_attention_backward(ref(bad), *[P] * 11, P, need, None) == EINVAL
    assert lib.wtconv_attention_forward(None, P, P, P, P, P, P, None, None, 0, None) == EINVAL
    assert lib.wtconv_attention_forward(ref(attn(T=0)), *[None] * 8, 0, None) == binding.WTC_OK
    # a long sequence of one head is split over workgroups, whose results need a place
    d = attn(T=8192, Hq=1, Hk=1)
    need = lib.wtconv_attention_forward_workspace(ref(d))
    assert need > 0
    assert lib.wtconv_attention_forward(ref(d), *[P] * 6, None, P, need - 1, None) == EWORKSPACE
    assert lib.wtconv_attention_forward(ref(d), *[P] * 6, None, None, need, None) == EWORKSPACE


def test_python_entry_points_refuse_host_tensors():
    x, w = torch.zeros(4, 16), torch.ones(16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        tokens.rms_norm(x, w)
    with pytest.raises(ValueError, match="residual has shape"):
        tokens.rms_norm(x, w, x[:3])
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        tokens.rotary(x.view(4, 1, 16), torch.zeros(4, 1, dtype=torch.int32), torch.ones(8), (8,))
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        tokens.attention(x.view(4, 2, 8), x.view(4, 2, 8), x.view(4, 2, 8), cu)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        tokens.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="qkv has shape"):
        tokens.rotary_attention(x.view(4, 2, 8), 2, 1, None, None, (4,), cu)


def test_image_positions_and_frequencies():
    pos, cu = tokens.image_positions([(2, 3), (0, 5), (1, 1)])
    assert pos.tolist() == [[0, 0], [0, 1], [0, 2], [1, 0], [1, 1], [1, 2], [0, 0]]
    assert cu.tolist() == [0, 6, 6, 7] and pos.dtype == cu.dtype == torch.int32
    f = tokens.rotary_frequencies((2, 1), base=100.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 1.0]))
