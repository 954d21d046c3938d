// PyTorch side of the token operators: checks of tensors, outputs and
// workspaces from PyTorch's allocator, the current stream, and gradients.
// Python module memory_bound_cnn_amd._tokens; memory_bound_cnn_amd/tokens.py
// documents what it offers.
//
// Every operator is registered with PyTorch's dispatcher (namespace
// wtconv_tokens) and called through it, its gradient's parts too, so that a
// trace holds the operator itself: one that saw the output's allocation alone
// would give back whatever that memory holds.  A graph may call any of them
// with other tensors, so each checks its own arguments.
//
// The gradients are C++ nodes because a backward pass runs on a thread of
// PyTorch's own: with Python nodes a step of a small norm spent 128 us on the
// host, two thirds of it there.
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/autograd_not_implemented_fallback.h>
#include <torch/extension.h>
#include <torch/library.h>

#include <cmath>
#include <limits>
#include <optional>
#include <tuple>
#include <vector>

#include "../../include/wtconv_tokens.h"

namespace {

using at::IntArrayRef;
using torch::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;
using OptDouble = std::optional<double>;
using Tensors = std::vector<Tensor>;
// Calls inside of it are not recorded for gradients.  Saved variables are taken before it begins: checkpointing
// computes the forward pass again there.
using NoGraph = at::AutoDispatchBelowADInplaceOrView;

void raise_on(int st, const char* where) {
    TORCH_CHECK(st == WTC_OK, where, ": ", wtconv_status_string(st), " (status ", st, ")");
}

// The device of a call, its current stream, and addresses on it.
struct On {
    c10::DeviceGuard guard;
    void* stream;
    explicit On(const Tensor& t)
        : guard(t.device()), stream(c10::hip::getCurrentHIPStream(t.device().index()).stream()) {}
};
const void* in(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void* out(const Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }
template <typename T>
const T* in_as(const Tensor& t) {
    return static_cast<const T*>(in(t));
}

Tensor empty(IntArrayRef shape, const Tensor& like) { return at::empty(shape, like.options()); }
Tensor empty(IntArrayRef shape, const Tensor& like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}
Tensor workspace(size_t bytes, const Tensor& like) {
    return bytes ? empty({(int64_t)bytes}, like, at::kByte) : Tensor();
}

bool dense(const Tensor& t) { return t.stride(-1) == 1 || t.size(-1) <= 1; }

int dtype_of(const Tensor& t) { return t.scalar_type() == at::kFloat ? WTC_FP32 : WTC_BF16; }
int activation(const Tensor& t, const char* name, int64_t dims) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16, name, " has dtype ",
                      t.scalar_type(), ", expected float32 or bfloat16");
    TORCH_CHECK_VALUE(dims < 0 || t.dim() == dims, name, " has shape ", t.sizes(), ", expected ", dims, " axes");
    return dtype_of(t);
}
void check(const Tensor& t, const char* name, at::ScalarType type, const Tensor& like, IntArrayRef shape,
           bool contiguous = true) {
    TORCH_CHECK_VALUE(t.device() == like.device(), name, " must be a CUDA tensor on ", like.device());
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " has dtype ", t.scalar_type(), ", expected ", type);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(!contiguous || t.is_contiguous(), name, " must be contiguous");
}
// like's type, device and shape
void check_like(const Tensor& t, const char* name, const Tensor& like) {
    check(t, name, like.scalar_type(), like, like.sizes(), false);
}
void check_residual(const Tensor& x, const OptTensor& r) {
    if (!r) return;
    TORCH_CHECK_VALUE(r->sizes() == x.sizes(), "residual has shape ", r->sizes(), ", expected ", x.sizes());
    check_like(*r, "residual", x);
}

template <typename... Ts>
bool wants_grad(const Ts&... ts) {
    return at::GradMode::is_enabled() && (... || ts.requires_grad());
}
bool wants_grad_opt(const OptTensor& t) { return t && wants_grad(*t); }

// A tangent that came with an input would silently not leave with the output.
bool has_tangent(const Tensor& t) { return t.defined() && t._fw_grad(0).defined(); }
bool has_tangent(const OptTensor& t) { return t && has_tangent(*t); }
template <typename... Ts>
void refuse_tangents(const Ts&... ts) {
    TORCH_CHECK(!(... || has_tangent(ts)) || !c10::AutogradState::get_tls_state().get_fw_grad_mode(),
                "the token operators have no forward-mode derivatives");
}

// A gradient's own gradient would have to be written down; without this it
// would silently be zero: that by the output's gradient, and where the operator
// is not linear, that by its inputs.
void once(const variable_list& grads, bool linear) {
    if (!at::GradMode::is_enabled()) return;   // create_graph
    TORCH_CHECK(linear, "the token operators have first derivatives only");
    for (const Tensor& g : grads)
        TORCH_CHECK(!g.defined() || !g.requires_grad(), "the token operators have first derivatives only");
}

// Sizes that the library takes as int.
int narrow(int64_t n, const char* what) {
    TORCH_CHECK_VALUE(n <= std::numeric_limits<int>::max(), what, ": ", n, " do not fit 32 bits");
    return (int)n;
}
int sequences(const Tensor& cu) {
    TORCH_CHECK_VALUE(cu.dim() == 1 && cu.size(0) >= 1, "cu_seqlens must be [n + 1]");
    return narrow(cu.size(0), "entries of cu_seqlens") - 1;
}

// [rows, C] with a contiguous last axis; a view where t allows it.
Tensor rows(const Tensor& t) {
    const Tensor r = t.dim() == 2 ? t : t.reshape({-1, t.size(-1)});
    return dense(r) ? r : r.contiguous();
}

// ================================================================== kernels
// An operator's work on its tensors, with no thought of gradients.  The
// functions of namespace op are the dispatcher's, under their own names.

// ------------------------------------------------------------------ root-mean-square norm
struct Rms {
    Tensor y, h, rstd, scale;
};
Rms rms_forward(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps, bool keep, bool fp8) {
    TORCH_CHECK_VALUE(x.dim() >= 1, "x has no axis");
    check_residual(x, residual);
    const int dtype = activation(x, "x", -1);
    const int C = narrow(x.size(-1), "channels of x");
    check(weight, "weight", at::kFloat, x, {C});
    const Tensor xr = rows(x), rr = residual ? rows(*residual) : Tensor();
    const int64_t n = xr.size(0);
    Rms o;
    o.y = fp8 ? empty(x.sizes(), x, at::kFloat8_e4m3fn) : empty(x.sizes(), x);
    if (residual) o.h = empty(x.sizes(), x);
    if (keep) o.rstd = empty({n}, x, at::kFloat);
    if (fp8) o.scale = empty(x.sizes().slice(0, x.dim() - 1), x, at::kFloat);
    const wtc_rms_desc d = {n, xr.stride(0), residual ? rr.stride(0) : 0, 0, C, dtype, fp8, (float)eps};
    const On on(x);
    raise_on(wtconv_rms_norm_forward(&d, in(xr), in(rr), in_as<float>(weight), out(o.y), out(o.h),
                                     static_cast<float*>(out(o.rstd)), static_cast<float*>(out(o.scale)), on.stream),
             "wtconv_rms_norm_forward");
    return o;
}

// ------------------------------------------------------------------ rotary positions
void rotary_check(const Tensor& x, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections) {
    activation(x, "x", 3);
    narrow(x.size(1), "heads of x");
    narrow(x.size(2), "channels of a head of x");
    TORCH_CHECK_VALUE(!sections.empty() && sections.size() <= WTC_ROTARY_MAX_AXES, sections.size(), " sections: 1 to ",
                      WTC_ROTARY_MAX_AXES, " axes are supported");
    int64_t P = 0;
    for (const int64_t n : sections) {
        TORCH_CHECK_VALUE(n >= 0 && n <= x.size(2), "sections must be pairs of channels of a head");
        P += n;
    }
    TORCH_CHECK_VALUE(2 * P <= x.size(2), P, " pairs do not fit ", x.size(2), " channels");
    check(positions, "positions", at::kInt, x, {x.size(0), (int64_t)sections.size()});
    check(inv_freq, "inv_freq", at::kFloat, x, {P});
}
// x to y, which may be x; what rotary_check has checked
void rotary_run(const Tensor& x, const Tensor& y, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections,
                bool interleaved, bool inverse) {
    wtc_rotary_desc d = {x.size(0),   x.stride(0),          x.stride(1), y.stride(0), y.stride(1), (int)x.size(1),
                         (int)x.size(2), dtype_of(x), (int)sections.size(), {},          interleaved, inverse};
    for (size_t i = 0; i < sections.size(); ++i) d.pairs[i] = (int)sections[i];
    const On on(x);
    raise_on(wtconv_rotary(&d, in(x), in_as<int>(positions), in_as<float>(inv_freq), out(y), on.stream),
             "wtconv_rotary");
}
Tensor turned(const Tensor& x, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections, bool interleaved,
              bool inverse) {
    const Tensor xd = dense(x) ? x : x.contiguous(), y = empty(x.sizes(), x);
    rotary_run(xd, y, positions, inv_freq, sections, interleaved, inverse);
    return y;
}

// ------------------------------------------------------------------ attention
// t [T, heads, D] as the kernels read it: tokens and heads start at multiples of 16 bytes; a copy where they do not.
Tensor heads(const Tensor& t) {
    const int64_t unit = 16 / t.element_size();
    if (t.stride(2) == 1 && t.stride(0) % unit == 0 && t.stride(1) % unit == 0 &&
        reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0 && t.stride(0) <= WTC_ATTN_MAX_TOKEN_STRIDE)
        return t;
    return t.clone(at::MemoryFormat::Contiguous);
}
wtc_attn_strides strides(const Tensor& t) { return {t.stride(0), t.stride(1)}; }

struct Setting {
    bool causal;
    OptDouble scale;
};
wtc_attn_desc attn_desc(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, const Setting& s) {
    wtc_attn_desc d = {};
    d.T = q.size(0);
    d.n_seq = sequences(cu);
    d.Hq = (int)q.size(1);
    d.Hk = (int)k.size(1);
    d.D = (int)q.size(2);
    d.dtype = dtype_of(q);
    d.causal = s.causal;
    d.scale = (float)(s.scale ? *s.scale : 1.0 / std::sqrt((double)q.size(2)));
    d.q = strides(q);
    d.k = strides(k);
    d.v = strides(v);
    return d;
}
void cu_check(const Tensor& cu, const Tensor& like) {
    sequences(cu);
    check(cu, "cu_seqlens", at::kInt, like, cu.sizes());
}
void attn_check(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu) {
    activation(q, "q", 3);
    narrow(q.size(1), "heads of q");
    narrow(q.size(2), "channels of a head of q");
    const int64_t Hk = k.dim() == 3 ? k.size(1) : 0;
    check(k, "k", q.scalar_type(), q, {q.size(0), Hk, q.size(2)}, false);
    check(v, "v", q.scalar_type(), q, {q.size(0), Hk, q.size(2)}, false);
    TORCH_CHECK_VALUE(Hk >= 1 && q.size(1) % Hk == 0, q.size(1), " heads of q do not divide into ", Hk, " of k and v");
    cu_check(cu, q);
}
struct AttnOut {
    Tensor o, lse, low;   // lse, low: kept for the backward pass (low: what was rounded off o, bfloat16)
    Tensors kept() const { return low.defined() ? Tensors{o, lse, low} : Tensors{o, lse}; }
};
AttnOut attn_forward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, const Setting& s,
                     bool keep) {
    wtc_attn_desc d = attn_desc(q, k, v, cu, s);
    const AttnOut r = {empty(q.sizes(), q), keep ? empty({q.size(1), q.size(0)}, q, at::kFloat) : Tensor(),
                       keep && q.scalar_type() == at::kBFloat16 ? empty(q.sizes(), q) : Tensor()};
    d.o = strides(r.o);
    const size_t bytes = wtconv_attention_forward_workspace(&d);
    const Tensor ws = workspace(bytes, q);
    const On on(q);
    raise_on(wtconv_attention_forward(&d, in(q), in(k), in(v), in_as<int>(cu), out(r.o), static_cast<float*>(out(r.lse)),
                                      out(r.low), out(ws), bytes, on.stream),
             "wtconv_attention_forward");
    return r;
}
// g and kept are checked here, by the q of what attn_check has checked
void attn_backward(const Tensor& g0, const Tensor& q, const Tensor& k, const Tensor& v, at::TensorList kept,
                   const Tensor& cu, const Setting& s, const Tensor& dq, const Tensor& dk, const Tensor& dv) {
    TORCH_CHECK_VALUE(kept.size() == 2 || kept.size() == 3, "kept has ", kept.size(), " tensors, expected 2 or 3");
    check_like(g0, "the gradient", q);
    check_like(kept[0], "out", q);
    check(kept[1], "lse", at::kFloat, q, {q.size(1), q.size(0)});
    if (kept.size() > 2) check(kept[2], "what was rounded off out", at::kBFloat16, q, q.sizes());
    const Tensor g = heads(g0), o = heads(kept[0]), low = kept.size() > 2 ? kept[2] : Tensor();
    wtc_attn_desc d = attn_desc(q, k, v, cu, s);
    d.o = strides(o);
    d.g = strides(g);
    d.dq = strides(dq);
    d.dk = strides(dk);
    d.dv = strides(dv);
    const size_t bytes = wtconv_attention_backward_workspace(&d);
    const Tensor ws = workspace(bytes, q);
    const On on(q);
    raise_on(wtconv_attention_backward(&d, in(q), in(k), in(v), in(o), in_as<float>(kept[1]), in(low), in(g),
                                       in_as<int>(cu), out(dq), out(dk), out(dv), out(ws), bytes, on.stream),
             "wtconv_attention_backward");
}

// the q and k heads of a projection, turned, and the attention of it
void projection_check(const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions, const Tensor& inv_freq,
                      IntArrayRef sections, const Tensor& cu) {
    TORCH_CHECK_VALUE(Hq >= 1 && Hk >= 1 && Hq % Hk == 0, Hq, " heads of q do not divide into ", Hk, " of k and v");
    activation(qkv, "qkv", 3);
    TORCH_CHECK_VALUE(qkv.size(1) == Hq + 2 * Hk, "qkv has ", qkv.size(1), " heads, expected ", Hq + 2 * Hk);
    rotary_check(qkv, positions, inv_freq, sections);
    cu_check(cu, qkv);
}
struct Turned {
    Tensor qk;
    AttnOut f;
};
Turned turned_forward(const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions, const Tensor& inv_freq,
                      IntArrayRef sections, const Tensor& cu, bool interleaved, const Setting& s, bool keep) {
    const Tensor qk = turned(qkv.narrow(1, 0, Hq + Hk), positions, inv_freq, sections, interleaved, false);
    return {qk, attn_forward(qk.narrow(1, 0, Hq), qk.narrow(1, Hq, Hk), qkv.narrow(1, Hq + Hk, Hk), cu, s, keep)};
}

// ------------------------------------------------------------------ the dispatcher's functions
namespace op {

// [y], or [y, h] with a residual
Tensors rms_norm(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
    const Rms o = rms_forward(x, weight, residual, eps, false, false);
    return residual ? Tensors{o.y, o.h} : Tensors{o.y};
}
// [y8, scale], or [y8, scale, h]
Tensors rms_norm_fp8(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
    const Rms o = rms_forward(x, weight, residual, eps, false, true);
    return residual ? Tensors{o.y, o.scale, o.h} : Tensors{o.y, o.scale};
}
// [rstd, y], or [rstd, y, h]
Tensors _rms_norm_forward(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
    const Rms o = rms_forward(x, weight, residual, eps, true, false);
    return residual ? Tensors{o.rstd, o.y, o.h} : Tensors{o.rstd, o.y};
}
// (dx, dw); h: what was normed (x without a residual)
std::tuple<Tensor, Tensor> _rms_norm_backward(const Tensor& dy0, const OptTensor& dh0, const Tensor& h0,
                                              const Tensor& weight, const Tensor& rstd) {
    TORCH_CHECK_VALUE(h0.dim() >= 1, "h has no axis");
    const int dtype = activation(h0, "h", -1);
    const int C = narrow(h0.size(-1), "channels of h");
    check(weight, "weight", at::kFloat, h0, {C});
    check_like(dy0, "dy", h0);
    if (dh0) check_like(*dh0, "dh", h0);
    const Tensor h = rows(h0), dy = rows(dy0), dh = dh0 ? rows(*dh0).contiguous() : Tensor();
    const int64_t n = h.size(0);
    check(rstd, "rstd", at::kFloat, h0, {n});
    const wtc_rms_desc d = {n, h.stride(0), 0, dy.stride(0), C, dtype, 0, 0.f};
    const size_t bytes = wtconv_rms_norm_backward_workspace(&d);
    const Tensor dx = empty(h0.sizes(), h), dw = empty({C}, h, at::kFloat), ws = workspace(bytes, h);
    const On on(h);
    raise_on(wtconv_rms_norm_backward(&d, in(dy), in(dh), in(h), in_as<float>(weight), in_as<float>(rstd), out(dx),
                                      static_cast<float*>(out(dw)), out(ws), bytes, on.stream),
             "wtconv_rms_norm_backward");
    return {dx, dw};
}

Tensor rotary(const Tensor& x, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections,
              bool interleaved) {
    rotary_check(x, positions, inv_freq, sections);
    return turned(x, positions, inv_freq, sections, interleaved, false);
}
Tensor _rotary_backward(const Tensor& dy, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections,
                        bool interleaved) {
    rotary_check(dy, positions, inv_freq, sections);
    return turned(dy, positions, inv_freq, sections, interleaved, true);
}

Tensor attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, bool causal, OptDouble scale) {
    attn_check(q, k, v, cu);
    return attn_forward(heads(q), heads(k), heads(v), cu, {causal, scale}, false).o;
}
// [out, lse], or bfloat16 [out, lse, what was rounded off out]
Tensors _attention_forward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, bool causal,
                           OptDouble scale) {
    attn_check(q, k, v, cu);
    return attn_forward(heads(q), heads(k), heads(v), cu, {causal, scale}, true).kept();
}
// (dq, dk, dv); kept: as _attention_forward gave it
std::tuple<Tensor, Tensor, Tensor> _attention_backward(const Tensor& g, const Tensor& q0, const Tensor& k0,
                                                       const Tensor& v0, at::TensorList kept, const Tensor& cu,
                                                       bool causal, OptDouble scale) {
    attn_check(q0, k0, v0, cu);
    const Tensor q = heads(q0), k = heads(k0), v = heads(v0);
    const Tensor dq = empty(q.sizes(), q), dk = empty(k.sizes(), q), dv = empty(v.sizes(), q);
    attn_backward(g, q, k, v, kept, cu, {causal, scale}, dq, dk, dv);
    return {dq, dk, dv};
}

Tensor rotary_attention(const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions, const Tensor& inv_freq,
                        IntArrayRef sections, const Tensor& cu, bool interleaved, bool causal, OptDouble scale) {
    projection_check(qkv, Hq, Hk, positions, inv_freq, sections, cu);
    return turned_forward(heads(qkv), Hq, Hk, positions, inv_freq, sections, cu, interleaved, {causal, scale}, false).f.o;
}
// [the turned q and k heads, then as _attention_forward]
Tensors _rotary_attention_forward(const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions,
                                  const Tensor& inv_freq, IntArrayRef sections, const Tensor& cu, bool interleaved,
                                  bool causal, OptDouble scale) {
    projection_check(qkv, Hq, Hk, positions, inv_freq, sections, cu);
    const Turned t = turned_forward(heads(qkv), Hq, Hk, positions, inv_freq, sections, cu, interleaved, {causal, scale}, true);
    Tensors all = t.f.kept();
    all.insert(all.begin(), t.qk);
    return all;
}
// the projection's gradient: written where it is wanted, and turned back there
Tensor _rotary_attention_backward(const Tensor& g, const Tensor& qkv0, const Tensor& qk0, at::TensorList kept, int64_t Hq,
                                  int64_t Hk, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections,
                                  const Tensor& cu, bool interleaved, bool causal, OptDouble scale) {
    projection_check(qkv0, Hq, Hk, positions, inv_freq, sections, cu);
    check(qk0, "the turned heads", qkv0.scalar_type(), qkv0, {qkv0.size(0), Hq + Hk, qkv0.size(2)}, false);
    const Tensor qkv = heads(qkv0), qk = heads(qk0);
    const Tensor d = empty(qkv.sizes(), qkv), dqk = d.narrow(1, 0, Hq + Hk);
    attn_backward(g, qk.narrow(1, 0, Hq), qk.narrow(1, Hq, Hk), qkv.narrow(1, Hq + Hk, Hk), kept, cu, {causal, scale},
                  d.narrow(1, 0, Hq), d.narrow(1, Hq, Hk), d.narrow(1, Hq + Hk, Hk));
    rotary_run(dqk, dqk, positions, inv_freq, sections, interleaved, true);
    return d;
}

Tensor dropout(const Tensor& x, double p, const Tensor& rng, const OptTensor& residual) {
    const int dtype = activation(x, "x", -1);
    check_residual(x, residual);
    check(rng, "rng", at::kLong, x, {2});
    TORCH_CHECK_VALUE(p >= 0.0 && p <= 1.0, "p = ", p, " is no probability");
    const Tensor xc = x.contiguous(), rc = residual ? residual->contiguous() : Tensor(), y = empty(x.sizes(), x);
    const On on(x);
    raise_on(wtconv_dropout(x.numel(), dtype, p, in(xc), in(rc), static_cast<const unsigned long long*>(in(rng)), out(y),
                            on.stream),
             "wtconv_dropout");
    return y;
}

}  // namespace op

// A dispatched operator with the arguments of its function above.
#define OP(name)                                                                                                  \
    ([]() -> const auto& {                                                                                        \
        static const auto handle =                                                                                \
            c10::Dispatcher::singleton().findSchemaOrThrow("wtconv_tokens::" #name, "").typed<decltype(op::name)>(); \
        return handle;                                                                                            \
    }())

// ================================================================== gradients
struct RmsNorm : torch::autograd::Function<RmsNorm> {
    // Saves the norm's input (h, or x without a residual) and one float per row.
    static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const OptTensor& residual,
                                 double eps) {
        const NoGraph guard;
        Tensors o = OP(_rms_norm_forward).call(x, weight, residual, eps);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({residual ? o[2] : x, weight, o[0]});
        o.erase(o.begin());
        return o;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        const variable_list s = ctx->get_saved_variables();
        const Tensor dh = g.size() > 1 ? g[1] : Tensor();
        if (!g[0].defined()) return {dh, Tensor(), dh, Tensor()};
        const NoGraph guard;
        const auto [dx, dw] =
            OP(_rms_norm_backward).call(g[0], dh.defined() ? OptTensor(dh) : std::nullopt, s[0], s[1], s[2]);
        return {dx, dw, g.size() > 1 ? dx : Tensor(), Tensor()};
    }
};

struct Rotary : torch::autograd::Function<Rotary> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& positions, const Tensor& inv_freq,
                          std::vector<int64_t> sections, bool interleaved) {
        const NoGraph guard;
        ctx->save_for_backward({positions, inv_freq});
        ctx->saved_data["sections"] = sections;
        ctx->saved_data["interleaved"] = interleaved;
        return OP(rotary).call(x, positions, inv_freq, sections, interleaved);
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, true);
        const variable_list s = ctx->get_saved_variables();
        const NoGraph guard;
        return {OP(_rotary_backward).call(g[0], s[0], s[1], ctx->saved_data["sections"].toIntVector(),
                                          ctx->saved_data["interleaved"].toBool()),
                Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

struct Attention : torch::autograd::Function<Attention> {
    // Saves its inputs, its output (with what was rounded off it) and one float per query and head.
    static Tensor forward(AutogradContext* ctx, const Tensor& q0, const Tensor& k0, const Tensor& v0, const Tensor& cu,
                          bool causal, OptDouble scale) {
        const NoGraph guard;
        attn_check(q0, k0, v0, cu);
        const Tensor q = heads(q0), k = heads(k0), v = heads(v0);   // copies, if any, are made once for both passes
        const Tensors kept = OP(_attention_forward).call(q, k, v, cu, causal, scale);
        variable_list save = {q, k, v, cu};
        save.insert(save.end(), kept.begin(), kept.end());
        ctx->save_for_backward(std::move(save));
        ctx->saved_data["causal"] = causal;
        ctx->saved_data["scale"] = scale;
        return kept[0];
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        const variable_list s = ctx->get_saved_variables();
        const NoGraph guard;
        const auto [dq, dk, dv] = OP(_attention_backward).call(
            g[0], s[0], s[1], s[2], at::TensorList(s).slice(4), s[3], ctx->saved_data["causal"].toBool(),
            ctx->saved_data["scale"].toOptional<double>());
        return {dq, dk, dv, Tensor(), Tensor(), Tensor()};
    }
};

struct RotaryAttention : torch::autograd::Function<RotaryAttention> {
    // rotary on q and k, then attention, on one projection
    static Tensor forward(AutogradContext* ctx, const Tensor& qkv0, int64_t Hq, int64_t Hk, const Tensor& positions,
                          const Tensor& inv_freq, std::vector<int64_t> sections, const Tensor& cu, bool interleaved,
                          bool causal, OptDouble scale) {
        const NoGraph guard;
        projection_check(qkv0, Hq, Hk, positions, inv_freq, sections, cu);
        const Tensor qkv = heads(qkv0);
        const Tensors all =
            OP(_rotary_attention_forward).call(qkv, Hq, Hk, positions, inv_freq, sections, cu, interleaved, causal, scale);
        variable_list save = {qkv, cu, positions, inv_freq};
        save.insert(save.end(), all.begin(), all.end());
        ctx->save_for_backward(std::move(save));
        ctx->saved_data["Hq"] = Hq;
        ctx->saved_data["Hk"] = Hk;
        ctx->saved_data["sections"] = sections;
        ctx->saved_data["interleaved"] = interleaved;
        ctx->saved_data["causal"] = causal;
        ctx->saved_data["scale"] = scale;
        return all[1];
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        const variable_list s = ctx->get_saved_variables();
        const NoGraph guard;
        auto& at = ctx->saved_data;
        variable_list r(10);
        r[0] = OP(_rotary_attention_backward).call(
            g[0], s[0], s[4], at::TensorList(s).slice(5), at["Hq"].toInt(), at["Hk"].toInt(), s[2], s[3],
            at["sections"].toIntVector(), s[1], at["interleaved"].toBool(), at["causal"].toBool(),
            at["scale"].toOptional<double>());
        return r;
    }
};

struct Dropout : torch::autograd::Function<Dropout> {
    // Saves the generator's two words; the decisions are drawn again.
    static Tensor forward(AutogradContext* ctx, const Tensor& x, double p, const Tensor& rng, const OptTensor& residual) {
        const NoGraph guard;
        ctx->save_for_backward({rng});
        ctx->saved_data["p"] = p;
        ctx->saved_data["residual"] = residual.has_value();
        return OP(dropout).call(x, p, rng, residual);
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, true);
        Tensor dx;
        if (ctx->needs_input_grad(0)) {
            const Tensor rng = ctx->get_saved_variables()[0];
            const NoGraph guard;
            dx = OP(dropout).call(g[0], ctx->saved_data["p"].toDouble(), rng, std::nullopt);
        }
        return {dx, Tensor(), Tensor(), ctx->saved_data["residual"].toBool() ? g[0] : Tensor()};
    }
};

// What the dispatcher runs ahead of the kernels.
namespace graph {

Tensors rms_norm(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
    refuse_tangents(x, weight, residual);
    if (wants_grad(x, weight) || wants_grad_opt(residual)) return RmsNorm::apply(x, weight, residual, eps);
    const NoGraph guard;
    return OP(rms_norm).call(x, weight, residual, eps);
}
Tensors rms_norm_fp8(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
    refuse_tangents(x, weight, residual);
    TORCH_CHECK_VALUE(!wants_grad(x, weight) && !wants_grad_opt(residual),
                      "rms_norm_fp8 has no gradient; call it under torch.no_grad()");
    const NoGraph guard;
    return OP(rms_norm_fp8).call(x, weight, residual, eps);
}
Tensor rotary(const Tensor& x, const Tensor& positions, const Tensor& inv_freq, IntArrayRef sections,
              bool interleaved) {
    refuse_tangents(x, inv_freq);
    if (wants_grad(x)) return Rotary::apply(x, positions, inv_freq, sections.vec(), interleaved);
    const NoGraph guard;
    return OP(rotary).call(x, positions, inv_freq, sections, interleaved);
}
Tensor attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, bool causal, OptDouble scale) {
    refuse_tangents(q, k, v);
    if (wants_grad(q, k, v)) return Attention::apply(q, k, v, cu, causal, scale);
    const NoGraph guard;
    return OP(attention).call(q, k, v, cu, causal, scale);
}
Tensor rotary_attention(const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions, const Tensor& inv_freq,
                        IntArrayRef sections, const Tensor& cu, bool interleaved, bool causal, OptDouble scale) {
    refuse_tangents(qkv, inv_freq);
    if (wants_grad(qkv))
        return RotaryAttention::apply(qkv, Hq, Hk, positions, inv_freq, sections.vec(), cu, interleaved, causal, scale);
    const NoGraph guard;
    return OP(rotary_attention).call(qkv, Hq, Hk, positions, inv_freq, sections, cu, interleaved, causal, scale);
}
Tensor dropout(const Tensor& x, double p, const Tensor& rng, const OptTensor& residual) {
    refuse_tangents(x, residual);
    if (wants_grad(x) || wants_grad_opt(residual)) return Dropout::apply(x, p, rng, residual);
    const NoGraph guard;
    return OP(dropout).call(x, p, rng, residual);
}

}  // namespace graph

// The CPU's registration is there for the message that its tensors get.
void kernels(torch::Library& m) {
    m.impl("rms_norm", &op::rms_norm);
    m.impl("rms_norm_fp8", &op::rms_norm_fp8);
    m.impl("rotary", &op::rotary);
    m.impl("attention", &op::attention);
    m.impl("rotary_attention", &op::rotary_attention);
    m.impl("dropout", &op::dropout);
    m.impl("_rms_norm_forward", &op::_rms_norm_forward);
    m.impl("_rms_norm_backward", &op::_rms_norm_backward);
    m.impl("_rotary_backward", &op::_rotary_backward);
    m.impl("_attention_forward", &op::_attention_forward);
    m.impl("_attention_backward", &op::_attention_backward);
    m.impl("_rotary_attention_forward", &op::_rotary_attention_forward);
    m.impl("_rotary_attention_backward", &op::_rotary_attention_backward);
}

}  // namespace

TORCH_LIBRARY(wtconv_tokens, m) {
    m.def("rms_norm(Tensor x, Tensor weight, Tensor? residual, float eps) -> Tensor[]");
    m.def("rms_norm_fp8(Tensor x, Tensor weight, Tensor? residual, float eps) -> Tensor[]");
    m.def("rotary(Tensor x, Tensor positions, Tensor inv_freq, int[] sections, bool interleaved) -> Tensor");
    m.def("attention(Tensor q, Tensor k, Tensor v, Tensor cu_seqlens, bool causal, float? scale) -> Tensor");
    m.def("rotary_attention(Tensor qkv, int Hq, int Hk, Tensor positions, Tensor inv_freq, int[] sections, "
          "Tensor cu_seqlens, bool interleaved, bool causal, float? scale) -> Tensor");
    m.def("dropout(Tensor x, float p, Tensor rng, Tensor? residual) -> Tensor");
    m.def("_rms_norm_forward(Tensor x, Tensor weight, Tensor? residual, float eps) -> Tensor[]");
    m.def("_rms_norm_backward(Tensor dy, Tensor? dh, Tensor h, Tensor weight, Tensor rstd) -> (Tensor, Tensor)");
    m.def("_rotary_backward(Tensor dy, Tensor positions, Tensor inv_freq, int[] sections, bool interleaved) -> Tensor");
    m.def("_attention_forward(Tensor q, Tensor k, Tensor v, Tensor cu_seqlens, bool causal, float? scale) -> Tensor[]");
    m.def("_attention_backward(Tensor g, Tensor q, Tensor k, Tensor v, Tensor[] kept, Tensor cu_seqlens, bool causal, "
          "float? scale) -> (Tensor, Tensor, Tensor)");
    m.def("_rotary_attention_forward(Tensor qkv, int Hq, int Hk, Tensor positions, Tensor inv_freq, int[] sections, "
          "Tensor cu_seqlens, bool interleaved, bool causal, float? scale) -> Tensor[]");
    m.def("_rotary_attention_backward(Tensor g, Tensor qkv, Tensor qk, Tensor[] kept, int Hq, int Hk, Tensor positions, "
          "Tensor inv_freq, int[] sections, Tensor cu_seqlens, bool interleaved, bool causal, float? scale) -> Tensor");
}
TORCH_LIBRARY_IMPL(wtconv_tokens, CUDA, m) { kernels(m); }
TORCH_LIBRARY_IMPL(wtconv_tokens, CPU, m) { kernels(m); }
TORCH_LIBRARY_IMPL(wtconv_tokens, Autograd, m) {
    m.impl("rms_norm", &graph::rms_norm);
    m.impl("rms_norm_fp8", &graph::rms_norm_fp8);
    m.impl("rotary", &graph::rotary);
    m.impl("attention", &graph::attention);
    m.impl("rotary_attention", &graph::rotary_attention);
    m.impl("dropout", &graph::dropout);
    // the parts of a gradient, where a graph calls them by themselves: theirs is refused
    for (const char* part : {"_rms_norm_forward", "_rms_norm_backward", "_rotary_backward", "_attention_forward",
                             "_attention_backward", "_rotary_attention_forward", "_rotary_attention_backward"})
        m.impl(part, torch::autograd::autogradNotImplementedFallback());
}

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    using nogil = py::call_guard<py::gil_scoped_release>;
    m.def("rms_norm", [](const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
        return OP(rms_norm).call(x, weight, residual, eps);
    }, nogil());
    m.def("rms_norm_fp8", [](const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
        return OP(rms_norm_fp8).call(x, weight, residual, eps);
    }, nogil());
    m.def("rotary", [](const Tensor& x, const Tensor& positions, const Tensor& inv_freq,
                       const std::vector<int64_t>& sections, bool interleaved) {
        return OP(rotary).call(x, positions, inv_freq, sections, interleaved);
    }, nogil());
    m.def("attention", [](const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, bool causal,
                          OptDouble scale) { return OP(attention).call(q, k, v, cu, causal, scale); }, nogil());
    m.def("rotary_attention", [](const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions,
                                 const Tensor& inv_freq, const std::vector<int64_t>& sections, const Tensor& cu,
                                 bool interleaved, bool causal, OptDouble scale) {
        return OP(rotary_attention).call(qkv, Hq, Hk, positions, inv_freq, sections, cu, interleaved, causal, scale);
    }, nogil());
    m.def("dropout", [](const Tensor& x, double p, const Tensor& rng, const OptTensor& residual) {
        return OP(dropout).call(x, p, rng, residual);
    }, nogil());
}
