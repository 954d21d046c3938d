// PyTorch side of the token operators: checks of tensors, outputs and
// workspaces from PyTorch's allocator, the current stream, and gradients.
// Python module memory_bound_cnn_amd._tokens; memory_bound_cnn_amd/tokens.py
// documents what it offers.
//
// The gradients are C++ nodes because a backward pass runs on a thread of
// PyTorch's own: with Python nodes a step of a small norm spent 128 us on the
// host, two thirds of it there.
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/extension.h>

#include <cmath>
#include <limits>
#include <optional>
#include <tuple>
#include <vector>

#include "../../include/wtconv_tokens.h"

namespace {

using torch::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;

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

Tensor empty(at::IntArrayRef shape, const Tensor& like) { return at::empty(shape, like.options()); }
Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}
Tensor workspace(size_t bytes, const Tensor& like) {
    return bytes ? empty({(int64_t)bytes}, like, at::kByte) : Tensor();
}

bool dense(const Tensor& t) { return t.stride(-1) == 1 || t.size(-1) <= 1; }

int activation(const Tensor& t, const char* name, int64_t dims) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16, name, " has dtype ",
                      t.scalar_type(), ", expected float32 or bfloat16");
    TORCH_CHECK_VALUE(dims < 0 || t.dim() == dims, name, " has shape ", t.sizes(), ", expected ", dims, " axes");
    return t.scalar_type() == at::kFloat ? WTC_FP32 : WTC_BF16;
}
void check(const Tensor& t, const char* name, at::ScalarType type, const Tensor& like, at::IntArrayRef shape,
           bool contiguous = true) {
    TORCH_CHECK_VALUE(t.device() == like.device(), name, " must be a CUDA tensor on ", like.device());
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " has dtype ", t.scalar_type(), ", expected ", type);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(!contiguous || t.is_contiguous(), name, " must be contiguous");
}
void check_residual(const Tensor& x, const OptTensor& r) {
    if (!r) return;
    TORCH_CHECK_VALUE(r->sizes() == x.sizes(), "residual has shape ", r->sizes(), ", expected ", x.sizes());
    check(*r, "residual", x.scalar_type(), x, x.sizes(), false);
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

struct RmsNorm : torch::autograd::Function<RmsNorm> {
    // Saves the norm's input (h, or x without a residual) and one float per row.
    static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const OptTensor& residual,
                                 double eps) {
        const Rms o = rms_forward(x, weight, residual, eps, true, false);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({residual ? o.h : x, weight, o.rstd});
        if (!residual) return {o.y};
        return {o.y, o.h};
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        const variable_list s = ctx->get_saved_variables();
        const Tensor dh = g.size() > 1 ? g[1] : Tensor();
        if (!g[0].defined()) return {dh, Tensor(), dh, Tensor()};
        const Tensor h = rows(s[0]), dy = rows(g[0]), dhr = dh.defined() ? rows(dh).contiguous() : Tensor();
        const int64_t n = h.size(0);
        const int C = (int)h.size(1);   // as the forward pass took it
        const wtc_rms_desc d = {n, h.stride(0), 0, dy.stride(0), C, h.scalar_type() == at::kFloat ? WTC_FP32 : WTC_BF16,
                                0, 0.f};
        const size_t bytes = wtconv_rms_norm_backward_workspace(&d);
        const Tensor dx = empty(s[0].sizes(), h), dw = empty({C}, h, at::kFloat), ws = workspace(bytes, h);
        const On on(h);
        raise_on(wtconv_rms_norm_backward(&d, in(dy), in(dhr), in(h), in_as<float>(s[1]), in_as<float>(s[2]), out(dx),
                                          static_cast<float*>(out(dw)), out(ws), bytes, on.stream),
                 "wtconv_rms_norm_backward");
        return {dx, dw, g.size() > 1 ? dx : Tensor(), Tensor()};
    }
};

std::tuple<Tensor, OptTensor> rms_norm(const Tensor& x, const Tensor& weight, const OptTensor& residual, double eps) {
    refuse_tangents(x, weight, residual);
    if (wants_grad(x, weight) || wants_grad_opt(residual)) {
        const variable_list o = RmsNorm::apply(x, weight, residual, eps);
        return {o[0], residual ? OptTensor(o[1]) : std::nullopt};
    }
    const Rms o = rms_forward(x, weight, residual, eps, false, false);
    return {o.y, residual ? OptTensor(o.h) : std::nullopt};
}

std::tuple<Tensor, Tensor, OptTensor> rms_norm_fp8(const Tensor& x, const Tensor& weight, const OptTensor& residual,
                                                   double eps) {
    refuse_tangents(x, weight, residual);
    TORCH_CHECK_VALUE(!wants_grad(x, weight) && !wants_grad_opt(residual),
                      "rms_norm_fp8 has no gradient; call it under torch.no_grad()");
    const Rms o = rms_forward(x, weight, residual, eps, false, true);
    return {o.y, o.scale, residual ? OptTensor(o.h) : std::nullopt};
}

// ------------------------------------------------------------------ rotary positions
void rotary_run(const Tensor& x, const Tensor& y, const Tensor& positions, const Tensor& inv_freq,
                const std::vector<int64_t>& sections, bool interleaved, bool inverse) {
    wtc_rotary_desc d = {x.size(0), x.stride(0), x.stride(1), y.stride(0), y.stride(1), (int)x.size(1), (int)x.size(2),
                         x.scalar_type() == at::kFloat ? WTC_FP32 : WTC_BF16, (int)sections.size(), {}, interleaved,
                         inverse};
    for (size_t i = 0; i < sections.size(); ++i) d.pairs[i] = (int)sections[i];
    const On on(x);
    raise_on(wtconv_rotary(&d, in(x), in_as<int>(positions), in_as<float>(inv_freq), out(y), on.stream),
             "wtconv_rotary");
}
void rotary_check(const Tensor& x, const Tensor& positions, const Tensor& inv_freq,
                  const std::vector<int64_t>& sections) {
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
Tensor rotary_forward(const Tensor& x, const Tensor& positions, const Tensor& inv_freq,
                      const std::vector<int64_t>& sections, bool interleaved, bool inverse) {
    const Tensor xd = dense(x) ? x : x.contiguous(), y = empty(x.sizes(), x);
    rotary_run(xd, y, positions, inv_freq, sections, interleaved, inverse);
    return y;
}

struct Rotary : torch::autograd::Function<Rotary> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& positions, const Tensor& inv_freq,
                          std::vector<int64_t> sections, bool interleaved) {
        ctx->save_for_backward({positions, inv_freq});
        ctx->saved_data["sections"] = sections;
        ctx->saved_data["interleaved"] = interleaved;
        return rotary_forward(x, positions, inv_freq, sections, interleaved, false);
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, true);
        const variable_list s = ctx->get_saved_variables();
        return {rotary_forward(g[0], s[0], s[1], ctx->saved_data["sections"].toIntVector(),
                               ctx->saved_data["interleaved"].toBool(), true),
                Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

Tensor rotary(const Tensor& x, const Tensor& positions, const Tensor& inv_freq, std::vector<int64_t> sections,
              bool interleaved) {
    refuse_tangents(x, inv_freq);
    rotary_check(x, positions, inv_freq, sections);
    if (wants_grad(x)) return Rotary::apply(x, positions, inv_freq, sections, interleaved);
    return rotary_forward(x, positions, inv_freq, sections, interleaved, false);
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
    double scale;
};
wtc_attn_desc attn_desc(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, const Setting& s) {
    wtc_attn_desc d = {};
    d.T = q.size(0);
    d.n_seq = sequences(cu);
    d.Hq = (int)q.size(1);
    d.Hk = (int)k.size(1);
    d.D = (int)q.size(2);
    d.dtype = q.scalar_type() == at::kFloat ? WTC_FP32 : WTC_BF16;
    d.causal = s.causal;
    d.scale = (float)s.scale;
    d.q = strides(q);
    d.k = strides(k);
    d.v = strides(v);
    return d;
}
void attn_check(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu) {
    activation(q, "q", 3);
    narrow(q.size(1), "heads of q");
    narrow(q.size(2), "channels of a head of q");
    const int64_t Hk = k.dim() == 3 ? k.size(1) : 0;
    check(k, "k", q.scalar_type(), q, {q.size(0), Hk, q.size(2)}, false);
    check(v, "v", q.scalar_type(), q, {q.size(0), Hk, q.size(2)}, false);
    TORCH_CHECK_VALUE(Hk >= 1 && q.size(1) % Hk == 0, q.size(1), " heads of q do not divide into ", Hk, " of k and v");
    sequences(cu);
    check(cu, "cu_seqlens", at::kInt, q, cu.sizes());
}
struct AttnOut {
    Tensor o, lse, low;   // lse, low: kept for the backward pass (low: what was rounded off o, bfloat16)
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
void attn_backward(const Tensor& q, const Tensor& k, const Tensor& v, const AttnOut& f, const Tensor& g,
                   const Tensor& cu, const Setting& s, const Tensor& dq, const Tensor& dk, const Tensor& dv) {
    wtc_attn_desc d = attn_desc(q, k, v, cu, s);
    d.o = strides(f.o);
    d.g = strides(g);
    d.dq = strides(dq);
    d.dk = strides(dk);
    d.dv = strides(dv);
    const size_t bytes = wtconv_attention_backward_workspace(&d);
    const Tensor ws = workspace(bytes, q);
    const On on(q);
    raise_on(wtconv_attention_backward(&d, in(q), in(k), in(v), in(f.o), in_as<float>(f.lse), in(f.low), in(g), in_as<int>(cu),
                                       out(dq), out(dk), out(dv), out(ws), bytes, on.stream),
             "wtconv_attention_backward");
}

struct Attention : torch::autograd::Function<Attention> {
    // Saves its inputs, its output (with what was rounded off it) and one float per query and head.
    static Tensor forward(AutogradContext* ctx, const Tensor& q0, const Tensor& k0, const Tensor& v0, const Tensor& cu,
                          bool causal, double scale) {
        const Tensor q = heads(q0), k = heads(k0), v = heads(v0);
        const AttnOut f = attn_forward(q, k, v, cu, {causal, scale}, true);
        ctx->save_for_backward({q, k, v, f.o, f.lse, f.low, cu});
        ctx->saved_data["causal"] = causal;
        ctx->saved_data["scale"] = scale;
        return f.o;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        const variable_list s = ctx->get_saved_variables();
        const Tensor dq = empty(s[0].sizes(), s[0]), dk = empty(s[1].sizes(), s[0]), dv = empty(s[2].sizes(), s[0]);
        attn_backward(s[0], s[1], s[2], {s[3], s[4], s[5]}, heads(g[0]), s[6],
                      {ctx->saved_data["causal"].toBool(), ctx->saved_data["scale"].toDouble()}, dq, dk, dv);
        return {dq, dk, dv, Tensor(), Tensor(), Tensor()};
    }
};

double scale_of(std::optional<double> scale, const Tensor& q) {
    return scale ? *scale : 1.0 / std::sqrt((double)q.size(2));
}

Tensor attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, bool causal,
                 std::optional<double> scale) {
    refuse_tangents(q, k, v);
    attn_check(q, k, v, cu);
    const double s = scale_of(scale, q);
    if (wants_grad(q, k, v)) return Attention::apply(q, k, v, cu, causal, s);
    return attn_forward(heads(q), heads(k), heads(v), cu, {causal, s}, false).o;
}

// the q and k heads of a projection, turned, and the attention of it
Tensor turned(const Tensor& qkv, int64_t n, const Tensor& positions, const Tensor& inv_freq,
              const std::vector<int64_t>& sections, bool interleaved) {
    const Tensor qk = empty({qkv.size(0), n, qkv.size(2)}, qkv);
    rotary_run(qkv.narrow(1, 0, n), qk, positions, inv_freq, sections, interleaved, false);
    return qk;
}
AttnOut turned_forward(const Tensor& qkv, const Tensor& qk, int64_t Hq, int64_t Hk, const Tensor& cu, const Setting& s,
                       bool keep) {
    return attn_forward(qk.narrow(1, 0, Hq), qk.narrow(1, Hq, Hk), qkv.narrow(1, Hq + Hk, Hk), cu, s, keep);
}

struct RotaryAttention : torch::autograd::Function<RotaryAttention> {
    // rotary on q and k, then attention, on one projection: the gradients are
    // written where the projection's are wanted, and turned back there.
    static Tensor forward(AutogradContext* ctx, const Tensor& qkv0, int64_t Hq, int64_t Hk, const Tensor& positions,
                          const Tensor& inv_freq, std::vector<int64_t> sections, const Tensor& cu, bool interleaved,
                          bool causal, double scale) {
        const Tensor qkv = heads(qkv0), qk = turned(qkv, Hq + Hk, positions, inv_freq, sections, interleaved);
        const AttnOut f = turned_forward(qkv, qk, Hq, Hk, cu, {causal, scale}, true);
        ctx->save_for_backward({qkv, qk, f.o, f.lse, f.low, cu, positions, inv_freq});
        ctx->saved_data["Hq"] = Hq;
        ctx->saved_data["Hk"] = Hk;
        ctx->saved_data["sections"] = sections;
        ctx->saved_data["interleaved"] = interleaved;
        ctx->saved_data["causal"] = causal;
        ctx->saved_data["scale"] = scale;
        return f.o;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        const variable_list s = ctx->get_saved_variables();
        auto& at = ctx->saved_data;
        const int64_t Hq = at["Hq"].toInt(), Hk = at["Hk"].toInt();
        const Tensor &qkv = s[0], &qk = s[1];
        const Tensor d = empty(qkv.sizes(), qkv), dqk = d.narrow(1, 0, Hq + Hk);
        attn_backward(qk.narrow(1, 0, Hq), qk.narrow(1, Hq, Hk), qkv.narrow(1, Hq + Hk, Hk), {s[2], s[3], s[4]},
                      heads(g[0]), s[5], {at["causal"].toBool(), at["scale"].toDouble()}, d.narrow(1, 0, Hq), d.narrow(1, Hq, Hk),
                      d.narrow(1, Hq + Hk, Hk));
        rotary_run(dqk, dqk, s[6], s[7], at["sections"].toIntVector(), at["interleaved"].toBool(), true);
        variable_list r(10);
        r[0] = d;
        return r;
    }
};

Tensor rotary_attention(const Tensor& qkv, int64_t Hq, int64_t Hk, const Tensor& positions, const Tensor& inv_freq,
                        std::vector<int64_t> sections, const Tensor& cu, bool interleaved, bool causal,
                        std::optional<double> scale) {
    refuse_tangents(qkv, inv_freq);
    TORCH_CHECK_VALUE(Hq >= 1 && Hk >= 1 && Hq % Hk == 0, Hq, " heads of q do not divide into ", Hk, " of k and v");
    activation(qkv, "qkv", 3);
    TORCH_CHECK_VALUE(qkv.size(1) == Hq + 2 * Hk, "qkv has ", qkv.size(1), " heads, expected ", Hq + 2 * Hk);
    rotary_check(qkv, positions, inv_freq, sections);
    sequences(cu);
    check(cu, "cu_seqlens", at::kInt, qkv, cu.sizes());
    const double s = scale_of(scale, qkv);
    if (wants_grad(qkv))
        return RotaryAttention::apply(qkv, Hq, Hk, positions, inv_freq, sections, cu, interleaved, causal, s);
    const Tensor x = heads(qkv);
    return turned_forward(x, turned(x, Hq + Hk, positions, inv_freq, sections, interleaved), Hq, Hk, cu, {causal, s},
                          false).o;
}

// ------------------------------------------------------------------ dropout
Tensor dropout_forward(const Tensor& x, double p, const Tensor& rng, const Tensor& residual) {
    const Tensor xc = x.contiguous(), rc = residual.defined() ? residual.contiguous() : Tensor(), y = empty(x.sizes(), x);
    const On on(x);
    raise_on(wtconv_dropout(x.numel(), x.scalar_type() == at::kFloat ? WTC_FP32 : WTC_BF16, p, in(xc), in(rc),
                            static_cast<const unsigned long long*>(in(rng)), out(y), on.stream),
             "wtconv_dropout");
    return y;
}

struct Dropout : torch::autograd::Function<Dropout> {
    // Saves the generator's two words; the decisions are drawn again.
    static Tensor forward(AutogradContext* ctx, const Tensor& x, double p, const Tensor& rng, const OptTensor& residual) {
        ctx->save_for_backward({rng});
        ctx->saved_data["p"] = p;
        ctx->saved_data["residual"] = residual.has_value();
        return dropout_forward(x, p, rng, residual.value_or(Tensor()));
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, true);
        Tensor dx;
        if (ctx->needs_input_grad(0))
            dx = dropout_forward(g[0], ctx->saved_data["p"].toDouble(), ctx->get_saved_variables()[0], Tensor());
        return {dx, Tensor(), Tensor(), ctx->saved_data["residual"].toBool() ? g[0] : Tensor()};
    }
};

Tensor dropout(const Tensor& x, double p, const Tensor& rng, const OptTensor& residual) {
    refuse_tangents(x, residual);
    activation(x, "x", -1);
    check_residual(x, residual);
    check(rng, "rng", at::kLong, x, {2});
    TORCH_CHECK_VALUE(p >= 0.0 && p <= 1.0, "p = ", p, " is no probability");
    if (wants_grad(x) || wants_grad_opt(residual)) return Dropout::apply(x, p, rng, residual);
    return dropout_forward(x, p, rng, residual.value_or(Tensor()));
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    using nogil = py::call_guard<py::gil_scoped_release>;
    m.def("rms_norm", &rms_norm, nogil());
    m.def("rms_norm_fp8", &rms_norm_fp8, nogil());
    m.def("rotary", &rotary, nogil());
    m.def("attention", &attention, nogil());
    m.def("rotary_attention", &rotary_attention, nogil());
    m.def("dropout", &dropout, nogil());
}
