// Host side of the token operators: argument checks and dispatch.  See
// include/wtconv_tokens.h for the contract.
#include <cmath>
#include <initializer_list>

#include "wtc_tok_internal.h"

namespace wtc {
namespace {

constexpr long long kMaxTokens = 1LL << 31;   // token and row indices are 32-bit in the kernels

bool is_dtype(int t) { return t == WTC_FP32 || t == WTC_BF16; }
int elem_bytes(int t) { return t == WTC_BF16 ? 2 : 4; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

int check_rms(const wtc_rms_desc* d) {
    if (!d) return WTC_EINVAL;
    if (d->rows < 0 || d->C < 1 || !(d->eps >= 0.f) || std::isinf(d->eps)) return WTC_EINVAL;
    if (d->x_stride < 0 || d->r_stride < 0 || d->g_stride < 0) return WTC_EINVAL;
    if (!is_dtype(d->dtype) || (d->fp8 != 0 && d->fp8 != 1)) return WTC_EDTYPE;
    if (d->C > WTC_RMS_MAX_C || d->rows >= kMaxTokens) return WTC_ESHAPE;
    return WTC_OK;
}

int check_rotary(const wtc_rotary_desc* d) {
    if (!d) return WTC_EINVAL;
    if (d->T < 0 || d->heads < 1 || d->D < 1) return WTC_EINVAL;
    if (d->axes < 1 || d->axes > WTC_ROTARY_MAX_AXES) return WTC_EINVAL;
    if (d->x_token < 0 || d->x_head < 0 || d->y_token < 0 || d->y_head < 0) return WTC_EINVAL;
    if ((d->interleaved != 0 && d->interleaved != 1) || (d->inverse != 0 && d->inverse != 1)) return WTC_EINVAL;
    if (!is_dtype(d->dtype)) return WTC_EDTYPE;
    long long P = 0;
    for (int a = 0; a < d->axes; ++a) {
        if (d->pairs[a] < 0) return WTC_EINVAL;
        P += d->pairs[a];
    }
    if (2 * P > d->D) return WTC_ESHAPE;
    if (d->T >= kMaxTokens || d->D > 65536 || d->heads > 65535) return WTC_ESHAPE;
    return WTC_OK;
}

int check_attn(const wtc_attn_desc* d) {
    if (!d) return WTC_EINVAL;
    if (d->T < 0 || d->n_seq < 0 || d->Hq < 1 || d->Hk < 1 || d->Hq % d->Hk != 0 || d->D < 1) return WTC_EINVAL;
    if ((d->causal != 0 && d->causal != 1) || !std::isfinite(d->scale)) return WTC_EINVAL;
    if (!is_dtype(d->dtype)) return WTC_EDTYPE;
    if (d->D % 8 != 0 || d->D > WTC_ATTN_MAX_D) return WTC_ESHAPE;
    if (d->T >= kMaxTokens || d->n_seq > (1 << 24) || d->Hq > 65535) return WTC_ESHAPE;
    return WTC_OK;
}

// 16-byte loads: tensors, tokens and heads start at multiples of 16 bytes; a
// tile's 64 rows are addressed with 32 bits
int check_strides(const wtc_attn_desc* d, const wtc_attn_strides& s, const void* p) {
    const int unit = 16 / elem_bytes(d->dtype);
    if (s.token < 0 || s.head < 0 || s.token % unit != 0 || s.head % unit != 0 || !aligned(p, 16)) return WTC_EINVAL;
    return s.token > WTC_ATTN_MAX_TOKEN_STRIDE ? WTC_ESHAPE : WTC_OK;
}

int check_low(const wtc_attn_desc* d, const void* low) {
    if (!low) return WTC_OK;
    return d->dtype != WTC_BF16 ? WTC_EDTYPE : aligned(low, 16) ? WTC_OK : WTC_EINVAL;
}

int first_error(std::initializer_list<int> all) {
    for (int s : all)
        if (s != WTC_OK) return s;
    return WTC_OK;
}

}  // namespace
}  // namespace wtc

using namespace wtc;

extern "C" {

int wtconv_rms_norm_forward(const wtc_rms_desc* d, const void* x, const void* residual, const float* weight, void* y,
                            void* h, float* rstd, float* scale, void* stream) {
    const int st = check_rms(d);
    if (st != WTC_OK) return st;
    if ((d->fp8 != 0) != (scale != nullptr) || (residual != nullptr) != (h != nullptr)) return WTC_EINVAL;
    if (d->rows == 0) return WTC_OK;
    if (!x || !weight || !y) return WTC_EINVAL;
    return launch_rms_forward(d, x, residual, weight, y, h, rstd, scale, stream);
}

size_t wtconv_rms_norm_backward_workspace(const wtc_rms_desc* d) {
    if (check_rms(d) != WTC_OK || d->fp8) return 0;
    return (size_t)rms_backward_parts(d) * d->C * sizeof(float);
}

int wtconv_rms_norm_backward(const wtc_rms_desc* d, const void* dy, const void* dh, const void* h, const float* weight,
                             const float* rstd, void* dx, float* dw, void* workspace, size_t workspace_bytes,
                             void* stream) {
    const int st = check_rms(d);
    if (st != WTC_OK) return st;
    if (d->fp8) return WTC_EDTYPE;
    if (!weight || !dw) return WTC_EINVAL;
    if (d->rows > 0 && (!dy || !h || !rstd || !dx)) return WTC_EINVAL;
    const size_t need = wtconv_rms_norm_backward_workspace(d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WTC_EWORKSPACE;
    return launch_rms_backward(d, dy, dh, h, weight, rstd, dx, dw, static_cast<float*>(workspace), stream);
}

int wtconv_rotary(const wtc_rotary_desc* d, const void* x, const int* positions, const float* inv_freq, void* y,
                  void* stream) {
    const int st = check_rotary(d);
    if (st != WTC_OK) return st;
    if (d->T == 0) return WTC_OK;
    int P = 0;
    for (int a = 0; a < d->axes; ++a) P += d->pairs[a];
    if (!x || !y || (P > 0 && (!positions || !inv_freq))) return WTC_EINVAL;
    return launch_rotary(d, x, positions, inv_freq, y, stream);
}

int wtconv_dropout(long long n, int dtype, double p, const void* x, const void* residual,
                   const unsigned long long* rng, void* y, void* stream) {
    if (n < 0 || !(p >= 0.0 && p <= 1.0)) return WTC_EINVAL;
    if (!is_dtype(dtype)) return WTC_EDTYPE;
    if (n == 0) return WTC_OK;
    if (!x || !rng || !y) return WTC_EINVAL;
    return launch_dropout(n, dtype, (unsigned)std::nearbyint(p * 65536.0), x, residual, rng, y, stream);
}

size_t wtconv_attention_forward_workspace(const wtc_attn_desc* d) {
    if (check_attn(d) != WTC_OK) return 0;
    return attn_forward_bytes(d);
}

int wtconv_attention_forward(const wtc_attn_desc* d, const void* q, const void* k, const void* v,
                             const int* cu_seqlens, void* out, float* lse, void* out_low, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const int st = check_attn(d);
    if (st != WTC_OK) return st;
    if (d->T == 0) return WTC_OK;
    if (!q || !k || !v || !cu_seqlens || !out) return WTC_EINVAL;
    const int bad = first_error({check_strides(d, d->q, q), check_strides(d, d->k, k), check_strides(d, d->v, v),
                                 check_strides(d, d->o, out), check_low(d, out_low)});
    if (bad != WTC_OK) return bad;
    const size_t need = attn_forward_bytes(d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WTC_EWORKSPACE;
    return launch_attn_forward(d, q, k, v, cu_seqlens, out, lse, out_low, workspace, stream);
}

size_t wtconv_attention_backward_workspace(const wtc_attn_desc* d) {
    if (check_attn(d) != WTC_OK) return 0;
    return attn_backward_bytes(d);
}

int wtconv_attention_backward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const void* out,
                              const float* lse, const void* out_low, const void* dout, const int* cu_seqlens,
                              void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_attn(d);
    if (st != WTC_OK) return st;
    if (d->T == 0) return WTC_OK;
    if (!q || !k || !v || !out || !lse || !dout || !cu_seqlens || !dq || !dk || !dv) return WTC_EINVAL;
    const int bad = first_error({check_strides(d, d->q, q), check_strides(d, d->k, k), check_strides(d, d->v, v),
                                 check_strides(d, d->o, out), check_strides(d, d->g, dout), check_strides(d, d->dq, dq),
                                 check_strides(d, d->dk, dk), check_strides(d, d->dv, dv), check_low(d, out_low)});
    if (bad != WTC_OK) return bad;
    if (!workspace || workspace_bytes < wtconv_attention_backward_workspace(d)) return WTC_EWORKSPACE;
    return launch_attn_backward(d, q, k, v, out, lse, out_low, dout, cu_seqlens, dq, dk, dv, workspace, stream);
}

}  // extern "C"
