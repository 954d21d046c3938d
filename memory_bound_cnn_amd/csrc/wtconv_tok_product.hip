// The experts' products: launches.  The kernels are wtc_tok_product_kernels.h,
// compiled for each type by wtconv_tok_product_bf16.hip and _fp32.hip.
#include <hip/hip_runtime.h>

#include "wtc_tok_product_launch.h"

namespace wtc {
namespace {

// Workgroups that share the rows of one tile of dW: to about 768 of them, which also evens out experts of unequal size,
// if each has 1024 rows (float32: 171, of six products) to pay for the partial sums' way through memory.  Measured (us, 8
// experts, whole / in 2 / in 3 / in 4): 512 tiles bfloat16, 12544 rows 49.5 / 53.0, 16384 63.1 / 60.3 / 68, 32768 121 / 93.7 /
// 99.6 / 126, 50176 186 / 147 / 158 / 165; 768 tiles, 25000 rows of 4 experts 159 / 205; 1024 tiles, 100000 rows 488 / 485 /
// 507; 256 tiles float32, 2048 rows 39.1 / 34.0 / 37.4, 6007 94.9 / 62.5 / 55.3 / 58.5, 12544 188 / 112 / 92.4 / 94.4.
int splits_of(const wtc_expert_desc* d) {
    const long long tiles = (long long)d->E * ((d->K + 127) / 128) * ((d->N + 127) / 128);
    const long long most = d->R / d->E * (d->dtype == WTC_BF16 ? 1 : 6) / 1024, want = (768 + tiles / 2) / tiles;
    return (int)(want < most ? (want < 1 ? 1 : want) : most < 1 ? 1 : most);
}

product::Args args_of(const wtc_expert_desc* d, const int* cu) {
    product::Args a = {};
    a.cu = cu;
    a.R = (int)d->R; a.E = d->E; a.K = d->K; a.N = d->N; a.splits = 1;
    a.x_stride = d->x_stride; a.g_stride = d->g_stride;
    return a;
}

}  // namespace

size_t expert_weights_workspace(const wtc_expert_desc* d) {
    const int s = splits_of(d);
    return s > 1 ? (size_t)s * d->E * ((size_t)d->N * d->K + d->N) * sizeof(float) : 0;
}

int launch_expert_forward(const wtc_expert_desc* d, const void* x, const void* w, const void* b, const int* cu, void* y,
                          void* stream) {
    product::Args a = args_of(d, cu);
    a.x = x; a.w = w; a.b = b; a.y = y;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? product::rows_bf16(a, false, st) : product::rows_fp32(a, false, st);
}
int launch_expert_input_grad(const wtc_expert_desc* d, const void* dy, const void* w, const int* cu, void* dx, void* stream) {
    product::Args a = args_of(d, cu);
    a.x = dy; a.x_stride = d->g_stride; a.w = w; a.y = dx;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? product::rows_bf16(a, true, st) : product::rows_fp32(a, true, st);
}
int launch_expert_weight_grad(const wtc_expert_desc* d, const void* dy, const void* x, const int* cu, void* dw, void* db,
                              void* workspace, void* stream) {
    product::Args a = args_of(d, cu);
    a.x = x; a.g = dy; a.y = dw; a.db = db; a.splits = splits_of(d); a.parts = static_cast<float*>(workspace);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? product::weights_bf16(a, st) : product::weights_fp32(a, st);
}

}  // namespace wtc
