// The experts' products: launches.  The kernels are wtc_tok_product_kernels.h,
// compiled for each type by wtconv_tok_product_bf16.hip and _fp32.hip.
#include <hip/hip_runtime.h>
#include <limits.h>

#include "wtc_tok_product_launch.h"

namespace wtc {
namespace {

// How the weights' gradients are shared out: tiles of 256 x 256 or of 128 x 128, and the rows of a part of an expert (see
// find_part): as many as leave a part to every place on the chip, and enough to pay for the partial sums' way through memory.
// Measured (us; 8 experts of bfloat16 unless said): experts whole, and in parts of 1/2, 1 and 3/2 of those rows; first experts
// of equal size, then one with two thirds of all rows.
//   128 x 128: 12544 rows x 512 -> 2048 35.5, 61, 37, 39 and 87, 51, 44, 44; float32 12544 x 512 -> 1024 95, 100, 92, 91 and
// 439, 108, 96, 102; 4 experts 30000 x 256 -> 256 401, 56, 47, 50 and 1398, 77, 62, 61.
//   256 x 256: 50176 x 1024 -> 4096 359, 359, 362, 361 and 729, 403, 393, 432; x 1024 -> 1024 147, 161, 118, 118 and 689, 168,
// 146, 139; 4 experts 25088 x 1024 -> 2048 141, 138, 113, 114 and 465, 152, 126, 130.
//   256 x 256 against 128 x 128, in parts of those rows: 50176 x 1024 -> 4096 362 and 458, 1024 -> 1024 118 and 147, 4 experts
// 100000 x 512 -> 512 (1562 rows a place) 84 and 106; 12544 x 512 -> 2048 (784) 54 and 37, 64 experts 8192 x 512 -> 1024 (256)
// 33 and 33.
struct Share {
    bool large;
    int rows;
    long long places;   // for sums of parts
};
Share share_of(const wtc_expert_desc* d) {
    auto tiles = [&](int side) { return (long long)((d->K + side - 1) / side) * ((d->N + side - 1) / side); };
    const bool wide = d->dtype != WTC_BF16;
    Share s;
    s.large = !wide && 3 * tiles(256) < tiles(128) && d->R * tiles(256) >= 256 * 1280;
    const long long each = s.large ? d->R * tiles(256) / 256 : d->R * tiles(128) / 512, least = wide ? 192 : 1024;
    s.rows = (int)(each < least ? least : each > INT_MAX / 2 ? INT_MAX / 2 : (each + 63) / 64 * 64);
    s.places = product::most_places(d->R, s.rows);
    return s;
}

product::Args args_of(const wtc_expert_desc* d, const int* cu) {
    product::Args a = {};
    a.cu = cu;
    a.R = (int)d->R; a.E = d->E; a.K = d->K; a.N = d->N;
    a.x_stride = d->x_stride; a.g_stride = d->g_stride;
    return a;
}

}  // namespace

size_t expert_weights_workspace(const wtc_expert_desc* d) {
    return (size_t)share_of(d).places * ((size_t)d->N * d->K + d->N) * sizeof(float);
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
    a.x = x; a.g = dy; a.y = dw; a.db = db; a.parts = static_cast<float*>(workspace);
    const Share s = share_of(d);
    a.rows = s.rows; a.slots = s.places;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? product::weights_bf16(a, s.large, st) : product::weights_fp32(a, false, st);
}

}  // namespace wtc
