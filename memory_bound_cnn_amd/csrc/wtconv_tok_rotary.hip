// Rotary positions with several axes: pair p of token t, of axis a, is turned
// by the angle pos[t, a] f[p]:  (u, v) -> (u cos - v sin, u sin + v cos).
//
// The bound is device memory (2 N e bytes): the angles' sines and cosines
// (some 40 operations a pair) are computed once per token and kept in
// registers while a thread goes over the heads, instead of being read from
// tables.  A thread takes the pairs of one 16-byte vector: kVec pairs whose
// halves lie P apart, or kVec / 2 neighbouring pairs; channels past the pairs
// are copied by further threads.  Heads are split over blockIdx.y where tokens
// alone do not fill the chip.  25088 tokens x 12 heads of 64 bfloat16 16.8 us (4.6
// TB/s), 65537 x 10 of 128 float32 with three axes 129 us (5.2 TB/s).
#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace {

struct RotaryArgs {
    const void* x;
    void* y;
    const int* pos;
    const float* freq;
    long long T, x_token, x_head, y_token, y_head;
    int heads, D, P, axes;
    int ends[WTC_ROTARY_MAX_AXES];   // first pair after each axis
    int units, pair_units;           // threads of a token; those that turn pairs
    int heads_per_block;
    float sign;                      // -1: the inverse rotation
};

__device__ __forceinline__ void angle_of(const RotaryArgs& a, long long t, int p, float& c, float& s) {
    int axis = 0;
#pragma unroll
    for (int i = 0; i < WTC_ROTARY_MAX_AXES - 1; ++i)
        if (i + 1 < a.axes && p >= a.ends[i]) axis = i + 1;
    sincosf((float)a.pos[t * a.axes + axis] * a.freq[p], &s, &c);
    s *= a.sign;
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(256) k_rotary(RotaryArgs a) {
    constexpr int V = kVec<T>;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long t = id / a.units;
    const int unit = (int)(id - t * a.units);
    if (t >= a.T) return;
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.heads, h0 + a.heads_per_block);
    const T* x = static_cast<const T*>(a.x) + t * a.x_token + h0 * a.x_head;
    T* y = static_cast<T*>(a.y) + t * a.y_token + h0 * a.y_head;
    if (unit >= a.pair_units) {   // channels that no pair holds
        const int c = 2 * a.P + (unit - a.pair_units) * V;
        for (int h = h0; h < h1; ++h, x += a.x_head, y += a.y_head) {
            float v[V];
            load_part(x + c, a.D - c, v);
            store_part(y + c, a.D - c, v);
        }
        return;
    }
    if constexpr (INTERLEAVED) {
        const int c0 = unit * V, n = 2 * a.P - c0;
        float c[V / 2], s[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            c[i] = s[i] = 0.f;
            if (2 * i < n) angle_of(a, t, c0 / 2 + i, c[i], s[i]);
        }
        x += c0;
        y += c0;
#pragma unroll 4
        for (int h = h0; h < h1; ++h, x += a.x_head, y += a.y_head) {
            float v[V], o[V];
            load_part(x, n, v);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                o[2 * i] = v[2 * i] * c[i] - v[2 * i + 1] * s[i];
                o[2 * i + 1] = v[2 * i] * s[i] + v[2 * i + 1] * c[i];
            }
            store_part(y, n, o);
        }
    } else {
        const int p0 = unit * V, n = a.P - p0;
        float c[V], s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = s[i] = 0.f;
            if (i < n) angle_of(a, t, p0 + i, c[i], s[i]);
        }
        x += p0;
        y += p0;
#pragma unroll 4
        for (int h = h0; h < h1; ++h, x += a.x_head, y += a.y_head) {
            float u[V], v[V], ou[V], ov[V];
            load_part(x, n, u);
            load_part(x + a.P, n, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ou[i] = u[i] * c[i] - v[i] * s[i];
                ov[i] = u[i] * s[i] + v[i] * c[i];
            }
            store_part(y, n, ou);
            store_part(y + a.P, n, ov);
        }
    }
}

}  // namespace

int launch_rotary(const wtc_rotary_desc* d, const void* x, const int* pos, const float* inv_freq, void* y,
                  void* stream) {
    RotaryArgs a = {};
    a.x = x; a.y = y; a.pos = pos; a.freq = inv_freq;
    a.T = d->T; a.x_token = d->x_token; a.x_head = d->x_head; a.y_token = d->y_token; a.y_head = d->y_head;
    a.heads = d->heads; a.D = d->D; a.axes = d->axes;
    for (int i = 0; i < d->axes; ++i) a.ends[i] = a.P += d->pairs[i];
    a.sign = d->inverse ? -1.f : 1.f;
    const int V = d->dtype == WTC_BF16 ? kVec<uint16_t> : kVec<float>;
    const int per = d->interleaved ? V / 2 : V;   // pairs of a thread
    a.pair_units = (a.P + per - 1) / per;
    a.units = a.pair_units + (d->D - 2 * a.P + V - 1) / V;
    // 2^31 threads at most along x; heads are split until there are some
    // 4096 waves, 4 on each of the 1024 vector units (12 heads of 64 bfloat16,
    // 196 tokens: 9.0 us whole, 4.5 split; 2000: 9.5, 4.6; 6272: 10.3, 7.8; 25088: 16.4, 16.2)
    const long long blocks = (d->T * a.units + 255) / 256;
    if (blocks > (1LL << 23)) return WTC_ESHAPE;
    const long long splits = 1024 / blocks + 1;
    a.heads_per_block = (int)((d->heads + splits - 1) / splits);
    const dim3 grid((unsigned)blocks, (unsigned)((d->heads + a.heads_per_block - 1) / a.heads_per_block)), block(256);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16) {
        if (d->interleaved)
            hipLaunchKernelGGL((k_rotary<uint16_t, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((k_rotary<uint16_t, false>), grid, block, 0, st, a);
    } else {
        if (d->interleaved)
            hipLaunchKernelGGL((k_rotary<float, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((k_rotary<float, false>), grid, block, 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace wtc
