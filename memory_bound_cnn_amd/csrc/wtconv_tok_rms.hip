// Root-mean-square norm over rows, with the residual's addition:
//   h = round(x + r),  s = 1 / sqrt(mean_c h^2 + eps),  y = h s w
// and its backward pass
//   xh = h s,  u = w dy,  dx = dh + s (u - xh mean_c(u xh)),  dw = sum_rows dy xh.
//
// One pass over the data: a row stays in the registers of a group of G lanes
// (G = 2 .. 64 inside a wave, or a workgroup of 256 or 1024), NV 16-byte
// vectors per lane, between the sum over its channels and the result.  The
// bound is device memory: 4 N e bytes forward with a residual (x, r in, h, y
// out), 4 N e backward (dy, dh, h in, dx out).  Workgroups walk rows in a
// grid-stride loop with the weight (float32, as wide as two bfloat16 rows) in
// registers, so that it is read once per workgroup; the backward pass sums dw
// in registers over those rows, and one record of C floats per workgroup is
// joined in a fixed order by a second kernel.  Rows on their way are held as
// they lie in memory.  Measured, means of 20 training steps: 65536 x 192
// bfloat16 with residual 17.5 us forward (5.8 TB/s; it fits the last-level
// cache) and 19.4 backward, 8192 x 4096 46.5 and 46.9 us (5.8 and 5.7 TB/s),
// 100003 x 387 float32 without 57.6 and 99.2 us (5.4 and 4.7 TB/s), 49 x 768
// 4.6 us.
//
// The norm is of the sum as the residual stream stores it: the backward pass
// then reads h alone, and its gradient is that of what was computed.
#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace {

constexpr float kF8Max = 448.f;             // the largest e4m3 value
constexpr float kF8Least = 0x1p-100f;       // smallest row scale: its inverse is finite

struct RmsArgs {
    const void *x, *r, *dy, *dh;   // x: h in the backward pass
    const float *w, *rstd_in;
    void *y, *h;                   // y: dx in the backward pass
    float *rstd, *scale, *parts;
    long long rows, x_stride, r_stride, g_stride;
    int C;
    float eps, inv_C;
};

// Sum (or maximum) over the G lanes of a row; every lane gets it.  `red`: one
// float per wave for groups wider than a wave (all threads of the workgroup
// call it together).
template <int G, bool MAX>
__device__ __forceinline__ float group_reduce(float v, float* red) {
#pragma unroll
    for (int o = 1; o < (G < 64 ? G : 64); o <<= 1) {
        const float other = __shfl_xor(v, o);
        v = MAX ? fmaxf(v, other) : v + other;
    }
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();   // the previous use of `red` is over
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < G / 64; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
    }
    return v;
}

// Weights of channels c .. c + V - 1, zero past the last one.
template <int V>
__device__ __forceinline__ void load_weight(const RmsArgs& a, int c, float (&w)[V]) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
        float part[4];
        load_part(a.w + c + k, a.C - c - k, part);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k + j] = part[j];
    }
}

template <typename T, int G, int NV>
__global__ void __launch_bounds__(G > 256 ? G : 256) k_rms_forward(RmsArgs a) {
    constexpr int V = kVec<T>, THREADS = G > 256 ? G : 256, RPB = THREADS / G;
    __shared__ float red[16];
    const int lane = threadIdx.x % G, sub = threadIdx.x / G;
    float w[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<V>(a, (lane + i * G) * V, w[i]);
    }
    const long long step = (long long)gridDim.x * RPB;
    Raw<T> xn[NV], rn[NV];   // of the row that comes next
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V, n = row < a.rows ? a.C - c : 0;
            xn[i] = load_raw(static_cast<const T*>(a.x) + row * a.x_stride + c, n);
            if (a.r) rn[i] = load_raw(static_cast<const T*>(a.r) + row * a.r_stride + c, n);
        }
    };
    fetch((long long)blockIdx.x * RPB + sub);
    for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step) {
        const long long row = first + sub;
        const bool live = row < a.rows;   // the same for all lanes of a row, and for a whole workgroup when G > 64
        float h[NV][V], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack(xn[i], h[i]);
            if (a.r) {
                const int c = (lane + i * G) * V, n = live ? a.C - c : 0;
                float r[V];
                unpack(rn[i], r);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = as_stored<T>(h[i][j] + r[j]);
                store_part(static_cast<T*>(a.h) + row * a.C + c, n, h[i]);
            }
        }
        if (first + step < a.rows) fetch(row + step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(h[i][j], h[i][j], ss);
        ss = group_reduce<G, false>(ss, red);
        const float s = 1.f / sqrtf(fmaf(ss, a.inv_C, a.eps));
        if (a.rstd && live && lane == 0) a.rstd[row] = s;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[i][j] = h[i][j] * s * w[i][j];
                amax = fmaxf(amax, fabsf(h[i][j]));
            }
        if (a.scale) {
            amax = group_reduce<G, true>(amax, red);
            const float scale = fmaxf(amax / kF8Max, kF8Least);
            const float inv = 1.f / scale;
            if (live && lane == 0) a.scale[row] = scale;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + i * G) * V, n = live ? a.C - c : 0;
                uint8_t* p = static_cast<uint8_t*>(a.y) + row * a.C + c;
                uint32_t q[V / 4];
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    int u = __builtin_amdgcn_cvt_pk_fp8_f32(h[i][j] * inv, h[i][j + 1] * inv, 0, false);
                    u = __builtin_amdgcn_cvt_pk_fp8_f32(h[i][j + 2] * inv, h[i][j + 3] * inv, u, true);
                    q[j / 4] = (uint32_t)u;
                }
                if (n >= V) {
                    __builtin_memcpy(p, q, V);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (j < n) p[j] = (uint8_t)(q[j / 4] >> (8 * (j % 4)));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + i * G) * V, n = live ? a.C - c : 0;
                store_part(static_cast<T*>(a.y) + row * a.C + c, n, h[i]);
            }
        }
    }
}

template <typename T, int G, int NV>
__global__ void __launch_bounds__(G > 256 ? G : 256) k_rms_backward(RmsArgs a) {
    constexpr int V = kVec<T>, THREADS = G > 256 ? G : 256, RPB = THREADS / G;
    constexpr int WIDTH = G * NV * V;   // >= C
    // The next row is read while this one is worked on, where that leaves three waves on a vector
    // unit, which three vectors do not: 8192 x 4096 bfloat16 48.2 -> 45.7 us
    constexpr bool AHEAD = NV <= 2 && G <= 256;
    __shared__ float red[16];
    __shared__ float join[G <= 64 ? 4 * WIDTH : 1];   // dw sums of the four waves
    const int lane = threadIdx.x % G, sub = threadIdx.x / G;
    float w[NV][V], dw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<V>(a, (lane + i * G) * V, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
    }
    const long long step = (long long)gridDim.x * RPB;
    Raw<T> xn[NV], gn[NV], dn[NV];   // of the row that comes next
    float sn = 0.f;
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V, n = row < a.rows ? a.C - c : 0;
            xn[i] = load_raw(static_cast<const T*>(a.x) + row * a.x_stride + c, n);
            gn[i] = load_raw(static_cast<const T*>(a.dy) + row * a.g_stride + c, n);
            dn[i] = a.dh ? load_raw(static_cast<const T*>(a.dh) + row * a.C + c, n) : Raw<T>{{0u, 0u, 0u, 0u}};
        }
        sn = row < a.rows ? a.rstd_in[row] : 0.f;
    };
    if (AHEAD) fetch((long long)blockIdx.x * RPB + sub);
    for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step) {
        const long long row = first + sub;
        const bool live = row < a.rows;
        if (!AHEAD) fetch(row);
        float xh[NV][V], g[NV][V], along = 0.f;
        Raw<T> dr[NV];
        const float s = sn;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack(xn[i], xh[i]);
            unpack(gn[i], g[i]);
            dr[i] = dn[i];
        }
        if (AHEAD && first + step < a.rows) fetch(row + step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[i][j] *= s;
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                g[i][j] *= w[i][j];
                along = fmaf(g[i][j], xh[i][j], along);
            }
        along = group_reduce<G, false>(along, red) * a.inv_C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V, n = live ? a.C - c : 0;
            float d[V];
            unpack(dr[i], d);
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(s, fmaf(-xh[i][j], along, g[i][j]), d[j]);
            store_part(static_cast<T*>(a.y) + row * a.C + c, n, d);
        }
    }
    // the workgroup's record: rows of a wave by shuffles, then its four waves
    float* rec = a.parts + (size_t)blockIdx.x * a.C;
    if constexpr (G <= 64) {
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int o = G; o < 64; o <<= 1) dw[i][j] += __shfl_xor(dw[i][j], o);
                if ((threadIdx.x & 63) < G) join[wave * WIDTH + (lane + i * G) * V + j] = dw[i][j];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += THREADS)
            rec[c] = (join[c] + join[WIDTH + c]) + (join[2 * WIDTH + c] + join[3 * WIDTH + c]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < a.C) rec[c + j] = dw[i][j];
        }
    }
}

// dw[c] = sum of the records' c, in a fixed order: 32 threads of a column take
// every 32nd record, then their sums are joined.
__global__ void __launch_bounds__(1024) k_rms_join(const float* __restrict__ parts, int n, int C,
                                                   float* __restrict__ dw) {
    __shared__ float sums[32][33];
    const int col = threadIdx.x & 31, part = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
    float v = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int p = part; p < n; p += 32) v += parts[(size_t)p * C + c];
    }
    sums[part][col] = v;
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (part < o) sums[part][col] += sums[part + o][col];
        __syncthreads();
    }
    if (part == 0 && c < C) dw[c] = sums[0][col];
}

// The group of G lanes and the NV vectors per lane for a row of n 16-byte
// vectors: the first of these shapes, in the order of G * NV, that holds it.
// Where two have the same G * NV the wider group stands here (longer runs of
// consecutive addresses).  Those marked `many` leave no lane idle in rows of 24,
// 48 and 96 vectors, and are for forward passes of kManyVectors and more, as
// bfloat16 (without, with the residual): 65536 x 192 9.5 and 16.5 us, 11.4 and
// 17.0 without them, 25088 x 384 8.4 and 13.3, 9.9 and 13.4; but 49 x 768 4.0
// and 5.4, 3.7 and 4.5 without.  Around kManyVectors, 192 channels in a graph:
// 5461 rows (2^17 vectors) 3.8 and 5.2, 3.3 and 4.0 without, 8192 rows 3.5 and
// 4.6, 3.6 and 4.6, 10922 rows 4.1 and 5.8, 4.3 and 5.6, 21845 rows 5.3 and 8.5,
// 5.8 and 7.8, 87381 rows 11.9 and 24.7, 13.4 and 24.8: the two meet between 2^17
// and 2^18 without a residual, and with one do not differ by more than 0.8 us
// from there on.  Nor for the backward pass, whose registers they
// fill: 22.2 us, 18.2 without them, and 18.0, 15.2.
struct RmsShape {
    int G, NV;
    bool many;
};
constexpr long long kManyVectors = 1 << 17;
constexpr RmsShape kRmsShapes[] = {{2, 1, false},    {4, 1, false},    {8, 1, false},   {16, 1, false}, {8, 3, true},
                                   {32, 1, false},   {16, 3, true},    {64, 1, false},  {32, 3, true},  {64, 2, false},
                                   {64, 3, false},   {64, 4, false},   {256, 2, false}, {256, 3, false}, {256, 4, false},
                                   {1024, 2, false}, {1024, 3, false}, {1024, 4, false}};
constexpr int kRmsShapeCount = (int)(sizeof(kRmsShapes) / sizeof(kRmsShapes[0]));
static_assert(1024 * 4 * kVec<float> >= WTC_RMS_MAX_C && 1024 * 2 * kVec<uint16_t> >= WTC_RMS_MAX_C, "the longest row");

int rms_shape(int C, int dtype, long long forward_rows) {
    const int V = dtype == WTC_BF16 ? kVec<uint16_t> : kVec<float>;
    const bool many = forward_rows * ((C + V - 1) / V) >= kManyVectors;
    int i = 0;
    while (kRmsShapes[i].G * kRmsShapes[i].NV * V < C || (kRmsShapes[i].many && !many)) ++i;
    return i;
}

// f<T, G, NV>() for shape number `at`; shapes past the longest row of T are
// not compiled.
template <typename T, int I = 0, typename F>
void rms_dispatch(int at, const F& f) {
    if (at == I) f.template operator()<T, kRmsShapes[I].G, kRmsShapes[I].NV>();
    if constexpr (I + 1 < kRmsShapeCount)
        if constexpr (kRmsShapes[I].G * kRmsShapes[I].NV * kVec<T> < WTC_RMS_MAX_C) rms_dispatch<T, I + 1>(at, f);
}

struct ForwardLaunch {
    const RmsArgs& a;
    hipStream_t st;
    template <typename T, int G, int NV>
    void operator()() const {
        constexpr int threads = G > 256 ? G : 256, rpb = threads / G;
        // what fits at once: the next row is then read ahead (65536 x 192 bfloat16 16.5 us, 17.4 with
        // 2048 workgroups; 200000 x 96, with fewer registers, 28.6 and 26.7)
        const long long blocks = (a.rows + rpb - 1) / rpb, cap = threads > 256 ? 512 : NV > 1 ? 1024 : 2048;
        hipLaunchKernelGGL((k_rms_forward<T, G, NV>), dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(threads), 0,
                           st, a);
    }
};
struct BackwardLaunch {
    const RmsArgs& a;
    hipStream_t st;
    int parts;
    template <typename T, int G, int NV>
    void operator()() const {
        if constexpr (G >= 64 || NV == 1)   // the others are for the forward pass
            hipLaunchKernelGGL((k_rms_backward<T, G, NV>), dim3((unsigned)parts), dim3(G > 256 ? G : 256), 0, st, a);
    }
};

}  // namespace

int rms_backward_parts(const wtc_rms_desc* d) {
    const int G = kRmsShapes[rms_shape(d->C, d->dtype, 0)].G, rpb = (G > 256 ? G : 256) / G;
    // a row to a workgroup: fewer, whose records of C floats are much of the traffic
    const long long blocks = (d->rows + rpb - 1) / rpb, most = G > 64 ? kRmsMaxParts / 2 : kRmsMaxParts;
    return (int)(blocks < most ? blocks : most);
}

int launch_rms_forward(const wtc_rms_desc* d, const void* x, const void* r, const float* w, void* y, void* h,
                       float* rstd, float* scale, void* stream) {
    RmsArgs a = {};
    a.x = x; a.r = r; a.w = w; a.y = y; a.h = h; a.rstd = rstd; a.scale = scale;
    a.rows = d->rows; a.x_stride = d->x_stride; a.r_stride = d->r_stride;
    a.C = d->C; a.eps = d->eps; a.inv_C = 1.f / (float)d->C;
    const ForwardLaunch f = {a, reinterpret_cast<hipStream_t>(stream)};
    const int at = rms_shape(d->C, d->dtype, d->rows);
    if (d->dtype == WTC_BF16)
        rms_dispatch<uint16_t>(at, f);
    else
        rms_dispatch<float>(at, f);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_rms_backward(const wtc_rms_desc* d, const void* dy, const void* dh, const void* h, const float* w,
                        const float* rstd, void* dx, float* dw, float* parts, void* stream) {
    RmsArgs a = {};
    a.x = h; a.dy = dy; a.dh = dh; a.w = w; a.rstd_in = rstd; a.y = dx; a.parts = parts;
    a.rows = d->rows; a.x_stride = d->x_stride; a.g_stride = d->g_stride;
    a.C = d->C; a.inv_C = 1.f / (float)d->C;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const int n = rms_backward_parts(d);
    if (n > 0) {
        const BackwardLaunch f = {a, st, n};
        const int at = rms_shape(d->C, d->dtype, 0);
        if (d->dtype == WTC_BF16)
            rms_dispatch<uint16_t>(at, f);
        else
            rms_dispatch<float>(at, f);
    }
    hipLaunchKernelGGL(k_rms_join, dim3((unsigned)((d->C + 31) / 32)), dim3(1024), 0, st, parts, n, d->C, dw);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace wtc
