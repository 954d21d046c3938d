// Layer norm over rows, with the residual's addition:
//   h = round(x + r),  m = mean_c h,  s = 1 / sqrt(mean_c (h - m)^2 + eps),  y = (h - m) s w + b
// and its backward pass, with xh = (h - m) s and u = w dy,
//   dx = dh + s (u - mean_c u - xh mean_c(u xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// A row stays in the registers of a group of lanes, as in the root-mean-square
// norm beside it (wtc_tok_rows.h), so the variance is taken of differences from
// the mean and not as a difference of large sums.  The bound is device memory:
// 4 N e bytes forward with a residual, 4 N e backward.  Measured: 131072 x 384
// bf16 with a residual 74 us forward and 84 backward (403 MB each, 5.4 and 4.8
// TB/s), 5 for the join of dw and db; 50021 x 389 float32 without 27, 41.5 and
// 4.3 (156 and 234 MB: 5.8, some of it from the last-level cache, and 5.6 TB/s);
// 49 x 768 bf16 4.9, three dependent trips to memory.
#include <hip/hip_runtime.h>

#include "wtc_tok_rows.h"

namespace wtc {
namespace {

struct LayerArgs {
    const void *x, *r, *dy, *dh;   // x: h in the backward pass
    const float *w, *b;
    const float2* stats_in;        // a row's mean and s
    void *y, *h;                   // y: dx in the backward pass
    float2* stats;
    float* parts;
    long long rows, x_stride, r_stride, g_stride;
    int C, W;                      // W: floats of a record, C or 2 C
    float eps, inv_C;
};

template <typename T, int G, int NV>
__global__ void __launch_bounds__(G > 256 ? G : 256) k_layer_forward(LayerArgs a) {
    constexpr int V = kVec<T>, THREADS = G > 256 ? G : 256, RPB = THREADS / G;
    __shared__ float red[16];
    const int lane = threadIdx.x % G, sub = threadIdx.x / G;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<V>(a.w, a.C, (lane + i * G) * V, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) b[i][j] = 0.f;
        if (a.b) load_weight<V>(a.b, a.C, (lane + i * G) * V, b[i]);
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
        float h[NV][V], sum = 0.f, ss = 0.f;
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
            for (int j = 0; j < V; ++j) sum += h[i][j];
        const float m = group_reduce<G, false>(sum, red) * a.inv_C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = a.C - (lane + i * G) * V;   // places past the row's end are no channels
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[i][j] = j < n ? h[i][j] - m : 0.f;
                ss = fmaf(h[i][j], h[i][j], ss);
            }
        }
        ss = group_reduce<G, false>(ss, red);
        const float s = 1.f / sqrtf(fmaf(ss, a.inv_C, a.eps));
        if (a.stats && live && lane == 0) a.stats[row] = make_float2(m, s);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V, n = live ? a.C - c : 0;
#pragma unroll
            for (int j = 0; j < V; ++j) h[i][j] = fmaf(h[i][j] * s, w[i][j], b[i][j]);
            store_part(static_cast<T*>(a.y) + row * a.C + c, n, h[i]);
        }
    }
}

// Sums of a row's two terms at once.
template <int G>
__device__ __forceinline__ void group_sums(float& p, float& q, float2* red) {
#pragma unroll
    for (int o = 1; o < (G < 64 ? G : 64); o <<= 1) {
        p += __shfl_xor(p, o);
        q += __shfl_xor(q, o);
    }
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();   // the previous use of `red` is over
        if ((threadIdx.x & 63) == 0) red[wave] = make_float2(p, q);
        __syncthreads();
        p = q = 0.f;
#pragma unroll
        for (int i = 0; i < G / 64; ++i) {
            p += red[i].x;
            q += red[i].y;
        }
    }
}

template <typename T, int G, int NV>
__global__ void __launch_bounds__(G > 256 ? G : 256) k_layer_backward(LayerArgs a) {
    constexpr int V = kVec<T>, THREADS = G > 256 ? G : 256, RPB = THREADS / G;
    constexpr int WIDTH = G * NV * V;   // >= C
    constexpr bool AHEAD = NV <= 2 && G <= 256;
    __shared__ float2 red[16];
    __shared__ float join[G <= 64 ? 4 * WIDTH : 1];   // one parameter's sums of the four waves
    const int lane = threadIdx.x % G, sub = threadIdx.x / G;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight<V>(a.w, a.C, (lane + i * G) * V, w[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.f;
    }
    const long long step = (long long)gridDim.x * RPB;
    Raw<T> xn[NV], gn[NV], dn[NV];   // of the row that comes next
    float2 sn = make_float2(0.f, 0.f);
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V, n = row < a.rows ? a.C - c : 0;
            xn[i] = load_raw(static_cast<const T*>(a.x) + row * a.x_stride + c, n);
            gn[i] = load_raw(static_cast<const T*>(a.dy) + row * a.g_stride + c, n);
            dn[i] = a.dh ? load_raw(static_cast<const T*>(a.dh) + row * a.C + c, n) : Raw<T>{{0u, 0u, 0u, 0u}};
        }
        sn = row < a.rows ? a.stats_in[row] : make_float2(0.f, 0.f);
    };
    if (AHEAD) fetch((long long)blockIdx.x * RPB + sub);
    for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += step) {
        const long long row = first + sub;
        const bool live = row < a.rows;
        if (!AHEAD) fetch(row);
        float xh[NV][V], g[NV][V], along = 0.f, mean = 0.f;
        Raw<T> dr[NV];
        const float m = sn.x, s = sn.y;
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
            for (int j = 0; j < V; ++j) {   // past the row's end g is zero
                xh[i][j] = (xh[i][j] - m) * s;
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                db[i][j] += g[i][j];
                g[i][j] *= w[i][j];
                mean += g[i][j];
                along = fmaf(g[i][j], xh[i][j], along);
            }
        group_sums<G>(mean, along, red);
        mean *= a.inv_C;
        along *= a.inv_C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * G) * V, n = live ? a.C - c : 0;
            float d[V];
            unpack(dr[i], d);
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(s, fmaf(-xh[i][j], along, g[i][j] - mean), d[j]);
            store_part(static_cast<T*>(a.y) + row * a.C + c, n, d);
        }
    }
    // the workgroup's record: rows of a wave by shuffles, then its four waves
    float* rec = a.parts + (size_t)blockIdx.x * a.W;
    auto record = [&](float (&v)[NV][V], float* to) {
        if constexpr (G <= 64) {
            const int wave = threadIdx.x >> 6;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
#pragma unroll
                    for (int o = G; o < 64; o <<= 1) v[i][j] += __shfl_xor(v[i][j], o);
                    if ((threadIdx.x & 63) < G) join[wave * WIDTH + (lane + i * G) * V + j] = v[i][j];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < a.C; c += THREADS)
                to[c] = (join[c] + join[WIDTH + c]) + (join[2 * WIDTH + c] + join[3 * WIDTH + c]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + i * G) * V;
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    const float part[4] = {v[i][j], v[i][j + 1], v[i][j + 2], v[i][j + 3]};
                    store_part(to + c + j, a.C - c - j, part);
                }
            }
        }
    };
    record(dw, rec);
    if (a.W > a.C) record(db, rec + a.C);
}

struct ForwardLaunch {
    const LayerArgs& a;
    hipStream_t st;
    template <typename T, int G, int NV>
    void operator()() const {
        constexpr int threads = G > 256 ? G : 256, rpb = threads / G;
        // what fits at once: the next row is then read ahead
        const long long blocks = (a.rows + rpb - 1) / rpb, cap = threads > 256 ? 512 : NV > 1 ? 1024 : 2048;
        hipLaunchKernelGGL((k_layer_forward<T, G, NV>), dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(threads), 0,
                           st, a);
    }
};
struct BackwardLaunch {
    const LayerArgs& a;
    hipStream_t st;
    int parts;
    template <typename T, int G, int NV>
    void operator()() const {
        if constexpr (G >= 64 || NV == 1)   // the others are for the forward pass
            hipLaunchKernelGGL((k_layer_backward<T, G, NV>), dim3((unsigned)parts), dim3(G > 256 ? G : 256), 0, st, a);
    }
};

}  // namespace

// The records of rows that a workgroup of 1024 holds, 8 C bytes each, are much of the traffic: one workgroup a unit. Measured
// (us, bfloat16, of 512 and of 256, with their join): 1000 x 16384 66 and 51, 5000 x 16384 198 and 178, 300 x 12000 36 and 28.
// Workgroups of 256: 4096 x 4096 26 and 30, 20000 x 6000 163 and 227; 1000 x 8192 29 and 22.
int layer_backward_parts(const wtc_layer_desc* d) {
    const int n = row_parts(d->rows, d->C, d->dtype);
    return kRowShapes[row_shape(d->C, d->dtype, 0)].G > 256 && n > 256 ? 256 : n;
}

int launch_layer_forward(const wtc_layer_desc* d, const void* x, const void* r, const float* w, const float* b, void* y,
                         void* h, float* stats, void* stream) {
    LayerArgs a = {};
    a.x = x; a.r = r; a.w = w; a.b = b; a.y = y; a.h = h; a.stats = reinterpret_cast<float2*>(stats);
    a.rows = d->rows; a.x_stride = d->x_stride; a.r_stride = d->r_stride;
    a.C = d->C; a.eps = d->eps; a.inv_C = 1.f / (float)d->C;
    const ForwardLaunch f = {a, reinterpret_cast<hipStream_t>(stream)};
    const int at = row_shape(d->C, d->dtype, d->rows);
    if (d->dtype == WTC_BF16)
        row_dispatch<uint16_t>(at, f);
    else
        row_dispatch<float>(at, f);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_layer_backward(const wtc_layer_desc* d, const void* dy, const void* dh, const void* h, const float* w,
                          const float* stats, void* dx, float* dw, float* db, float* parts, void* stream) {
    LayerArgs a = {};
    a.x = h; a.dy = dy; a.dh = dh; a.w = w; a.stats_in = reinterpret_cast<const float2*>(stats); a.y = dx; a.parts = parts;
    a.rows = d->rows; a.x_stride = d->x_stride; a.g_stride = d->g_stride;
    a.C = d->C; a.W = db ? 2 * d->C : d->C; a.inv_C = 1.f / (float)d->C;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const int n = layer_backward_parts(d);
    if (n > 0) {
        const BackwardLaunch f = {a, st, n};
        const int at = row_shape(d->C, d->dtype, 0);
        if (d->dtype == WTC_BF16)
            row_dispatch<uint16_t>(at, f);
        else
            row_dispatch<float>(at, f);
    }
    hipLaunchKernelGGL(k_row_join, dim3((unsigned)((a.W + 31) / 32)), dim3(1024), 0, st, parts, n, a.W, dw, d->C, db);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace wtc
