// Rows sorted by expert and back.
//
// order:   pairs of a token and one of its k experts, p = t k + j, in the order
//          of the experts and of p among one expert's: a stable counting sort.
// gather:  rows[slot[t, j]] = x[t]
// sum:     y[t] = sum_j w[t, j] rows[slot[t, j]]   (gather's gradient with w = 1)
// and sum's gradient: drows[slot[t, j]] = w[t, j] dy[t], dw[t, j] = dy[t] . rows[slot[t, j]].
//
// The sort counts each run of pairs in shared memory (whole numbers, whose order
// does not show), sums the counts, and ranks 64 pairs at a time: the lanes with a
// lane's expert are found by one ballot a bit of the expert's number, and a wave
// walks a run of its own with its experts' next places in shared memory, so that
// it meets no other wave.  Up to kOneGroup pairs one workgroup does it all;
// beyond, a first kernel counts, a second sums the counts of each expert and a
// third places.  Bound by latency: 50176 pairs of 8 experts 2.9 + 2.4 + 3.9 us,
// 265638 of 118 3.9 + 3.5 + 6.2, one workgroup 3.7 (64 pairs) to 7.9 (6000).
//   The others are copies bound by device memory, by token: a token's row is
// read (or written) once for its k.  Rows of no pair, which follow those of the
// last expert, get zeros.  25088 x 384 bf16, two rows a token: gather 14.7 us
// (58 MB, 3.9 TB/s), sum 14.6, its gradient 18.6 (96 MB, 5.2 TB/s); 20011 x 771
// float32, three rows: 43, 62 and 98 us (247, 247 and 432 MB: 5.7, 4.0 and 4.4
// TB/s; rows of 3084 bytes begin inside a cache line, and sum's are anywhere).
#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace {

// ------------------------------------------------------------------ order
// One workgroup or three kernels (us, 8 / 64 / 512 experts): 4096 pairs 6.2 / 6.4 / 7.5 and 7.6 / 7.8 / 8.9, 6000 7.5 / 8.3 /
// 9.9 and 7.6 / 8.1 / 9.1, 8192 9.1 / 9.6 / 11.7 and 8.0 / 8.2 / 9.2, 32768 27.5 / 29 / 35 and 7.9 / 8.4 / 10.1.
constexpr int kOneGroup = 6144, kMostUnits = 1024;

struct OrderArgs {
    const int* experts;
    int *slot, *pair, *cu;
    int *counts, *totals;      // [E][units]: a unit's pairs of an expert, then where they begin; [E]
    int n, E, bits, units, run;   // run: pairs of a wave, a multiple of 64
};

// Lanes with this lane's expert, of those that have one.
__device__ __forceinline__ uint64_t same_expert(int e, bool there, int bits) {
    uint64_t m = __builtin_amdgcn_ballot_w64(there);
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __builtin_amdgcn_ballot_w64((e >> b) & 1);
        m &= (e >> b) & 1 ? one : ~one;
    }
    return m;
}
__device__ __forceinline__ int lanes_below(uint64_t m) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}
// f(p, expert, there, same, rank) for the pairs of a run, 64 at a time.
template <typename F>
__device__ __forceinline__ void walk(const OrderArgs& a, int first, int last, int lane, const F& f) {
    int next = first + lane < last ? a.experts[first + lane] : -1;
    for (int p0 = first; p0 < last; p0 += 64) {
        const int e = next, p = p0 + lane;
        next = p + 64 < last ? a.experts[p + 64] : -1;
        const bool there = p < last && e >= 0 && e < a.E;
        const uint64_t same = same_expert(e, there, a.bits);
        f(p, e, there, same, lanes_below(same));
    }
}
// Pairs of each expert in a run, added to counts in shared memory: whole numbers, in any order.
__device__ __forceinline__ void count_run(const OrderArgs& a, int first, int last, int lane, int* mine) {
#pragma unroll 4
    for (int p = first + lane; p < last; p += 64) {
        const int e = a.experts[p];
        if (e >= 0 && e < a.E) atomicAdd(mine + e, 1);
    }
}
__device__ __forceinline__ void place_run(const OrderArgs& a, int first, int last, int lane, int* mine) {
    walk(a, first, last, lane, [&](int p, int e, bool there, uint64_t same, int rank) {
        int at = -1;
        if (there) at = mine[e] + rank;
        __builtin_amdgcn_wave_barrier();   // all lanes have read before the first of each expert goes on
        if (there && rank == 0) mine[e] += __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
        if (p < last) a.slot[p] = at;
        if (there) a.pair[at] = p;
    });
}
// Exclusive sums over the threads of a workgroup of WAVES waves; all get the sum of all.
template <int WAVES>
__device__ __forceinline__ int expert_starts(int total, int* sums, int& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int v = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    if (lane == 63) sums[wave] = v;
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < WAVES; ++w) {
        if (w < wave) before += sums[w];
        all += sums[w];
    }
    return before + v - total;
}

__global__ void __launch_bounds__(1024) k_order_one(OrderArgs a) {
    extern __shared__ int count[];   // [16][E]
    __shared__ int sums[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int* mine = count + wave * a.E;
    for (int e = lane; e < a.E; e += 64) mine[e] = 0;
    const int first = min(wave * a.run, a.n), last = min(first + a.run, a.n);
    __syncthreads();
    count_run(a, first, last, lane, mine);
    __syncthreads();
    const int e = threadIdx.x;
    int total = 0, all;
    if (e < a.E)
        for (int w = 0; w < 16; ++w) {
            const int v = count[w * a.E + e];
            count[w * a.E + e] = total;
            total += v;
        }
    const int start = expert_starts<16>(total, sums, all);
    if (e < a.E) {
        a.cu[e] = start;
        for (int w = 0; w < 16; ++w) count[w * a.E + e] += start;
    }
    if (e == 0) a.cu[a.E] = all;
    __syncthreads();
    place_run(a, first, last, lane, mine);
    for (int r = all + threadIdx.x; r < a.n; r += 1024) a.pair[r] = -1;
}

// The run of one of a unit's four waves.
struct Run {
    int first, last;
};
__device__ __forceinline__ Run run_of(const OrderArgs& a, int wave) {
    const long long first = min(((long long)blockIdx.x * 4 + wave) * a.run, (long long)a.n);
    return {(int)first, (int)min(first + a.run, (long long)a.n)};
}
__global__ void __launch_bounds__(256) k_order_count(OrderArgs a) {
    extern __shared__ int count[];   // [E]
    const int lane = threadIdx.x & 63;
    for (int e = threadIdx.x; e < a.E; e += 256) count[e] = 0;
    __syncthreads();
    const Run r = run_of(a, threadIdx.x >> 6);
    count_run(a, r.first, r.last, lane, count);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) a.counts[(size_t)e * a.units + blockIdx.x] = count[e];
}
// Counts of an expert to the places, among the expert's own, where each unit's pairs of it begin; its total.
__global__ void __launch_bounds__(64) k_order_sum(OrderArgs a) {
    const int lane = threadIdx.x, e = blockIdx.x;
    int* row = a.counts + (size_t)e * a.units;
    int4 v[kMostUnits / 256];   // of four units a lane, all on their way at once
#pragma unroll
    for (int i = 0; i < kMostUnits / 256; ++i) {
        const int u = 256 * i + 4 * lane;
        v[i] = u < a.units ? *reinterpret_cast<const int4*>(row + u) : make_int4(0, 0, 0, 0);
    }
    int before = 0;
#pragma unroll
    for (int i = 0; i < kMostUnits / 256; ++i) {
        const int u = 256 * i + 4 * lane, s = v[i].x + v[i].y + v[i].z + v[i].w;
        if (256 * i >= a.units) break;
        int up = s;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int t = __shfl_up(up, o);
            if (lane >= o) up += t;
        }
        const int at = before + up - s;
        if (u < a.units)
            *reinterpret_cast<int4*>(row + u) = make_int4(at, at + v[i].x, at + v[i].x + v[i].y, at + v[i].x + v[i].y + v[i].z);
        before += __shfl(up, 63);
    }
    if (lane == 0) a.totals[e] = before;
}
__global__ void __launch_bounds__(256) k_order_place(OrderArgs a) {
    extern __shared__ int next[];   // [4][E]
    __shared__ int sums[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < 4 * a.E; e += 256) next[e] = 0;
    const Run r = run_of(a, wave);
    __syncthreads();
    count_run(a, r.first, r.last, lane, next + wave * a.E);
    // every unit finds the experts' first places for itself, two experts a thread
    int total[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) total[i] = 2 * (int)threadIdx.x + i < a.E ? a.totals[2 * threadIdx.x + i] : 0;
    int all, start = expert_starts<4>(total[0] + total[1], sums, all);   // the counts are whole behind its barrier
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * (int)threadIdx.x + i;
        if (e < a.E) {
            if (blockIdx.x == 0) a.cu[e] = start;
            int at = start + a.counts[(size_t)e * a.units + blockIdx.x];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int v = next[w * a.E + e];
                next[w * a.E + e] = at;
                at += v;
            }
        }
        start += total[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.cu[a.E] = all;
    __syncthreads();
    place_run(a, r.first, r.last, lane, next + wave * a.E);
    for (long long p = (long long)all + blockIdx.x * 256 + threadIdx.x; p < a.n; p += (long long)a.units * 256) a.pair[p] = -1;
}
static_assert(WTC_EXPERTS_MAX <= 512, "two experts a thread");

// ------------------------------------------------------------------ rows
struct RowsArgs {
    const void *x, *rows, *dy;
    const float* w;
    const int *slot, *cu;
    void *y;          // what is written by token
    void *out;        // what is written by row
    float* dw;
    long long T, n, x_stride, r_stride;   // n = T k
    int k, C, chunks, E;
    FastDiv div;      // by chunks
};

// f(token, channel) for 16-byte chunks in the order of memory: one a thread, so that as many as possible are on their way
// (four one after another: 25088 x 384 bf16 gather 16.5 us and 14.5 so, 2213 x 2005 sum 18.8 and 10.3).
template <typename T, typename F>
__device__ __forceinline__ void each_chunk(const RowsArgs& a, const F& f) {
    for (long long u0 = (long long)blockIdx.x * 256; u0 < a.T * a.chunks; u0 += (long long)gridDim.x * 256) {
        const long long t0 = u0 / a.chunks;
        const int v = (int)(u0 - t0 * a.chunks) + (int)threadIdx.x, q = fdiv(v, a.div);
        if (t0 + q < a.T) f(t0 + q, (v - q * a.chunks) * kVec<T>);
    }
}
__device__ __forceinline__ bool is_row(const RowsArgs& a, int r) { return r >= 0 && r < a.n; }

// Zeros to the rows of no pair, by all workgroups of the grid.
template <typename T>
__device__ __forceinline__ void clear_rest(const RowsArgs& a) {
    const long long first = min(max((long long)a.cu[a.E], 0ll), a.n);
    const float zero[kVec<T>] = {};
    const long long all = (a.n - first) * a.chunks;
    for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < all; u += (long long)gridDim.x * 256) {
        const long long r = u / a.chunks;
        const int c = (int)(u - r * a.chunks) * kVec<T>;
        store_part(static_cast<T*>(a.out) + (first + r) * a.C + c, a.C - c, zero);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_rows_gather(RowsArgs a) {
    each_chunk<T>(a, [&](long long t, int c) {
        const int n = a.C - c;
        float v[kVec<T>];
        unpack(load_raw(static_cast<const T*>(a.x) + t * a.x_stride + c, n), v);
        for (int j = 0; j < a.k; ++j) {
            const int r = a.slot[t * a.k + j];
            if (is_row(a, r)) store_part(static_cast<T*>(a.out) + (long long)r * a.C + c, n, v);
        }
    });
    clear_rest<T>(a);
}

template <typename T>
__global__ void __launch_bounds__(256) k_rows_sum(RowsArgs a) {
    constexpr int V = kVec<T>;
    each_chunk<T>(a, [&](long long t, int c) {
        const int n = a.C - c;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            Raw<T> r[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool there = j0 + j < a.k;
                const int at = there ? a.slot[t * a.k + j0 + j] : -1;
                const bool row = is_row(a, at);
                w[j] = row && a.w ? a.w[t * a.k + j0 + j] : 1.f;
                r[j] = load_raw(static_cast<const T*>(a.rows) + (row ? at : 0) * a.r_stride + c, row ? n : 0);
                if (!row) w[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[V];
                unpack(r[j], x);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = fmaf(w[j], x[i], v[i]);
            }
        }
        store_part(static_cast<T*>(a.y) + t * a.C + c, n, v);
    });
}

// G lanes a token: the products' sums of its weights' gradients are theirs.
template <typename T, int G>
__global__ void __launch_bounds__(256) k_rows_sum_back(RowsArgs a) {
    constexpr int V = kVec<T>;
    const int lane = threadIdx.x % G;
    for (long long t = (long long)blockIdx.x * (256 / G) + threadIdx.x / G; t < a.T; t += (long long)gridDim.x * (256 / G)) {
        for (int j0 = 0; j0 < a.k; j0 += 2) {
            int at[2];
            float w[2], dot[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                at[j] = j0 + j < a.k ? a.slot[t * a.k + j0 + j] : -1;
                if (!is_row(a, at[j])) at[j] = -1;
                w[j] = at[j] >= 0 ? a.w[t * a.k + j0 + j] : 0.f;
            }
            for (int c = lane * V; c < a.C; c += G * V) {
                const int n = a.C - c;
                float g[V], x[2][V];
                unpack(load_raw(static_cast<const T*>(a.dy) + t * a.x_stride + c, n), g);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    unpack(load_raw(static_cast<const T*>(a.rows) + (at[j] >= 0 ? at[j] : 0) * a.r_stride + c, at[j] >= 0 ? n : 0),
                           x[j]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (at[j] < 0) continue;
                    float d[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dot[j] = fmaf(g[i], x[j][i], dot[j]);
                        d[i] = w[j] * g[i];
                    }
                    store_part(static_cast<T*>(a.out) + (long long)at[j] * a.C + c, n, d);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int o = 1; o < G; o <<= 1) dot[j] += __shfl_xor(dot[j], o);
                if (lane == 0 && j0 + j < a.k) a.dw[t * a.k + j0 + j] = dot[j];
            }
        }
    }
    clear_rest<T>(a);
}

RowsArgs rows_args(const wtc_rows_desc* d, const int* slot, const int* cu) {
    RowsArgs a = {};
    const int V = d->dtype == WTC_BF16 ? kVec<uint16_t> : kVec<float>;
    a.slot = slot; a.cu = cu;
    a.T = d->T; a.k = d->k; a.n = d->T * d->k; a.C = d->C; a.E = d->E;
    a.x_stride = d->x_stride; a.r_stride = d->r_stride;
    a.chunks = (d->C + V - 1) / V;
    a.div = make_div(a.chunks);
    return a;
}
dim3 chunk_grid(const RowsArgs& a) {
    const long long blocks = (a.T * a.chunks + 255) / 256;
    return dim3((unsigned)(blocks < (1 << 23) ? blocks : 1 << 23));
}

struct OrderPlan {
    int units, run;
};
OrderPlan order_plan(long long n, int E) {
    OrderPlan p;
    if (n <= kOneGroup) {
        p.units = 16;   // waves of the one workgroup
        p.run = (int)(((n + 15) / 16 + 63) / 64 * 64);
    } else {   // a unit has four waves; counts are summed four at a time
        const long long most = (n + 255) / 256;
        p.units = (int)(((most < kMostUnits ? most : kMostUnits) + 3) / 4 * 4);
        const long long waves = 4LL * p.units;
        p.run = (int)(((n + waves - 1) / waves + 63) / 64 * 64);
    }
    return p;
}

}  // namespace

size_t order_workspace(long long n, int E) {
    return n <= kOneGroup ? 0 : (size_t)E * (order_plan(n, E).units + 1) * sizeof(int);
}

int launch_expert_order(long long n, int E, const int* experts, int* slot, int* pair, int* cu, void* workspace, void* stream) {
    OrderArgs a = {};
    const OrderPlan p = order_plan(n, E);
    a.experts = experts; a.slot = slot; a.pair = pair; a.cu = cu; a.counts = static_cast<int*>(workspace);
    a.n = (int)n; a.E = E; a.units = p.units; a.run = p.run;
    while ((1 << a.bits) < E) ++a.bits;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (n <= kOneGroup) {
        hipLaunchKernelGGL(k_order_one, dim3(1), dim3(1024), 16 * E * sizeof(int), st, a);
    } else {
        a.totals = a.counts + (size_t)E * a.units;
        hipLaunchKernelGGL(k_order_count, dim3((unsigned)p.units), dim3(256), E * sizeof(int), st, a);
        hipLaunchKernelGGL(k_order_sum, dim3((unsigned)E), dim3(64), 0, st, a);
        hipLaunchKernelGGL(k_order_place, dim3((unsigned)p.units), dim3(256), 4 * E * sizeof(int), st, a);
    }
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_rows_gather(const wtc_rows_desc* d, const void* x, const int* slot, const int* cu, void* rows, void* stream) {
    RowsArgs a = rows_args(d, slot, cu);
    a.x = x; a.out = rows;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16)
        hipLaunchKernelGGL(k_rows_gather<uint16_t>, chunk_grid(a), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(k_rows_gather<float>, chunk_grid(a), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_rows_sum(const wtc_rows_desc* d, const void* rows, const float* weights, const int* slot, void* y, void* stream) {
    RowsArgs a = rows_args(d, slot, nullptr);
    a.rows = rows; a.w = weights; a.y = y;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16)
        hipLaunchKernelGGL(k_rows_sum<uint16_t>, chunk_grid(a), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(k_rows_sum<float>, chunk_grid(a), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

namespace {
template <typename T>
void run_sum_back(const RowsArgs& a, hipStream_t st) {
    // Lanes of a token: 4 up to 4 chunks, 16 up to 64, and a wave beyond, which has four steps in rows of 256 chunks and more in
    // longer ones.  Measured (us): 48 chunks (25088 x 384 bf16) by 16 lanes 18.6, by 64 22.2; 9 chunks (44273 x 35 float32, six
    // rows a token) by 4 30.9, by 16 27.9
    const int G = a.chunks <= 4 ? 4 : a.chunks <= 64 ? 16 : 64;
    const long long blocks = (a.T * G + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
    if (G == 4)
        hipLaunchKernelGGL((k_rows_sum_back<T, 4>), grid, dim3(256), 0, st, a);
    else if (G == 16)
        hipLaunchKernelGGL((k_rows_sum_back<T, 16>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_rows_sum_back<T, 64>), grid, dim3(256), 0, st, a);
}
}  // namespace

int launch_rows_sum_backward(const wtc_rows_desc* d, const void* dy, const void* rows, const float* weights, const int* slot,
                             const int* cu, void* drows, float* dweights, void* stream) {
    RowsArgs a = rows_args(d, slot, cu);
    a.dy = dy; a.rows = rows; a.w = weights; a.out = drows; a.dw = dweights;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16)
        run_sum_back<uint16_t>(a, st);
    else
        run_sum_back<float>(a, st);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace wtc
