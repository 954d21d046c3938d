// Gated linear recurrence inside each sequence of a pack:
//   a = sigmoid(f),  h_t = a_t h_(t-1) + (1 - a_t) x_t,  y = h
// from the sequence's first token to its last, or the other way, and its
// backward pass: with G_t = a_(t+1) dh_(t+1) (the last state's gradient at the end),
//   dh_t = dy_t + G_t,  dx = (1 - a) dh,  df = dh (h_(t-1) - x) a (1 - a).
//
// Both are compositions of maps h -> A h + B, which are associative: a token's
// map, a thread's four tokens, a wave's eight such groups (by shuffles), the
// four waves of a workgroup (through shared memory).  A workgroup walks one
// part of the pack, 128 tokens by 128 bytes of channels at a time, with the
// state in registers.  With several parts a first kernel composes each part's
// map, so that a part can begin with the state that those before it leave: it
// reads only the tokens behind the part's last sequence start, and none of the
// part is read twice where sequences are short.  A token that starts a sequence
// has A = 0, and a composition with A = 0 takes nothing from what came before
// it, not even a NaN.
//
// Bound by device memory: 3 T C e bytes forward (x, f in, y out), 5 T C e
// backward (x, f, dy in, dx, df out), which takes the state at each tile's start
// from the forward pass (4 bytes for 128 tokens and channel) and computes the others
// again.  All of it is float32.
#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace {

constexpr int kLanes = 8;                       // lanes along the channels, 16 bytes each
constexpr int kGroups = 256 / kLanes;           // groups along the tokens
constexpr int kEach = kScanTile / kGroups;      // tokens of a thread, consecutive
static_assert(kEach * kGroups == kScanTile, "whole groups");
template <typename T>
constexpr int kWidth = kLanes * kVec<T>;        // channels of a workgroup

struct ScanArgs {
    const void *x, *f, *dy;
    const int* cu;
    const float *state, *dlast, *kept_in;
    void *y, *df;                // y: dx in the backward pass
    float *last, *kept;          // last: the gradient of state in the backward pass
    float2* maps;                // [parts][C], of each part
    long long x_stride, f_stride, g_stride;
    int T, n_seq, C, reverse, parts, part_tiles;
};

// h -> A h + B; A = 0 exactly where a sequence starts in it (or a gate is that small).
struct Map {
    float A, B;
};
__device__ __forceinline__ float apply(const Map& m, float h) { return m.A == 0.f ? m.B : fmaf(m.A, h, m.B); }
// first one, then the other
__device__ __forceinline__ Map after(const Map& one, const Map& other) {
    return {other.A == 0.f ? 0.f : other.A * one.A, apply(other, one.B)};
}

// sigmoid(f) and 1 - sigmoid(f).  float32: the exponent's product is rounded at
// its own size, so exp is of float32's accuracy only with its lower part; what
// bfloat16 holds of f is coarser than that.
template <typename T>
__device__ __forceinline__ void gate(float f, float& a, float& take) {
    float e;
    if constexpr (sizeof(T) == 2) {
        const float t = f * -1.4426950408889634f;
        e = __builtin_amdgcn_exp2f(t > 126.f ? 126.f : t);
    } else {
        const float v = f < -87.f ? 87.f : f > 104.f ? -104.f : -f, t = v * 1.4426950408889634f;   // a NaN stays one
        const float low = fmaf(v, 1.4426950408889634f, -t) + v * 1.9259629911266175e-8f;
        e = __builtin_amdgcn_exp2f(t);
        e = fmaf(e, low * 0.6931471805599453f, e);
    }
    a = __builtin_amdgcn_rcpf(1.f + e);
    take = e * a;
}

// Places of a pack in the order they are walked: place p is token p, or with
// `reverse` token T - 1 - p.  Sequence s = 0 .. n_seq - 1 in that order is
// places begin(s) .. begin(s + 1) - 1; number(s) is its row of the states.
__device__ __forceinline__ int begin_of(const ScanArgs& a, int s) {
    const int v = min(max(a.cu[a.reverse ? a.n_seq - s : s], 0), a.T);
    return a.reverse ? a.T - v : v;
}
__device__ __forceinline__ int number_of(const ScanArgs& a, int s) { return a.reverse ? a.n_seq - 1 - s : s; }
__device__ __forceinline__ long long row_of(const ScanArgs& a, int p) { return a.reverse ? a.T - 1 - p : p; }

// The last sequence that begins at place p or before, by all lanes of a wave;
// -1 if none does.
__device__ __forceinline__ int find_sequence(const ScanArgs& a, int p, int lane) {
    int lo = -1, hi = a.n_seq;   // it is in lo .. hi - 1; begin(lo) <= p < begin(hi), as far as those are sequences
    while (hi - lo > 1) {
        const int step = (hi - lo - 1 + 63) / 64, s = lo + 1 + lane * step;
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(s < hi && begin_of(a, min(s, hi - 1)) <= p));
        const int found = n > 0 ? lo + 1 + (n - 1) * step : lo;
        hi = min(hi, lo + 1 + n * step);
        lo = found;
    }
    return lo;
}

// Which sequence starts, and which ends, at each place of a tile (-1: none).
struct Marks {
    int start[kScanTile], end[kScanTile];
};

// The places of sequences, and the one that a workgroup is in.
struct Where {
    int lo, hi;           // places outside of these belong to no sequence
    int from, to;         // places strictly between them have no start and no end
};
__device__ __forceinline__ Where where_begin(const ScanArgs& a) {
    Where w;
    w.lo = a.n_seq > 0 ? begin_of(a, 0) : 0;
    w.hi = a.n_seq > 0 ? begin_of(a, a.n_seq) : 0;
    w.from = 0;
    w.to = -1;
    return w;
}
// Whether the tile at p0 has marks, which are then in `m` (for all threads).
__device__ __forceinline__ bool mark(const ScanArgs& a, int p0, Where& w, Marks& m, int lane) {
    const int end = min(p0 + kScanTile, a.T);
    if (p0 > w.from && end < w.to) return false;
    const int s0 = find_sequence(a, p0, lane);
    if (s0 >= 0 && s0 < a.n_seq) {
        w.from = begin_of(a, s0);
        w.to = begin_of(a, s0 + 1);
        if (p0 > w.from && end < w.to) return false;
    }
    __syncthreads();   // the marks' last use is over
    if (threadIdx.x < kScanTile) m.start[threadIdx.x] = m.end[threadIdx.x] = -1;
    __syncthreads();
    for (int s = max(s0, 0) + (int)threadIdx.x; s < a.n_seq; s += 256) {
        const int b = begin_of(a, s), e = begin_of(a, s + 1);
        if (b >= end) break;
        if (e <= b) continue;
        if (b >= p0) m.start[b - p0] = s;
        if (e > p0 && e <= end) m.end[e - 1 - p0] = s;
    }
    __syncthreads();
    return true;
}

// One float per channel of a row of the states.
template <int V>
__device__ __forceinline__ void load_state(const float* row, int n, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        float part[4];
        load_part(row + i, n - i, part);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = part[j];
    }
}
template <int V>
__device__ __forceinline__ void store_state(float* row, int n, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float part[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
        store_part(row + i, n - i, part);
    }
}

// The maps of the groups of tokens composed over the workgroup, in their order
// or (BACK) the other way.  `m` becomes the composition of all before this
// thread's group in its wave; waves: that of each whole wave, in `sums`.
template <int V>
struct Sums {
    float2 m[2][4][kLanes][V];   // two, in turn: one barrier a scan
};
template <bool BACK, int V>
__device__ __forceinline__ void scan_wave(Map (&m)[V], float2 (&sums)[4][kLanes][V], int lane, int wave) {
#pragma unroll
    for (int o = kLanes; o < 64; o <<= 1) {
        const bool there = BACK ? lane + o < 64 : lane >= o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Map p;
            p.A = BACK ? __shfl_down(m[i].A, o) : __shfl_up(m[i].A, o);
            p.B = BACK ? __shfl_down(m[i].B, o) : __shfl_up(m[i].B, o);
            if (there) m[i] = after(p, m[i]);
        }
    }
    if (BACK ? lane < kLanes : lane >= 64 - kLanes) {
#pragma unroll
        for (int i = 0; i < V; ++i) sums[wave][lane % kLanes][i] = make_float2(m[i].A, m[i].B);
    }
    const bool first = BACK ? lane >= 64 - kLanes : lane < kLanes;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        Map p;
        p.A = BACK ? __shfl_down(m[i].A, kLanes) : __shfl_up(m[i].A, kLanes);
        p.B = BACK ? __shfl_down(m[i].B, kLanes) : __shfl_up(m[i].B, kLanes);
        m[i] = first ? Map{1.f, 0.f} : p;
    }
}
// After a barrier: `at` is the state before this thread's group, `carry` that
// after the whole workgroup's.
template <bool BACK, int V>
__device__ __forceinline__ void scan_apply(const Map (&m)[V], const float2 (&sums)[4][kLanes][V], int lane, int wave,
                                           float (&carry)[V], float (&at)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float c = carry[i], mine = c;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int w = BACK ? 3 - k : k;
            if (w == wave) mine = c;
            const float2 s = sums[w][lane % kLanes][i];
            c = apply(Map{s.x, s.y}, c);
        }
        carry[i] = c;
        at[i] = apply(m[i], mine);
    }
}

// The state that the parts before (BACK: after) this one leave: their maps
// composed, a run of them by each group.
template <bool BACK, int V>
__device__ __forceinline__ void carry_in(const ScanArgs& a, int part, int c, int n, float2 (&sums)[4][kLanes][V], int lane,
                                         int wave, float (&carry)[V]) {
    const int group = threadIdx.x / kLanes, many = BACK ? a.parts - 1 - part : part, run = (many + kGroups - 1) / kGroups;
    Map m[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        m[i] = {1.f, 0.f};
        carry[i] = 0.f;
    }
    if (many == 0) return;
    const int turn = BACK ? kGroups - 1 - group : group;   // scan_wave's order of the groups
    for (int k = turn * run; k < min((turn + 1) * run, many); ++k) {
        const float2* p = a.maps + (size_t)(BACK ? a.parts - 1 - k : k) * a.C + c;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) {
                const float2 v = p[i];
                m[i] = after(m[i], Map{v.x, v.y});
            }
    }
    float at[V];
    scan_wave<BACK>(m, sums, lane, wave);
    __syncthreads();
    scan_apply<BACK>(m, sums, lane, wave, carry, at);
    __syncthreads();
}

// A thread's four tokens of a tile, as they lie in memory.
template <typename T>
struct Rows {
    Raw<T> v[kEach];
    __device__ __forceinline__ void fetch(const void* base, long long stride, const ScanArgs& a, int p, int c, int n) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const bool there = p + j < a.T;
            v[j] = load_raw(static_cast<const T*>(base) + row_of(a, there ? p + j : 0) * stride + c, there ? n : 0);
        }
    }
};

// The maps of a thread's tokens (a: A, b: B) and their composition.
template <typename T>
struct Tokens {
    static constexpr int V = kVec<T>;
    float a[kEach][V], b[kEach][V];
    int start[kEach];   // the sequence that starts there, or -1

    __device__ __forceinline__ void make(const ScanArgs& s, const Rows<T>& x, const Rows<T>& f, bool marks, const Marks& m,
                                         const Where& w, int p, int at, int c, int n) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            float xv[V], fv[V];
            unpack(x.v[j], xv);
            unpack(f.v[j], fv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float take;
                gate<T>(fv[i], a[j][i], take);
                b[j][i] = take * xv[i];
            }
            start[j] = -1;
            if (marks) {
                start[j] = m.start[at + j];
                const bool none = p + j < w.lo || p + j >= w.hi;
                if (none || start[j] >= 0) {
                    float h[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) h[i] = 0.f;
                    if (!none && s.state) load_state(s.state + (size_t)number_of(s, start[j]) * s.C + c, n, h);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        b[j][i] = none ? 0.f : s.state ? fmaf(a[j][i], h[i], b[j][i]) : b[j][i];
                        a[j][i] = 0.f;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void compose(Map (&m)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m[i] = {a[0][i], b[0][i]};
#pragma unroll
            for (int j = 1; j < kEach; ++j) m[i] = after(m[i], Map{a[j][i], b[j][i]});
        }
    }
};

// The map of a part: of its tokens from the last sequence start on.
template <typename T>
__global__ void __launch_bounds__(256) k_scan_parts(ScanArgs a) {
    constexpr int V = kVec<T>;
    __shared__ Sums<V> sums;
    __shared__ Marks marks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = (int)(threadIdx.x / kLanes) * kEach;
    const int part = blockIdx.y, c = blockIdx.x * kWidth<T> + (lane % kLanes) * V, n = a.C - c;
    const int first = part * a.part_tiles, end = first + a.part_tiles;   // the last part has none
    Where w = where_begin(a);
    const int s = find_sequence(a, end * kScanTile - 1, lane);
    int tile = s < 0 ? end - 1 : max(first, min(begin_of(a, s) / kScanTile, end - 1));
    float A[V], B[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        A[i] = 1.f;
        B[i] = 0.f;
    }
    Rows<T> x, f;
    x.fetch(a.x, a.x_stride, a, tile * kScanTile + at, c, n);
    f.fetch(a.f, a.f_stride, a, tile * kScanTile + at, c, n);
    for (; tile < end; ++tile) {
        const int p0 = tile * kScanTile;
        const bool marked = mark(a, p0, w, marks, lane);
        Tokens<T> t;
        t.make(a, x, f, marked, marks, w, p0 + at, at, c, n);
        if (tile + 1 < end) {
            x.fetch(a.x, a.x_stride, a, p0 + kScanTile + at, c, n);
            f.fetch(a.f, a.f_stride, a, p0 + kScanTile + at, c, n);
        }
        Map m[V];
        t.compose(m);
        scan_wave<false>(m, sums.m[tile & 1], lane, wave);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 v = sums.m[tile & 1][k][lane % kLanes][i];
                const Map r = after(Map{A[i], B[i]}, Map{v.x, v.y});
                A[i] = r.A;
                B[i] = r.B;
            }
    }
    if (threadIdx.x < kLanes) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) a.maps[(size_t)part * a.C + c + i] = make_float2(A[i], B[i]);
    }
}

// What sequences with no token leave behind.
template <int V>
__device__ __forceinline__ void pass_on(const ScanArgs& a, const float* from, float* to, int part, int c, int n) {
    for (int s = part * kGroups + (int)(threadIdx.x / kLanes); s < a.n_seq; s += a.parts * kGroups) {
        if (begin_of(a, s + 1) > begin_of(a, s)) continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        const size_t row = (size_t)number_of(a, s) * a.C + c;
        if (from) load_state(from + row, n, v);
        store_state(to + row, n, v);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_scan_forward(ScanArgs a) {
    constexpr int V = kVec<T>;
    __shared__ Sums<V> sums;
    __shared__ Marks marks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = (int)(threadIdx.x / kLanes) * kEach;
    const int part = blockIdx.y, c = blockIdx.x * kWidth<T> + (lane % kLanes) * V, n = a.C - c;
    const int first = part * a.part_tiles, end = min(first + a.part_tiles, (a.T + kScanTile - 1) / kScanTile);
    if (a.last) pass_on<V>(a, a.state, a.last, part, c, n);
    if (first >= end) return;
    Rows<T> x, f;
    x.fetch(a.x, a.x_stride, a, first * kScanTile + at, c, n);
    f.fetch(a.f, a.f_stride, a, first * kScanTile + at, c, n);
    Where w = where_begin(a);
    float carry[V];
    carry_in<false>(a, part, c, n, sums.m[0], lane, wave, carry);
    for (int tile = first; tile < end; ++tile) {
        const int p0 = tile * kScanTile;
        const bool marked = mark(a, p0, w, marks, lane);
        Tokens<T> t;
        t.make(a, x, f, marked, marks, w, p0 + at, at, c, n);
        if (tile + 1 < end) {
            x.fetch(a.x, a.x_stride, a, p0 + kScanTile + at, c, n);
            f.fetch(a.f, a.f_stride, a, p0 + kScanTile + at, c, n);
        }
        Map m[V];
        t.compose(m);
        scan_wave<false>(m, sums.m[tile & 1], lane, wave);
        if (a.kept && threadIdx.x < kLanes) store_state(a.kept + (size_t)tile * a.C + c, n, carry);
        __syncthreads();
        float h[V];
        scan_apply<false>(m, sums.m[tile & 1], lane, wave, carry, h);
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = apply(Map{t.a[j][i], t.b[j][i]}, h[i]);
            const int p = p0 + at + j;
            if (p < a.T) store_part(static_cast<T*>(a.y) + row_of(a, p) * a.C + c, n, h);
            if (marked && a.last) {
                const int s = marks.end[at + j];
                if (s >= 0) store_state(a.last + (size_t)number_of(a, s) * a.C + c, n, h);
            }
        }
    }
}

// Backward.  What a token hands to the one before it is G = a (dy + G'), with
// the last state's gradient added to dy at a sequence's end; a token that
// starts a sequence hands on nothing (a = 0, as in the forward pass).
template <typename T>
struct Grads {
    static constexpr int V = kVec<T>;
    float g[kEach][V];   // dy, and the last state's gradient

    __device__ __forceinline__ void make(const ScanArgs& s, const Rows<T>& dy, bool marks, const Marks& m, const Where& w,
                                         int p, int at, int c, int n) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            unpack(dy.v[j], g[j]);
            if (marks) {
                const int e = m.end[at + j];
                if (e >= 0 && s.dlast) {
                    float d[V];
                    load_state(s.dlast + (size_t)number_of(s, e) * s.C + c, n, d);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[j][i] += d[i];
                }
                if (p + j < w.lo || p + j >= w.hi) {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[j][i] = 0.f;
                }
            }
        }
    }
    __device__ __forceinline__ void compose(const float (&a)[kEach][V], Map (&m)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m[i] = {1.f, 0.f};
#pragma unroll
            for (int j = kEach - 1; j >= 0; --j) {
                m[i].B = a[j][i] == 0.f ? 0.f : a[j][i] * (g[j][i] + m[i].B);
                m[i].A = a[j][i] == 0.f ? 0.f : a[j][i] * m[i].A;
            }
        }
    }
};

// The map of a part for the backward pass: of its tokens up to the first sequence start.
template <typename T>
__global__ void __launch_bounds__(256) k_scan_parts_back(ScanArgs a) {
    constexpr int V = kVec<T>;
    __shared__ Sums<V> sums;
    __shared__ Marks marks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = (int)(threadIdx.x / kLanes) * kEach;
    const int part = blockIdx.y + 1, c = blockIdx.x * kWidth<T> + (lane % kLanes) * V, n = a.C - c;   // the first has none
    const int tiles = (a.T + kScanTile - 1) / kScanTile;
    const int first = part * a.part_tiles, end = min(first + a.part_tiles, tiles);
    Where w = where_begin(a);
    const int s = find_sequence(a, first * kScanTile - 1, lane) + 1;   // the next to begin
    int tile = s >= a.n_seq ? end - 1 : min(max(begin_of(a, s) / kScanTile, first), end - 1);
    float A[V], B[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        A[i] = 1.f;
        B[i] = 0.f;
    }
    Rows<T> dy, f;
    dy.fetch(a.dy, a.g_stride, a, tile * kScanTile + at, c, n);
    f.fetch(a.f, a.f_stride, a, tile * kScanTile + at, c, n);
    for (; tile >= first; --tile) {
        const int p0 = tile * kScanTile;
        const bool marked = mark(a, p0, w, marks, lane);
        Tokens<T> t;
        Grads<T> g;
        t.make(a, f, f, marked, marks, w, p0 + at, at, c, n);   // its B is not used
        g.make(a, dy, marked, marks, w, p0 + at, at, c, n);
        if (tile > first) {
            dy.fetch(a.dy, a.g_stride, a, p0 - kScanTile + at, c, n);
            f.fetch(a.f, a.f_stride, a, p0 - kScanTile + at, c, n);
        }
        Map m[V];
        g.compose(t.a, m);
        scan_wave<true>(m, sums.m[tile & 1], lane, wave);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const float2 v = sums.m[tile & 1][k][lane % kLanes][i];
                const Map r = after(Map{A[i], B[i]}, Map{v.x, v.y});
                A[i] = r.A;
                B[i] = r.B;
            }
    }
    if (threadIdx.x < kLanes) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) a.maps[(size_t)part * a.C + c + i] = make_float2(A[i], B[i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_scan_backward(ScanArgs a) {
    constexpr int V = kVec<T>;
    __shared__ Sums<V> ahead, back;
    __shared__ Marks marks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = (int)(threadIdx.x / kLanes) * kEach;
    const int part = blockIdx.y, c = blockIdx.x * kWidth<T> + (lane % kLanes) * V, n = a.C - c;
    const int first = part * a.part_tiles, end = min(first + a.part_tiles, (a.T + kScanTile - 1) / kScanTile);
    if (a.last) pass_on<V>(a, a.dlast, a.last, part, c, n);
    if (first >= end) return;
    Rows<T> x, f, dy;
    auto fetch = [&](int tile) {
        x.fetch(a.x, a.x_stride, a, tile * kScanTile + at, c, n);
        f.fetch(a.f, a.f_stride, a, tile * kScanTile + at, c, n);
        dy.fetch(a.dy, a.g_stride, a, tile * kScanTile + at, c, n);
    };
    fetch(end - 1);
    Where w = where_begin(a);
    float carry[V];
    carry_in<true>(a, part, c, n, back.m[0], lane, wave, carry);
    for (int tile = end - 1; tile >= first; --tile) {
        const int p0 = tile * kScanTile;
        const bool marked = mark(a, p0, w, marks, lane);
        Tokens<T> t;
        Grads<T> g;
        t.make(a, x, f, marked, marks, w, p0 + at, at, c, n);
        g.make(a, dy, marked, marks, w, p0 + at, at, c, n);
        const Rows<T> xr = x, fr = f;
        if (tile > first) fetch(tile - 1);
        float kept[V];
        load_state(a.kept_in + (size_t)tile * a.C + c, n, kept);
        Map m[V], r[V];
        t.compose(m);
        g.compose(t.a, r);
        scan_wave<false>(m, ahead.m[tile & 1], lane, wave);
        scan_wave<true>(r, back.m[tile & 1], lane, wave);
        __syncthreads();
        float h[kEach + 1][V], G[V];   // the states before each token and after the last
        scan_apply<false>(m, ahead.m[tile & 1], lane, wave, kept, h[0]);
        scan_apply<true>(r, back.m[tile & 1], lane, wave, carry, G);
#pragma unroll
        for (int j = 0; j < kEach; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) h[j + 1][i] = apply(Map{t.a[j][i], t.b[j][i]}, h[j][i]);
#pragma unroll
        for (int j = kEach - 1; j >= 0; --j) {
            float xv[V], fv[V], dx[V], df[V];
            unpack(xr.v[j], xv);
            unpack(fr.v[j], fv);
            const int p = p0 + at + j;
            const bool none = marked && (p < w.lo || p >= w.hi);
            if (t.start[j] >= 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) h[j][i] = 0.f;
                if (a.state) load_state(a.state + (size_t)number_of(a, t.start[j]) * a.C + c, n, h[j]);
            }
            float ds[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float keep, take;
                gate<T>(fv[i], keep, take);
                const float dh = g.g[j][i] + G[i];
                dx[i] = none ? 0.f : take * dh;
                df[i] = none ? 0.f : dh * (h[j][i] - xv[i]) * (keep * take);
                ds[i] = keep * dh;
                G[i] = t.a[j][i] == 0.f ? 0.f : t.a[j][i] * dh;
            }
            if (p < a.T) {
                store_part(static_cast<T*>(a.y) + row_of(a, p) * a.C + c, n, dx);
                store_part(static_cast<T*>(a.df) + row_of(a, p) * a.C + c, n, df);
            }
            if (t.start[j] >= 0 && a.last && !none) store_state(a.last + (size_t)number_of(a, t.start[j]) * a.C + c, n, ds);
        }
    }
}

struct StepArgs {
    const void *x, *f;
    const float* state;
    void* y;
    float* out;
    long long x_stride, f_stride, rows;
    int C, chunks;   // chunks: of 16 bytes of x, a row
};

template <typename T>
__global__ void __launch_bounds__(256) k_scan_step(StepArgs a) {
    constexpr int V = kVec<T>;
    const long long all = a.rows * a.chunks;
    for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < all; u += (long long)gridDim.x * 256) {
        const long long row = u / a.chunks;
        const int c = (int)(u - row * a.chunks) * V, n = a.C - c;
        float x[V], f[V], h[V];
        unpack(load_raw(static_cast<const T*>(a.x) + row * a.x_stride + c, n), x);
        unpack(load_raw(static_cast<const T*>(a.f) + row * a.f_stride + c, n), f);
        load_state(a.state + row * a.C + c, n, h);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float keep, take;
            gate<T>(f[i], keep, take);
            h[i] = fmaf(keep, h[i], take * x[i]);
        }
        store_part(static_cast<T*>(a.y) + row * a.C + c, n, h);
        store_state(a.out + row * a.C + c, n, h);
    }
}

// Parts of the pack: enough workgroups to fill the chip four times.
struct Split {
    int groups, parts, part_tiles;   // groups: of channels
};
Split split_of(const wtc_scan_desc* d) {
    const int width = d->dtype == WTC_BF16 ? kWidth<uint16_t> : kWidth<float>;
    Split s;
    s.groups = (d->C + width - 1) / width;
    const long long tiles = (d->T + kScanTile - 1) / kScanTile;
    long long parts = 1024 / s.groups;
    parts = parts < 1 ? 1 : parts > tiles ? (tiles < 1 ? 1 : tiles) : parts;
    s.part_tiles = (int)((tiles + parts - 1) / parts);
    s.parts = s.part_tiles < 1 ? 1 : (int)((tiles + s.part_tiles - 1) / s.part_tiles);
    return s;
}

ScanArgs scan_args(const wtc_scan_desc* d, const Split& s, const void* x, const void* f, const int* cu, const float* state,
                   void* maps) {
    ScanArgs a = {};
    a.x = x; a.f = f; a.cu = cu; a.state = state; a.maps = static_cast<float2*>(maps);
    a.x_stride = d->x_stride; a.f_stride = d->f_stride; a.g_stride = d->g_stride;
    a.T = (int)d->T; a.n_seq = d->n_seq; a.C = d->C; a.reverse = d->reverse;
    a.parts = s.parts; a.part_tiles = s.part_tiles;
    return a;
}

template <typename T>
void run_forward(const ScanArgs& a, const Split& s, hipStream_t st) {
    if (s.parts > 1)
        hipLaunchKernelGGL(k_scan_parts<T>, dim3((unsigned)s.groups, (unsigned)(s.parts - 1)), dim3(256), 0, st, a);
    hipLaunchKernelGGL(k_scan_forward<T>, dim3((unsigned)s.groups, (unsigned)s.parts), dim3(256), 0, st, a);
}
template <typename T>
void run_backward(const ScanArgs& a, const Split& s, hipStream_t st) {
    if (s.parts > 1)
        hipLaunchKernelGGL(k_scan_parts_back<T>, dim3((unsigned)s.groups, (unsigned)(s.parts - 1)), dim3(256), 0, st, a);
    hipLaunchKernelGGL(k_scan_backward<T>, dim3((unsigned)s.groups, (unsigned)s.parts), dim3(256), 0, st, a);
}

}  // namespace

size_t scan_workspace(const wtc_scan_desc* d) {
    const Split s = split_of(d);
    return s.parts > 1 ? (size_t)s.parts * d->C * sizeof(float2) : 0;
}

int launch_scan_forward(const wtc_scan_desc* d, const void* x, const void* f, const int* cu, const float* state, void* y,
                        float* last, float* kept, void* workspace, void* stream) {
    const Split s = split_of(d);
    ScanArgs a = scan_args(d, s, x, f, cu, state, workspace);
    a.y = y; a.last = last; a.kept = kept;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16)
        run_forward<uint16_t>(a, s, st);
    else
        run_forward<float>(a, s, st);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_scan_backward(const wtc_scan_desc* d, const void* x, const void* f, const int* cu, const float* state,
                         const float* kept, const void* dy, const float* dlast, void* dx, void* df, float* dstate,
                         void* workspace, void* stream) {
    const Split s = split_of(d);
    ScanArgs a = scan_args(d, s, x, f, cu, state, workspace);
    a.kept_in = kept; a.dy = dy; a.dlast = dlast; a.y = dx; a.df = df; a.last = dstate;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16)
        run_backward<uint16_t>(a, s, st);
    else
        run_backward<float>(a, s, st);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_scan_step(const wtc_scan_desc* d, const void* x, const void* f, const float* state, void* y, float* out,
                     void* stream) {
    StepArgs a = {};
    const int V = d->dtype == WTC_BF16 ? kVec<uint16_t> : kVec<float>;
    a.x = x; a.f = f; a.state = state; a.y = y; a.out = out;
    a.x_stride = d->x_stride; a.f_stride = d->f_stride; a.rows = d->T; a.C = d->C; a.chunks = (d->C + V - 1) / V;
    const long long blocks = (a.rows * a.chunks + 255) / 256;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d->dtype == WTC_BF16)
        hipLaunchKernelGGL(k_scan_step<uint16_t>, grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(k_scan_step<float>, grid, dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace wtc
