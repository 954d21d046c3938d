// Gated linear recurrence inside each sequence of a pack:
//   a = sigmoid(f),  h_t = a_t h_(t-1) + (1 - a_t) x_t,  y = h
// from the sequence's first token to its last, or the other way, and its
// backward pass: with G_t = a_(t+1) dh_(t+1) (the last state's gradient at the end),
//   dh_t = dy_t + G_t,  dx = (1 - a) dh,  df = dh (h_(t-1) - x) a (1 - a).
//
// A thread walks the tokens of one part of the pack, two channels of them, with
// the state in registers: no lane waits for another, and the loads of the next
// tokens are on their way meanwhile.  What a part does to the state that enters
// it is a map h -> A h + B.  With several parts a first kernel computes each
// part's map, and a second one composes them to the state that each part begins
// with.  A map needs only the tokens behind the part's last sequence start
// (before its first end, in the backward pass), so that little is read twice
// where sequences are short.  A sequence that starts in the part is marked by A <
// 0: nothing is then taken from what came before, not even a NaN.  An A of 0 is
// one that became too small for float32; a NaN and an infinity pass it, as they
// would pass every one of the part's steps.
//
// Eight tokens are taken as if all were finite, where no sequence starts or ends
// among them; if that leaves a NaN where there was none, they are taken again with
// a look for infinities.  Packs full of these: 2 x 65536 x 512 bf16 192 us forward
// and 342 backward for 141 and 212.  What the check costs the others shows in a
// single part, 64 tokens 19.7 us backward for 18.9 without.
//
// Bound by device memory: 3 T C e bytes forward (x, f in, y out), 5 T C e
// backward (x, f, dy in, dx, df out), and the maps' reading of two tensors in
// long sequences, which is 2 T C e more in either pass: the price of all parts
// being walked at once.  The forward pass keeps the state of every 8th token (4
// bytes a channel) for the backward pass, which computes the others again (every
// 16th, half the memory: 139 us backward for 125).  All of it is float32.
// Measured: 2 sequences of 65536 x 512 bf16, forward maps 69 us, starts 7, the
// states 73 (436 MB with what is kept, 6.0 TB/s, the inputs partly from the
// last-level cache), backward 65, 7 and 130 (738 MB, 5.7 TB/s); float32 28782 x
// 387 22 + 5 + 26 us; one token of 128 sequences of 768 channels 3.0 us.  Two
// channels of four tokens ahead instead of eight: 107 us for 101 of 130219 x 384;
// sixteen: no gain, and twice the registers.  The backward pass of bfloat16 stays
// within 128 registers, four waves a vector unit: with 129, 150 us for 130.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"
#include "wtc_tok_scan.h"

namespace wtc {
namespace {

constexpr int V = 2;                  // channels of a thread
constexpr int kAhead = 8;              // tokens whose loads are on their way together
static_assert(kScanKept % kAhead == 0, "what is kept is kept at the start of a step");

struct ScanArgs {
    const void *x, *f, *dy;
    const int* cu;
    const float *state, *dlast, *kept_in;
    void *y, *df;                // y: dx in the backward pass
    float *last, *kept;          // last: the gradient of state in the backward pass
    float2* maps;                // [parts][C]
    float* starts;               // [parts][C]: the state that a part begins with
    long long x_stride, f_stride, g_stride;
    int T, n_seq, C, pairs, reverse, parts, len;   // pairs: of channels; len: tokens of a part
    unsigned blocks;             // workgroups that walk parts
};

// ------------------------------------------------------------------ two channels
// Two elements as they lie in memory.  ONE: rows of a single channel; else the
// last thread of a row has its last two, the first of which may be another's
// too: both then compute and store the same.
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(4)));
template <typename T>
struct Two {
    uint32_t u[sizeof(T) / 2];
};
template <bool ONE, typename T>
__device__ __forceinline__ Two<T> load_two(const T* p) {
    Two<T> r;
    if constexpr (sizeof(T) == 2) {
        r.u[0] = ONE ? (uint32_t)p[0] : *reinterpret_cast<const u32_any*>(p);
    } else if constexpr (ONE) {
        r.u[0] = __builtin_bit_cast(uint32_t, p[0]);
        r.u[1] = 0u;
    } else {
        const u32x2_any v = *reinterpret_cast<const u32x2_any*>(p);
        r.u[0] = v[0];
        r.u[1] = v[1];
    }
    return r;
}
template <typename T>
__device__ __forceinline__ float value(const Two<T>& r, int i) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(float, i ? r.u[0] & 0xFFFF0000u : r.u[0] << 16);
    return __builtin_bit_cast(float, r.u[i % (sizeof(T) / 2)]);
}
template <bool ONE, typename T>
__device__ __forceinline__ void store_two(T* p, const float (&v)[V]) {
    if constexpr (ONE) {
        p[0] = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<u32_any*>(p) = bf16x2_rne(v[0], v[1]);
    } else {
        *reinterpret_cast<u32x2_any*>(p) = u32x2_any{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1])};
    }
}
template <bool ONE>
__device__ __forceinline__ void load_state(const float* p, float (&v)[V]) {
    const Two<float> r = load_two<ONE>(p);
    v[0] = value(r, 0);
    v[1] = value(r, 1);
}

// A token's gate: with e = exp(-|f|) the smaller of a and 1 - a is e / (1 + e),
// the larger 1 less that.  The state then moves from the nearer of itself and
// the input by the smaller one's share of their difference: the same as a h +
// (1 - a) x, but where a is close to 1 an error of a's last bit, made again in
// each step, does not add up over 1 / (1 - a) of them.
//   float32: the exponent's product is rounded at its own size, so exp is of
// float32's accuracy only with its lower part, and the reciprocal with a Newton
// step; what bfloat16 holds of f is coarser than either.
struct Gate {
    float m;   // the smaller one, negative if that is a
    __device__ __forceinline__ bool slow() const { return __builtin_bit_cast(int, m) >= 0; }   // a is the larger
};
template <typename T>
__device__ __forceinline__ Gate gate(float f) {
    constexpr float L = 1.4426950408889634f;
    const float t = -fabsf(f) * L;
    float e = __builtin_amdgcn_exp2f(t);
    if constexpr (sizeof(T) == 4) {
        const float v = fabsf(f) < 200.f ? f : 0.f;   // beyond, e is 0 (an infinity's lower part would be a NaN)
        const float low = fmaf(-fabsf(v), L, fabsf(v) * L) - fabsf(v) * 1.9259629911266175e-8f;
        e = fmaf(e, low * 0.6931471805599453f, e);
    }
    const float d = 1.f + e;
    float r = __builtin_amdgcn_rcpf(d);
    if constexpr (sizeof(T) == 4) r = fmaf(fmaf(-d, r, 1.f), r, r);
    const float m = e * r;
    return {f >= 0.f ? m : -m};
}
// a h + (1 - a) x, a v, (1 - a) v, and a (1 - a) v.  Differences make a NaN of an infinity that should stay one (and so
// does a gate that became 0): ANY looks for infinities, whose step is their sum, and is for what turned into a NaN.
template <bool ANY = false>
__device__ __forceinline__ float move(const Gate& g, float h, float x) {
    const float v = fmaf(g.m, x - h, g.slow() ? h : x);
    return ANY && (isinf(h) || isinf(x)) ? (h + x) + (g.m - g.m) : v;
}
template <bool ANY = false>
__device__ __forceinline__ float keep(const Gate& g, float v) {
    const float w = fmaf(g.m, -v, g.slow() ? v : 0.f);
    return ANY && isinf(v) ? v + (g.m - g.m) : w;
}
__device__ __forceinline__ float take(const Gate& g, float v) { return (g.slow() ? g.m : 1.f + g.m) * v; }
__device__ __forceinline__ float both(const Gate& g, float v) { return fabsf(g.m) * (1.f - fabsf(g.m)) * v; }

// A value of the two became a NaN (first, their sum: one comparison where there is none).
__device__ __forceinline__ bool turned(const float (&before)[V], const float (&now)[V]) {
    return __builtin_expect(isnan(now[0] + now[1]), 0) && ((isnan(now[0]) && !isnan(before[0])) || (isnan(now[1]) && !isnan(before[1])));
}
typedef std::false_type Finite;   // how a step is taken, see move
typedef std::true_type Any;

// ------------------------------------------------------------------ places
// Places of a pack in the order they are walked: place p is token p, or with
// `reverse` token T - 1 - p.  Sequence s = 0 .. n_seq - 1 in that order is
// places begin(s) .. begin(s + 1) - 1.
__device__ __forceinline__ int begin_of(const ScanArgs& a, int s) {
    const int v = min(max(a.cu[a.reverse ? a.n_seq - s : s], 0), a.T);
    return a.reverse ? a.T - v : v;
}
__device__ __forceinline__ size_t state_of(const ScanArgs& a, int s, int c) {
    return (size_t)(a.reverse ? a.n_seq - 1 - s : s) * a.C + c;
}
__device__ __forceinline__ long long row_of(const ScanArgs& a, int p) { return a.reverse ? a.T - 1 - p : p; }

// The sequence of a place: its number, and the places from .. to - 1 of it.
// Places of no sequence have number -1.
struct Where {
    int s, from, to;
};
__device__ __forceinline__ Where find(const ScanArgs& a, int p) {
    int lo = -1, hi = a.n_seq;   // begin(lo) <= p < begin(hi), as far as those are sequences
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (begin_of(a, mid) <= p)
            lo = mid;
        else
            hi = mid;
    }
    if (lo >= 0) {
        const Where w = {lo, begin_of(a, lo), begin_of(a, lo + 1)};
        if (p >= w.from && p < w.to) return w;
        if (lo == a.n_seq - 1 && p >= w.to) return {-1, w.to, a.T};
    } else if (a.n_seq > 0) {
        return {-1, 0, begin_of(a, 0)};
    }
    return {-1, p, p + 1};
}
// That of place p, which lies in the sequence after w's (before it) or anywhere else.
template <bool BACK>
__device__ __forceinline__ void move_to(const ScanArgs& a, int p, Where& w) {
    if (p >= w.from && p < w.to) return;
    const int s = BACK ? w.s - 1 : w.s + 1;
    if (w.s >= 0 && s >= 0 && s < a.n_seq) {
        const Where next = BACK ? Where{s, begin_of(a, s), w.from} : Where{s, w.to, begin_of(a, s + 1)};
        if (p >= next.from && p < next.to) {
            w = next;
            return;
        }
    }
    w = find(a, p);
}

// A thread's part and channels.
struct Mine {
    int part, c;
};
template <bool ONE>
__device__ __forceinline__ Mine mine_of(const ScanArgs& a) {
    const unsigned id = blockIdx.x * 256u + threadIdx.x;
    const int part = (int)(id / (unsigned)a.pairs);
    return {part, ONE ? 0 : min((int)(id % (unsigned)a.pairs) * V, a.C - V)};
}

// Rows of tokens p .. p + N - 1, as they lie in memory; those from `end` on are the last one's.
template <typename T, bool ONE, int N>
struct Rows {
    Two<T> v[N];
    __device__ __forceinline__ void fetch(const void* base, long long stride, const ScanArgs& a, int p, int end, int c) {
        const T* q = static_cast<const T*>(base) + c;
        const long long step = a.reverse ? -stride : stride;
        q += row_of(a, min(p, end - 1)) * stride;
        const int there = end - p;
        if (there >= N) {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = load_two<ONE>(q + j * step);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = load_two<ONE>(q + (j < there ? j : max(there - 1, 0)) * step);
        }
    }
};

// ------------------------------------------------------------------ maps of parts
constexpr float kCut = -1.f;   // in A's place: what comes before does not count
template <typename T, bool BACK, bool ONE>
__global__ void __launch_bounds__(256) k_scan_maps(ScanArgs a) {
    auto [part, c] = mine_of<ONE>(a);
    if (BACK) ++part;                     // the first has none; forward, the last
    if (part >= (BACK ? a.parts : a.parts - 1)) return;
    const int first = part * a.len, end = part_end(first, a.len, a.T);
    float A[V] = {}, B[V] = {};
    const Where w = find(a, BACK ? first : end - 1);
    int from = first, to = first;         // the places that count; with none the state is zero
    bool cut = true;
    if (BACK ? w.s >= 0 && w.from < first : w.s >= 0) {
        cut = BACK ? w.to <= end : w.from >= first;   // the sequence ends (starts) in the part
        from = BACK ? first : max(w.from, first);
        to = BACK ? min(w.to, end) : end;
        const float* in = BACK ? a.dlast : a.state;
        if (cut && in) load_state<ONE>(in + state_of(a, w.s, c), B);
#pragma unroll
        for (int i = 0; i < V; ++i) A[i] = 1.f;
    }
    const void* xs = BACK ? a.dy : a.x;
    const long long stride = BACK ? a.g_stride : a.x_stride;
    Rows<T, ONE, kAhead> x, f;
    // BACK: the tokens up to place q - 1, from the last one
    auto fetch = [&](int q) {
        const int p = BACK ? max(q - kAhead, from) : q;
        x.fetch(xs, stride, a, p, to, c);
        f.fetch(a.f, a.f_stride, a, p, to, c);
    };
    if (from < to) fetch(BACK ? to : from);
    for (int done = 0; done < to - from; done += kAhead) {
        const int count = min(to - from - done, kAhead);
        const Rows<T, ONE, kAhead> xr = x, fr = f;
        if (done + kAhead < to - from) fetch(BACK ? to - done - kAhead : from + done + kAhead);
        const float before[V] = {B[0], B[1]};
        auto tokens = [&](auto any) {
            constexpr bool ANY = decltype(any)::value;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = BACK ? kAhead - 1 - k : k;
                const bool there = j < count;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const Gate g = gate<T>(value(fr.v[j], i));
                    const float in = value(xr.v[j], i);
                    const float next = BACK ? keep<ANY>(g, in + B[i]) : move<ANY>(g, B[i], in);
                    if (!ANY) A[i] = there ? keep(g, A[i]) : A[i];
                    B[i] = there ? next : B[i];
                }
            }
        };
        tokens(Finite());
        if (turned(before, B)) {
            B[0] = before[0];
            B[1] = before[1];
            tokens(Any());
        }
    }
#pragma unroll
    for (int i = 0; i < (ONE ? 1 : V); ++i) a.maps[(size_t)part * a.C + c + i] = make_float2(cut ? kCut : A[i], B[i]);
}

// The state that each part begins with (BACK: G behind its last token): 128
// threads of a channel have up to kRun parts each, in order, and take what the
// threads before them leave.
constexpr int kRun = kMostParts / 128, kCols = 8;
template <bool ANY>   // see move; an A of 0 keeps an infinity too
__device__ __forceinline__ float apply(const float2& m, float h) {
    const float v = ANY && isinf(h) ? (h + m.y) + (m.x - m.x) : fmaf(m.x, h, m.y);
    return m.x < 0.f ? m.y : v;
}
// first one, then the other
template <bool ANY>
__device__ __forceinline__ float2 after(const float2& one, const float2& other) {
    return make_float2(one.x < 0.f || other.x < 0.f ? kCut : other.x * one.x, apply<ANY>(other, one.y));
}

template <bool BACK>
__global__ void __launch_bounds__(1024) k_scan_starts(ScanArgs a) {
    __shared__ float2 whole[16][kCols];   // of a wave's eight threads of a channel
    __shared__ bool some[16];             // a wave has met an infinity
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane % kCols, c = blockIdx.x * kCols + col;
    const int run = (a.parts + 127) / 128, first = (int)(threadIdx.x / kCols) * run;
    auto part_of = [&](int k) { return BACK ? a.parts - 1 - k : k; };
    auto map_of = [&](int k) {   // the last part's map (BACK: the first one's) is not there, nor needed
        const bool there = k < run && first + k + 1 < a.parts && c < a.C;
        return there ? a.maps[(size_t)part_of(first + k) * a.C + c] : make_float2(1.f, 0.f);
    };
    auto start = [&](int k, float h) {
        if (k < run && first + k < a.parts && c < a.C) a.starts[(size_t)part_of(first + k) * a.C + c] = h;
    };
    auto join = [&](float2 all, auto any) {   // with the threads before it in the wave
#pragma unroll
        for (int o = kCols; o < 64; o <<= 1) {
            const float2 p = make_float2(__shfl_up(all.x, o), __shfl_up(all.y, o));
            if (lane >= o) all = after<decltype(any)::value>(p, all);
        }
        return all;
    };
    float2 m[kRun];
    float2 all = make_float2(1.f, 0.f);
    bool infinite = false;
#pragma unroll
    for (int k = 0; k < kRun; ++k) m[k] = map_of(k);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        infinite |= isinf(m[k].y);
        all = after<false>(all, m[k]);
    }
    all = join(all, Finite());
    const bool rare = __builtin_amdgcn_ballot_w64(infinite) != 0;
    if (__builtin_expect(rare, 0)) {
        all = make_float2(1.f, 0.f);
#pragma unroll 1
        for (int k = 0; k < run; ++k) all = after<true>(all, map_of(k));
        all = join(all, Any());
    }
    if (lane >= 64 - kCols) whole[wave][col] = all;
    if (lane == 0) some[wave] = rare;
    const float2 p = make_float2(__shfl_up(all.x, kCols), __shfl_up(all.y, kCols));
    __syncthreads();
    float h = 0.f;
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(some[lane & 15]) == 0, 1)) {
        for (int w = 0; w < wave; ++w) h = apply<false>(whole[w][col], h);
        if (lane >= kCols) h = apply<false>(p, h);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            start(k, h);
            h = apply<false>(m[k], h);
        }
    } else {
        for (int w = 0; w < wave; ++w) h = apply<true>(whole[w][col], h);
        if (lane >= kCols) h = apply<true>(p, h);
#pragma unroll 1
        for (int k = 0; k < run; ++k) {
            start(k, h);
            h = apply<true>(map_of(k), h);
        }
    }
}

// What sequences with no token leave behind, by the workgroups from a.blocks on.
template <bool ONE>
__device__ __forceinline__ void pass_on(const ScanArgs& a, const float* from, float* to) {
    const long long step = (long long)(gridDim.x - a.blocks) * 256;
    for (long long u = (long long)(blockIdx.x - a.blocks) * 256 + threadIdx.x; u < (long long)a.n_seq * a.pairs; u += step) {
        const int s = (int)(u / a.pairs), c = ONE ? 0 : min((int)(u - (long long)s * a.pairs) * V, a.C - V);
        if (begin_of(a, s + 1) > begin_of(a, s)) continue;
        float v[V] = {};
        if (from) load_state<ONE>(from + state_of(a, s, c), v);
        store_two<ONE>(to + state_of(a, s, c), v);
    }
}

// ------------------------------------------------------------------ forward
template <typename T, bool ONE>
__global__ void __launch_bounds__(256) k_scan_forward(ScanArgs a) {
    if (blockIdx.x >= a.blocks) return pass_on<ONE>(a, a.state, a.last);
    const auto [part, c] = mine_of<ONE>(a);
    if (part >= a.parts) return;
    const int first = part * a.len, end = part_end(first, a.len, a.T);
    if (first >= end) return;
    Rows<T, ONE, kAhead> x, f;
    x.fetch(a.x, a.x_stride, a, first, end, c);
    f.fetch(a.f, a.f_stride, a, first, end, c);
    float h[V] = {};
    if (part > 0) load_state<ONE>(a.starts + (size_t)part * a.C + c, h);
    Where w = find(a, first);
    const long long step = a.reverse ? -a.C : a.C;
    for (int p0 = first; p0 < end; p0 += kAhead) {
        const Rows<T, ONE, kAhead> xr = x, fr = f;
        if (p0 + kAhead < end) {
            x.fetch(a.x, a.x_stride, a, p0 + kAhead, end, c);
            f.fetch(a.f, a.f_stride, a, p0 + kAhead, end, c);
        }
        if (a.kept && p0 % kScanKept == 0) store_two<ONE>(a.kept + (size_t)(p0 / kScanKept) * a.C + c, h);
        T* y = static_cast<T*>(a.y) + row_of(a, p0) * a.C + c;
        auto token = [&](int j, auto any) {
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = move<decltype(any)::value>(gate<T>(value(fr.v[j], i)), h[i], value(xr.v[j], i));
        };
        bool plain = w.s >= 0 && p0 > w.from && p0 + kAhead < w.to;   // no start and no end
        if (plain) {
            const float before[V] = {h[0], h[1]};
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                token(j, Finite());
                store_two<ONE>(y + j * step, h);
            }
            if (turned(before, h)) {
                plain = false;
                h[0] = before[0];
                h[1] = before[1];
            }
        }
        if (!plain) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int p = p0 + j;
                if (p >= end) break;
                move_to<false>(a, p, w);
                if (w.s < 0) {
                    h[0] = h[1] = 0.f;
                } else {
                    if (p == w.from) {
                        h[0] = h[1] = 0.f;
                        if (a.state) load_state<ONE>(a.state + state_of(a, w.s, c), h);
                    }
                    token(j, Any());
                    if (p + 1 == w.to && a.last) store_two<ONE>(a.last + state_of(a, w.s, c), h);
                }
                store_two<ONE>(y + j * step, h);
            }
        }
    }
}

// ------------------------------------------------------------------ backward
// From the last token to the first, kScanKept at a time: their states again from
// the kept one, and then the gradients.
template <typename T, bool ONE>
__global__ void __launch_bounds__(256) k_scan_backward(ScanArgs a) {
    constexpr int N = kScanKept;
    if (blockIdx.x >= a.blocks) return pass_on<ONE>(a, a.dlast, a.last);
    const auto [part, c] = mine_of<ONE>(a);
    if (part >= a.parts) return;
    const int first = part * a.len, end = part_end(first, a.len, a.T);
    if (first >= end) return;
    float G[V] = {};
    if (part + 1 < a.parts) load_state<ONE>(a.starts + (size_t)part * a.C + c, G);
    Where w = find(a, end - 1);
    const long long step = a.reverse ? -a.C : a.C;
    bool again = false;   // the same tokens, as the ones with a start or an end among them are taken
    for (int p0 = first + (end - first - 1) / N * N; p0 >= first; p0 -= again ? 0 : N) {
        Rows<T, ONE, N> x, f, dy;
        x.fetch(a.x, a.x_stride, a, p0, end, c);
        f.fetch(a.f, a.f_stride, a, p0, end, c);
        dy.fetch(a.dy, a.g_stride, a, p0, end, c);
        float now[V], h[N][V];   // h: the states before each token
        Gate g[N][V];
        load_state<ONE>(a.kept_in + (size_t)(p0 / N) * a.C + c, now);
        const long long to = row_of(a, p0) * a.C + c;
        T *dx = static_cast<T*>(a.y) + to, *df = static_cast<T*>(a.df) + to;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) g[j][i] = gate<T>(value(f.v[j], i));
        auto forward = [&](int j, auto any) {
#pragma unroll
            for (int i = 0; i < V; ++i) now[i] = move<decltype(any)::value>(g[j][i], now[i], value(x.v[j], i));
        };
        auto token = [&](int j, auto any) {   // G becomes what the token hands to the one before it
            float vx[V], vf[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float dh = G[i] + value(dy.v[j], i);
                vx[i] = take(g[j][i], dh);
                vf[i] = both(g[j][i], dh) * (h[j][i] - value(x.v[j], i));
                G[i] = keep<decltype(any)::value>(g[j][i], dh);
            }
            store_two<ONE>(dx + j * step, vx);
            store_two<ONE>(df + j * step, vf);
        };
        if (w.s >= 0 && p0 > w.from && p0 + N < w.to && !again) {   // no start and no end
            const float behind[V] = {G[0], G[1]};
#pragma unroll
            for (int j = 0; j < N; ++j) {
#pragma unroll
                for (int i = 0; i < V; ++i) h[j][i] = now[i];
                if (j + 1 < N) forward(j, Finite());
            }
            again = turned(h[0], now);
#pragma unroll
            for (int j = N - 1; j >= 0; --j) token(j, Finite());
            again |= turned(behind, G);
            if (again) {
                G[0] = behind[0];
                G[1] = behind[1];
            }
        } else {
            again = false;
            const Where last = w;
            Where up = find(a, p0);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int p = p0 + j;
                if (p < end) {
                    move_to<false>(a, p, up);
                    if (p == up.from) {   // of a sequence, or a place of none
                        now[0] = now[1] = 0.f;
                        if (up.s >= 0 && a.state) load_state<ONE>(a.state + state_of(a, up.s, c), now);
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) h[j][i] = now[i];
                if (j + 1 < N) forward(j, Any());
            }
            w = last;
#pragma unroll
            for (int j = N - 1; j >= 0; --j) {
                const int p = p0 + j;
                if (p >= end) continue;
                move_to<true>(a, p, w);
                if (w.s < 0) {
                    const float zero[V] = {};
                    store_two<ONE>(dx + j * step, zero);
                    store_two<ONE>(df + j * step, zero);
                    G[0] = G[1] = 0.f;
                    continue;
                }
                if (p + 1 == w.to) {
                    G[0] = G[1] = 0.f;
                    if (a.dlast) load_state<ONE>(a.dlast + state_of(a, w.s, c), G);
                }
                token(j, Any());
                if (p == w.from && a.last) store_two<ONE>(a.last + state_of(a, w.s, c), G);
            }
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

// One float per channel of a row of the states.
template <int N>
__device__ __forceinline__ void load_states(const float* row, int n, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float part[4];
        load_part(row + i, n - i, part);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = part[j];
    }
}
template <int N>
__device__ __forceinline__ void store_states(float* row, int n, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float part[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
        store_part(row + i, n - i, part);
    }
}

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
        load_states(a.state + row * a.C + c, n, h);
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = move<true>(gate<T>(f[i]), h[i], x[i]);
        store_part(static_cast<T*>(a.y) + row * a.C + c, n, h);
        store_states(a.out + row * a.C + c, n, h);
    }
}

ScanArgs scan_args(const wtc_scan_desc* d, const ScanSplit& s, const void* x, const void* f, const int* cu, const float* state,
                   void* workspace) {
    ScanArgs a = {};
    a.x = x; a.f = f; a.cu = cu; a.state = state;
    a.maps = static_cast<float2*>(workspace);
    a.starts = reinterpret_cast<float*>(a.maps + (size_t)s.parts * d->C);
    a.x_stride = d->x_stride; a.f_stride = d->f_stride; a.g_stride = d->g_stride;
    a.T = (int)d->T; a.n_seq = d->n_seq; a.C = d->C; a.pairs = (d->C + 1) / 2; a.reverse = d->reverse;
    a.parts = s.parts; a.len = s.len;
    return a;
}

template <typename T, bool BACK, bool ONE>
void run_scan(ScanArgs a, hipStream_t st) {
    a.blocks = (unsigned)(((long long)a.parts * a.pairs + 255) / 256);
    if (a.parts > 1) {
        hipLaunchKernelGGL((k_scan_maps<T, BACK, ONE>), dim3(a.blocks), dim3(256), 0, st, a);
        hipLaunchKernelGGL(k_scan_starts<BACK>, dim3((unsigned)((a.C + kCols - 1) / kCols)), dim3(1024), 0, st, a);
    }
    // Workgroups of their own look for sequences with no token.  By the parts' threads, 30 tokens of 384 channels beside 4096
    // such sequences took 862 us forward, a thread after 4096 others' bounds.
    const long long pass = a.last ? ((long long)a.n_seq * a.pairs + 255) / 256 : 0;
    const dim3 grid(a.blocks + (unsigned)(pass < 2048 ? pass : 2048));
    if constexpr (BACK)
        hipLaunchKernelGGL((k_scan_backward<T, ONE>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_scan_forward<T, ONE>), grid, dim3(256), 0, st, a);
}
template <typename T, bool BACK>
void run_scan(const ScanArgs& a, hipStream_t st) {
    a.C == 1 ? run_scan<T, BACK, true>(a, st) : run_scan<T, BACK, false>(a, st);
}

}  // namespace

size_t scan_workspace(const wtc_scan_desc* d) {
    const ScanSplit s = scan_split(d->T, d->C);
    return s.parts > 1 ? (size_t)s.parts * d->C * (sizeof(float2) + sizeof(float)) : 0;
}

int launch_scan_forward(const wtc_scan_desc* d, const void* x, const void* f, const int* cu, const float* state, void* y,
                        float* last, float* kept, void* workspace, void* stream) {
    const ScanSplit s = scan_split(d->T, d->C);
    ScanArgs a = scan_args(d, s, x, f, cu, state, workspace);
    a.y = y; a.last = last; a.kept = kept;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    d->dtype == WTC_BF16 ? run_scan<uint16_t, false>(a, st) : run_scan<float, false>(a, st);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

int launch_scan_backward(const wtc_scan_desc* d, const void* x, const void* f, const int* cu, const float* state,
                         const float* kept, const void* dy, const float* dlast, void* dx, void* df, float* dstate,
                         void* workspace, void* stream) {
    const ScanSplit s = scan_split(d->T, d->C);
    ScanArgs a = scan_args(d, s, x, f, cu, state, workspace);
    a.kept_in = kept; a.dy = dy; a.dlast = dlast; a.y = dx; a.df = df; a.last = dstate;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    d->dtype == WTC_BF16 ? run_scan<uint16_t, true>(a, st) : run_scan<float, true>(a, st);
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
