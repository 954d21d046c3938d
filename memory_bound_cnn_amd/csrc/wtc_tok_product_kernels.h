// The experts' products, of the rows x[r] of each expert e (rows cu[e] to
// cu[e + 1] - 1) with its weights W[e] [N, K]:
//   k_product_rows, forward   y[r]  = W[e] x[r] + b[e]          terms K, columns N
//   k_product_rows, back      dx[r] = dy[r] W[e]                 terms N, columns K
//   k_product_few             the forward one, of a few rows
//   k_product_weights         dW[e] = sum_r dy[r] x[r]^T,  db[e] = sum_r dy[r]
//
// Bound by the matrix units where there are many rows, and by the weights' way from memory where there are few.  A
// workgroup's tiles of the two operands are copied to shared memory a step ahead, and read from there half a step ahead,
// of their products.  Measured: 50176 rows of 8 uneven experts, 1024 -> 4096, bfloat16: 401 to 452 us forward (1050 to 930
// TFLOP/s), 416 to 469 for the input's gradient, 372 to 511 for the weights' (one kernel over and over, and all in turn as a
// training step has them, when the card's power holds the clocks down; a library product of the same size and one expert:
// 383, 429 and 594); matrix units busy 60 to 68 % of the time.  The copies' way is what holds the large tiles back: without
// them (timed alone, on tiles that do not change) the loop runs at 1200 to 1300 TFLOP/s, at the clocks that power allows.
// float32, 6007 rows of 5 experts, 392 -> 1544: 74 to 79 us forward, 90 to 99 for the input's gradient, 82 to 91 and 8 for
// the weights' (98, 81 and 84 TFLOP/s at best; the float32 matrix instructions reach 153), where splitting the factors in
// three takes the vector units 54 to 59 % of the time and the products the matrix units 37 to 46, side by side for little
// of it.
#pragma once

#include <limits.h>

#include <type_traits>

#include "wtc_tok_product.h"

namespace wtc {
namespace product {

struct Args {
    const void *x, *w, *b;      // x: dy in the backward pass
    const void* g;              // k_product_weights: dy, beside x
    const int* cu;
    void* y;                    // dx, dW
    void* db;
    float* parts;               // k_product_weights: sums of experts' parts, [slots][N][K], then [slots][N]
    long long x_stride, g_stride, slots;
    long long first;            // k_product_rows: of the launch's slots
    int R, E, K, N, rows;       // rows: of a part of an expert, about
};

// For the weights' gradients an expert's rows are taken in `parts` equal parts, of 5/8 to 5/4 of `rows` each, or in one if
// it has less.  Parts of experts with several have a place for their sums, in the experts' order.
struct Part {
    int expert, part, parts, place;   // place: of the expert's first part
};
__host__ __device__ __forceinline__ int parts_of(int count, int rows) {
    const int n = (int)((count + 3LL * rows / 4) / rows);
    return n < 1 ? 1 : n;
}
inline long long most_parts(long long R, int E, int rows) { return E + R / rows; }
inline long long most_places(long long R, int rows) {   // parts of an expert with several: at most 8/5 of its rows / `rows`
    return 4 * R < 5LL * rows ? 0 : (8 * R + 5LL * rows - 1) / (5LL * rows);
}
// The number-th part: of up to 16 experts those with the longest parts first, beyond in the experts' order (parts are then
// many to a place, and finding the order takes longer than it gives).  expert -1: none.
__device__ __forceinline__ Part find_part(const int* cu, int E, int R, int rows, int number, int lane) {
    constexpr int RANKED = 16;
    int before = 0, place = 0;   // parts and places of the experts before the 64 at e0
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        const int count = e < E ? max(segment_begin(cu, E, R, e + 2) - segment_begin(cu, E, R, e + 1), 0) : 0;
        const int parts = e < E ? parts_of(count, rows) : 0, length = parts > 0 ? count / parts : 0;
        int first = parts, mine = parts > 1 ? parts : 0;   // parts and places up to this expert
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int p = __shfl_up(first, o), m = __shfl_up(mine, o);
            if (lane >= o) first += p, mine += m;
        }
        const int all = __builtin_amdgcn_readlane(first, 63), places = __builtin_amdgcn_readlane(mine, 63);
        first -= parts;
        mine -= parts > 1 ? parts : 0;
        if (E <= RANKED) {
            first = 0;
            for (int i = 0; i < E; ++i) {
                const int l = __builtin_amdgcn_readlane(length, i);
                if (l > length || (l == length && i < lane)) first += __builtin_amdgcn_readlane(parts, i);
            }
        }
        first += before;
        const uint64_t found = __builtin_amdgcn_ballot_w64(e < E && number >= first && number < first + parts);
        if (found) {
            const int at = __builtin_ctzll(found);
            return {e0 + at, number - __builtin_amdgcn_readlane(first, at), __builtin_amdgcn_readlane(parts, at),
                    place + __builtin_amdgcn_readlane(mine, at)};
        }
        before += all;
        place += places;
    }
    return {-1, 0, 0, 0};
}

// With rows in no order experts can have more of them together than there are: those without a place remain whole.
__device__ __forceinline__ bool no_place(const Args& a, int place, int parts) { return parts > 1 && place + parts > a.slots; }

// Waits until at most N of the wave's copies are on their way.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Half a step's terms of a wave's blocks, as they lie in shared memory, and their products.
template <typename T, int NB, int MB, bool INTERLEAVE>
struct Half {
    static constexpr int READS = 64 / (int)sizeof(T) / kRead;
    Eight<T> a[READS][NB], b[READS][MB];
    static constexpr int LOADS = READS * (NB + MB), PRODUCTS = READS * NB * MB;
    template <typename Cols, typename RowsOp>
    __device__ __forceinline__ void read_one(int i, const char* cols, const char* rows, int cpart, int rpart, int col0, int row0,
                                             int lane, int half) {
        const int at = i / (NB + MB), block = i % (NB + MB);
        if (block < NB)
            a[at][block] = Cols::read(cols, cpart, col0 + 32 * block, READS * half + at, lane);
        else
            b[at][block - NB] = RowsOp::read(rows, rpart, row0 + 32 * (block - NB), READS * half + at, lane);
    }
    template <typename Cols, typename RowsOp>
    __device__ __forceinline__ void read(const char* cols, const char* rows, int cpart, int rpart, int col0, int row0, int lane,
                                         int half) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) read_one<Cols, RowsOp>(i, cols, rows, cpart, rpart, col0, row0, lane, half);
    }
    // f(n) behind the n-th product, where its instructions stay.
    template <typename F>
    __device__ __forceinline__ void products(Sum<T, f32x16> (&acc)[MB][NB], const F& f) const {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) {
            const int at = n / (MB * NB), mb = n / NB % MB, nb = n % NB;
            mma(frag(a[at][nb]), frag(b[at][mb]), acc[mb][nb]);
            __builtin_amdgcn_sched_barrier(0);
            f(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void products(Sum<T, f32x16> (&acc)[MB][NB]) const {
        // reads and products in turn, or what was to be read is on its way before the first product
        if (!INTERLEAVE) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int at = 0; at < READS; ++at) {
            Frag<T> fa[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fa[nb] = frag(a[at][nb]);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const Frag<T> fb = frag(b[at][mb]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma(fa[nb], fb, acc[mb][nb]);
            }
        }
        if (INTERLEAVE) {
#pragma unroll
            for (int i = 0; i < PRODUCTS; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);     // a matrix instruction
                if ((i + 1) * LOADS / PRODUCTS > i * LOADS / PRODUCTS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // a read
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
};

// Steps begin .. end - 1 with STAGES buffers: copy(s, buffer) sends a step's tiles on their way (COPIES of a wave),
// read(half, set, buffer) reads half a step, last(buffer) clears what the final step lacks.  A half is read while the
// one before it is multiplied.
//   SPREAD: a step's second half has the copies and reads one by one between its products (copy's and read's last
// argument is which one) instead of all before the first: for one workgroup a unit, whose waves are all at this point at
// once.  256 x 256, 50176 rows x 1024 -> 4096: 426 -> 401 us forward, 428 -> 416 back.  With two workgroups the other's
// products fill the time, and the products between the copies come late: 128 x 128, 449 -> 479, 459 -> 501.
template <typename Set, int STAGES, int COPIES, bool SPREAD, typename Copy, typename Read, typename Last, typename Products>
__device__ __forceinline__ void run_steps(int begin, int end, bool partial, const Copy& copy, const Read& read, const Last& last,
                                          const Products& products) {
    if (begin >= end) return;
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
        if (begin + s < end) copy(begin + s, s);
    if (begin + STAGES <= end)
        wait_copies<(STAGES - 1) * COPIES>();
    else
        wait_copies<0>();
    meet();
    if (partial && begin + 1 == end) {
        last(0);
        meet();
    }
    Set p, q;
    read(0, p, 0);
    for (int s = begin; s < end; ++s) {
        const int here = (s - begin) % STAGES, next = (s + 1 - begin) % STAGES;
        read(1, q, here);
        products(p);
        if (STAGES > 2 && s + STAGES <= end)
            wait_copies<(STAGES - 2) * COPIES>();
        else
            wait_copies<0>();
        meet();   // step s + 1 has come, and all of step s is in registers
        if (partial && s + 2 == end) {
            last(next);
            meet();
        }
        if constexpr (SPREAD) {
            const bool more = s + STAGES < end, whole = more && !(partial && s + STAGES + 1 == end);
            if (more && !whole) copy(s + STAGES, here);
            products(q, [&](int n) {   // behind the last step, reads of a buffer that nothing is made of
#pragma unroll
                for (int i = n * Set::LOADS / Set::PRODUCTS; i < (n + 1) * Set::LOADS / Set::PRODUCTS; ++i) read(0, p, next, i);
#pragma unroll
                for (int i = n * COPIES / Set::PRODUCTS; i < (n + 1) * COPIES / Set::PRODUCTS; ++i)
                    if (whole) copy(s + STAGES, here, i);
            });
        } else {
            if (s + STAGES < end) copy(s + STAGES, here);
            if (s + 1 < end) read(0, p, next);
            products(q);
        }
    }
}

template <typename T>
__device__ __forceinline__ float add_terms(const Eight<T>& v) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
        float x[kVec<T>];
        unpack(Raw<T>{v.u[k]}, x);
#pragma unroll
        for (int i = 0; i < kVec<T>; i += 4) s += (x[i] + x[i + 1]) + (x[i + 2] + x[i + 3]);
    }
    return s;
}

// WM x WN waves of MB x NB blocks each; three workgroups a unit of the tiles of 64 x 128, as many as shared memory holds.
template <typename T, bool BACK, int WM, int WN, int MB, int NB, int STAGES, bool SPREAD>
__global__ void __launch_bounds__(64 * WM * WN, WM * WN * MB * NB == 8 ? 3 : 2) k_product_rows(Args a) {
    constexpr int WAVES = WM * WN, BM = 32 * WM * MB, BN = 32 * WN * NB, TERMS = kStepBytes / (int)sizeof(T);
    using X = Along<T, BM, WAVES>;
    using W = typename std::conditional<BACK, Across<T, BN, WAVES>, Along<T, BN, WAVES>>::type;
    constexpr int STAGE = X::kBytes + W::kBytes, COPIES = X::kCopies + W::kCopies;
    constexpr int STORE = WAVES * kStoreBytes<T, NB>, LDS = STAGES * STAGE > STORE ? STAGES * STAGE : STORE;
    static_assert(LDS <= 160 * 1024, "shared memory");
    using Set = Half<T, NB, MB, sizeof(T) == 2>;
    __shared__ __align__(16) char lds[LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int terms = BACK ? a.N : a.K, columns = BACK ? a.K : a.N, tiles = (columns + BN - 1) / BN;
    // workgroups next to each other: 8 tiles of rows, then the next columns of those
    const int id = spread(blockIdx.x, gridDim.x), group = id / (8 * tiles), in = id % (8 * tiles);
    const int high = min(8, (int)a.slots - 8 * group), col0 = in / high * BN;
    const Rows r = find_rows<BM>(a.cu, a.E, a.R, (int)a.first + 8 * group + in % high, lane);
    if (r.count == 0) return;
    const bool none = r.expert < 0;
    const size_t expert = none ? 0 : r.expert;
    const int col = col0 + 32 * NB * wn;
    Sum<T, f32x16> acc[MB][NB];
    if (!BACK && !none && a.b) {   // the sums start from the bias
        const T* bias = static_cast<const T*>(a.b) + expert * a.N;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
                load_four(bias, min(col + 32 * nb + 8 * g + 4 * (lane >> 5), columns - 4), v);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[mb][nb].v[4 * g + i] = v[i];
            }
    }
    if (!none) {
        constexpr int SZ = (int)sizeof(T);
        const uint32_t xrow = (uint32_t)a.x_stride * SZ, wrow = (uint32_t)a.K * SZ;
        const char* x = static_cast<const char*>(a.x) + (long long)r.start * a.x_stride * SZ;
        const char* w = static_cast<const char*>(a.w) + expert * a.N * a.K * SZ +
                        (BACK ? (size_t)col0 * SZ : (size_t)col0 * a.K * SZ);
        const int here = min(columns - col0, BN);
        X xt;
        W wt;
        xt.place(xrow, r.count - 1, wave, lane);
        if constexpr (BACK)
            wt.place(wrow, here / kVec<T> - 1, wave, lane);
        else
            wt.place(wrow, here - 1, wave, lane);
        const uint32_t lds0 = lds_address(lds);
        const int steps = (terms + TERMS - 1) / TERMS;
        const int xpart = X::lane_part(lane), wpart = W::lane_part(lane);
        run_steps<Set, STAGES, COPIES, SPREAD>(
            0, steps, terms % TERMS != 0,
            [&](int s, int buffer, int one = -1) {
                const uint32_t at = lds0 + (uint32_t)buffer * STAGE;
                const int left = terms - s * TERMS;
                const char* xs = x + (size_t)s * kStepBytes;
                const char* ws = w + (BACK ? (size_t)s * TERMS * wrow : (size_t)s * kStepBytes);
                if (one >= X::kCopies) {
                    wt.copy_one(one - X::kCopies, at + X::kBytes, ws, wave);
                } else if (one >= 0) {
                    xt.copy_one(one, at, xs, wave);
                } else {
                    xt.copy(at, xs, left / kVec<T>, wave, lane);
                    if constexpr (BACK)
                        wt.copy(at + X::kBytes, ws, wrow, left - 1, wave, lane);
                    else
                        wt.copy(at + X::kBytes, ws, left / kVec<T>, wave, lane);
                }
            },
            [&](int half, Set& set, int buffer, int one = -1) {
                const char* at = lds + buffer * STAGE;
                if (one >= 0)
                    set.template read_one<W, X>(one, at + X::kBytes, at, wpart, xpart, 32 * NB * wn, 32 * MB * wm, lane, half);
                else
                    set.template read<W, X>(at + X::kBytes, at, wpart, xpart, 32 * NB * wn, 32 * MB * wm, lane, half);
            },
            [&](int buffer) {
                char* at = lds + buffer * STAGE;
                X::clear(at, terms % TERMS / kVec<T>);
                W::clear(at + X::kBytes, BACK ? terms % TERMS : terms % TERMS / kVec<T>);
            },
            [&](const Set& set, const auto&... between) { set.products(acc, between...); });
        meet();   // no tile is read any more
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int row = 32 * (MB * wm + mb);
        if (row >= r.count || col >= columns) break;
        store_block<T, NB>(lds + wave * kStoreBytes<T, NB>, static_cast<T*>(a.y) + (long long)(r.start + row) * columns + col,
                           columns, r.count - row, columns - col, lane, acc[mb]);
    }
}

// Forward, of few rows: 16 of them by 16 columns, whose terms WAVES waves share.  Nothing is read twice in a tile, so the
// operands come straight into registers, AHEAD reads of 32 terms on their way while those before are multiplied; the waves'
// sums are added in their order.  A lane has row (column) lane % 16 and terms 8 (lane / 16) .. of a read.
template <typename T, int WAVES, bool BY_ROW>
__global__ void __launch_bounds__(64 * WAVES) k_product_few(Args a) {
    constexpr int AHEAD = 16 / (int)sizeof(T), SIDE = 16, READ = 32;
    __shared__ __align__(16) f32x4 sums[WAVES][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = 8 * (lane / SIDE);
    const int tiles = (a.N + SIDE - 1) / SIDE, col0 = (int)(blockIdx.x % tiles) * SIDE;
    const Rows r = find_rows<SIDE, BY_ROW>(a.cu, a.E, a.R, (int)(blockIdx.x / tiles), lane);
    if (r.count == 0) return;
    Sum<T, f32x4> acc;
    if (r.expert >= 0) {
        const T* x = static_cast<const T*>(a.x) + (r.start + min(lane % SIDE, r.count - 1)) * a.x_stride;
        const T* w = static_cast<const T*>(a.w) + ((size_t)r.expert * a.N + min(col0 + lane % SIDE, a.N - 1)) * a.K;
        const int reads = (a.K + READ - 1) / READ, begin = reads * wave / WAVES, end = reads * (wave + 1) / WAVES;
        Eight<T> xn[AHEAD], wn[AHEAD];
        auto fetch = [&](int s0) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int at = min(READ * (s0 + k) + part, a.K - 8);   // past the end: the last terms that are there
#pragma unroll
                for (int u = 0; u < (int)sizeof(T) / 2; ++u) {
                    wn[k].u[u] = *reinterpret_cast<const u32x4*>(w + at + u * kVec<T>);
                    xn[k].u[u] = *reinterpret_cast<const u32x4*>(x + at + u * kVec<T>);
                }
            }
        };
        if (begin < end) fetch(begin);
        for (int s0 = begin; s0 < end; s0 += AHEAD) {
            Eight<T> xs[AHEAD], ws[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const bool there = s0 + k < end && READ * (s0 + k) + part < a.K;
#pragma unroll
                for (int u = 0; u < (int)sizeof(T) / 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ws[k].u[u][i] = there ? wn[k].u[u][i] : 0u;
                        xs[k].u[u][i] = there ? xn[k].u[u][i] : 0u;
                    }
            }
            if (s0 + AHEAD < end) fetch(s0 + AHEAD);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) mma(frag(ws[k]), frag(xs[k]), acc);
        }
        sums[wave][lane] = acc.all();
    }
    __syncthreads();
    const int row = lane % SIDE, col = col0 + part / 2;
    if (wave > 0 || row >= r.count || col >= a.N) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (r.expert >= 0) {
        if (a.b) {
            float b[4];
            load_four(static_cast<const T*>(a.b) + (size_t)r.expert * a.N, col, b);
            v = f32x4{b[0], b[1], b[2], b[3]};
        }
#pragma unroll
        for (int k = 0; k < WAVES; ++k) v += sums[k][lane];
    }
    T* to = static_cast<T*>(a.y) + (long long)(r.start + row) * a.N + col;
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<u32x2*>(to) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
    else
        *reinterpret_cast<f32x4*>(to) = v;
}

template <typename T, int WM, int WN, int MB, int NB, int STAGES, bool SPREAD>
__global__ void __launch_bounds__(64 * WM * WN, 2) k_product_weights(Args a) {
    constexpr int WAVES = WM * WN, BM = 32 * WM * MB, BN = 32 * WN * NB, TERMS = kStepBytes / (int)sizeof(T);
    using G = Across<T, BM, WAVES>;
    using X = Across<T, BN, WAVES>;
    constexpr int STAGE = G::kBytes + X::kBytes, COPIES = G::kCopies + X::kCopies;
    constexpr int STORE = WAVES * kStoreBytes<float, NB>, LDS = STAGES * STAGE > STORE ? STAGES * STAGE : STORE;
    static_assert(LDS <= 160 * 1024, "shared memory");
    using Set = Half<T, NB, MB, sizeof(T) == 2>;
    __shared__ __align__(16) char lds[LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int ktiles = (a.K + BN - 1) / BN, ntiles = (a.N + BM - 1) / BM;
    // the longest parts first; the tiles of one are spread over the XCDs by runs
    const int per = ktiles * ntiles, id = spread(blockIdx.x % per, per);
    // no places: no expert has several parts, and few rows
    Part part = {(int)(blockIdx.x / per), 0, 1, 0};
    if (a.slots > 0) part = find_part(a.cu, a.E, a.R, a.rows, blockIdx.x / per, lane);
    if (part.expert < 0) return;
    if (no_place(a, part.place, part.parts)) {
        if (part.part > 0) return;
        part.parts = 1;
    }
    const int e = part.expert, col0 = id % ktiles * BN, row0 = id / ktiles * BM;
    const int first = segment_begin(a.cu, a.E, a.R, e + 1), count = max(segment_begin(a.cu, a.E, a.R, e + 2) - first, 0);
    const int all = (count + TERMS - 1) / TERMS;
    const int begin = (int)((long long)all * part.part / part.parts), end = (int)((long long)all * (part.part + 1) / part.parts);
    Sum<T, f32x16> acc[MB][NB];
    float sum[MB] = {};   // of dy's columns: the lane's half of the terms
    const bool sums = a.db && col0 == 0 && wn == 0;
    constexpr int SZ = (int)sizeof(T);
    const uint32_t grow = (uint32_t)a.g_stride * SZ, xrow = (uint32_t)a.x_stride * SZ;
    const char* g = static_cast<const char*>(a.g) + ((long long)first * a.g_stride + row0) * SZ;
    const char* x = static_cast<const char*>(a.x) + ((long long)first * a.x_stride + col0) * SZ;
    G gt;
    X xt;
    gt.place(grow, min(a.N - row0, BM) / kVec<T> - 1, wave, lane);
    xt.place(xrow, min(a.K - col0, BN) / kVec<T> - 1, wave, lane);
    const uint32_t lds0 = lds_address(lds);
    const int gpart = G::lane_part(lane), xpart = X::lane_part(lane);
    run_steps<Set, STAGES, COPIES, SPREAD>(
        begin, end, end == all && count % TERMS != 0,
        [&](int s, int buffer, int one = -1) {
            const uint32_t at = lds0 + (uint32_t)buffer * STAGE;
            const int last = count - 1 - s * TERMS;
            const char *gs = g + (size_t)s * TERMS * grow, *xs = x + (size_t)s * TERMS * xrow;
            if (one >= G::kCopies) {
                xt.copy_one(one - G::kCopies, at + G::kBytes, xs, wave);
            } else if (one >= 0) {
                gt.copy_one(one, at, gs, wave);
            } else {
                gt.copy(at, gs, grow, last, wave, lane);
                xt.copy(at + G::kBytes, xs, xrow, last, wave, lane);
            }
        },
        [&](int half, Set& set, int buffer, int one = -1) {
            const char* at = lds + buffer * STAGE;
            if (one >= 0)
                set.template read_one<X, G>(one, at + G::kBytes, at, xpart, gpart, 32 * NB * wn, 32 * MB * wm, lane, half);
            else
                set.template read<X, G>(at + G::kBytes, at, xpart, gpart, 32 * NB * wn, 32 * MB * wm, lane, half);
        },
        [&](int buffer) {
            char* at = lds + buffer * STAGE;
            G::clear(at, count % TERMS);
            X::clear(at + G::kBytes, count % TERMS);
        },
        [&](const Set& set, const auto&... between) {
            set.products(acc, between...);
            if (sums) {
#pragma unroll
                for (int k = 0; k < Set::READS; ++k)
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) sum[mb] += add_terms<T>(set.b[k][mb]);
            }
        });
    meet();
    const int col = col0 + 32 * NB * wn;
    const size_t weights = (size_t)a.N * a.K, place = part.place + part.part;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int row = row0 + 32 * (MB * wm + mb);
        if (row >= a.N) break;
        if (sums) {
            const float both = sum[mb] + __shfl_xor(sum[mb], 32);
            if (lane < 32 && row + lane < a.N) {
                if (part.parts == 1)
                    static_cast<T*>(a.db)[(size_t)e * a.N + row + lane] = from_f32<T>(both);
                else
                    a.parts[a.slots * weights + place * a.N + row + lane] = both;
            }
        }
        if (col >= a.K) continue;
        const size_t to = (size_t)row * a.K + col;
        if (part.parts == 1)
            store_block<T, NB>(lds + wave * kStoreBytes<T, NB>, static_cast<T*>(a.y) + e * weights + to, a.K, a.N - row,
                               a.K - col, lane, acc[mb]);
        else
            store_block<float, NB>(lds + wave * kStoreBytes<float, NB>, a.parts + place * weights + to, a.K, a.N - row,
                                   a.K - col, lane, acc[mb]);
    }
}

// The sums of the experts' parts in their order: N K weights of an expert, then N of db.  Every gridDim.y-th such
// expert is one row of workgroups'.
template <typename T>
__global__ void __launch_bounds__(256) k_product_join(Args a) {
    const int lane = threadIdx.x & 63;
    const long long n = (long long)a.N * a.K, m = a.db ? a.N : 0;
    int place = 0, p0 = 0;
    unsigned nth = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int mine = e0 + lane;
        const int count = mine < a.E ? segment_begin(a.cu, a.E, a.R, mine + 2) - segment_begin(a.cu, a.E, a.R, mine + 1) : 0;
        const int p = parts_of(max(count, 0), a.rows);
        for (uint64_t split = __builtin_amdgcn_ballot_w64(p > 1); split; split &= split - 1, place += p0) {
            const int at = __builtin_ctzll(split), parts = __builtin_amdgcn_readlane(p, at);
            p0 = parts;
            const long long e = e0 + at;
            if (nth++ % gridDim.y != blockIdx.y || no_place(a, place, parts)) continue;
            for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; 4 * u < n + m; u += (long long)gridDim.x * 256) {
                const bool bias = 4 * u >= n;   // n and m are multiples of 8
                const float* sums = a.parts + (bias ? a.slots * n + place * m + 4 * u - n : place * n + 4 * u);
                const long long far = bias ? m : n;
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
                for (int s = 0; s < parts; ++s) v += *reinterpret_cast<const f32x4*>(sums + s * far);
                T* to = bias ? static_cast<T*>(a.db) + e * m + (4 * u - n) : static_cast<T*>(a.y) + e * n + 4 * u;
                if constexpr (sizeof(T) == 2)
                    *reinterpret_cast<u32x2*>(to) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
                else
                    *reinterpret_cast<f32x4*>(to) = v;
            }
        }
    }
}

template <typename T, bool BACK, int WM, int WN, int MB, int NB, int STAGES, bool SPREAD = false>
int launch_rows(Args a, hipStream_t st) {
    constexpr int BM = 32 * WM * MB, BN = 32 * WN * NB;
    const long long all = row_slots(a.R, a.E, BM), tiles = ((BACK ? a.K : a.N) + BN - 1) / BN;
    const long long most = ((1 << 22) / tiles) & ~7LL;   // a launch has less than 2^32 threads
    for (; a.first < all; a.first += most) {
        a.slots = most < all - a.first ? most : all - a.first;
        hipLaunchKernelGGL((k_product_rows<T, BACK, WM, WN, MB, NB, STAGES, SPREAD>), dim3((unsigned)(a.slots * tiles)),
                           dim3(64 * WM * WN), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}
template <typename T>
int launch_few(const Args& a, long long slots, hipStream_t st) {
    constexpr int WAVES = 4;
    const dim3 grid((unsigned)(slots * ((a.N + 15) / 16)));
    if (slots == a.R)
        hipLaunchKernelGGL((k_product_few<T, WAVES, true>), grid, dim3(64 * WAVES), 0, st, a);
    else
        hipLaunchKernelGGL((k_product_few<T, WAVES, false>), grid, dim3(64 * WAVES), 0, st, a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

// The tile, by what the rounds of workgroups take.  Measured (us, 8 experts, bfloat16; rows x terms -> columns):
//   256 x 256 against 128 x 128 where the estimates are near each other: 12544 x 1024 -> 1024 29.0 and 33.6, 16384 49.4 and
// 44.4, 24000 52.4 and 61.1, 32768 77.2 and 74.9, 50176 106.6 and 107.2; 12544 x 512 -> 2048 33.6 and 35.7; 25088 x 2048 ->
// 512 49.3 and 59.0, 40000 91.6 and 87.5; far from there, 50176 x 1024 -> 4096 401 and 451, 4096 x 1024 -> 1024 25.4 and
// 18.4.  The worst found is 8192 x 1024 -> 1024: 29.6 taken, 26.5.
//   128 x 128 against 64 x 128 around 384 tiles: 216 of them 25.1 and 23.8, 320 17.5 and 18.1, 384 11.3 and 11.1, 424 31.4
// and 45.5; float32 200 84.6 and 80.3, 432 45.6 and 52.0.
//   64 x 128 against 32 x 128 around 256 tiles: 160 of them 20.5 and 16.9, 192 11.7 and 11.2, 320 14.0 and 17.8; float32
// 128 19.1 and 15.3, 160 37.4 and 38.5, 320 30.8 and 32.6.  Few tiles wait for their weights: four stages of the smallest
// 6.9 us for 98 rows x 512 -> 2048, two 8.9, eight 7.8.
//   Forward, tiles of 16 x 16 with the terms shared by four waves, against 32 x 128, by the number of those tiles.  bfloat16:
// 128 of them (one row x 512 -> 2048) 4.1 and 5.4, 448 (98 x 2048 -> 512) 9.8 and 14.1, 512 (8 x 8192 -> 1024) 22.5 and 47.5,
// 640 (196 x 2048 -> 512) 13.6 and 14.1, 1024 (392) 17.7 and 14.4; with few terms 64 (4 x 256 -> 256) 4.2 and 5.3, 160 (98)
// 4.7 and 4.1.  float32: 226 (2 x 88 -> 1808) 4.0 and 5.6, 256 (2 x 512 -> 2048) 4.6 and 14.7, 1017 (98 x 88 -> 1808) 7.4 and
// 5.9, 1056 (400 x 2048 -> 512) 33.8 and 52.3, 1792 (98 x 512 -> 2048) 14.4 and 16.3, 2240 (1000 x 2048 -> 512) 68 and 52.
template <typename T, bool BACK>
int run_rows_way(const Args& a, hipStream_t st) {
    const int columns = BACK ? a.K : a.N, steps = ((BACK ? a.N : a.K) + 63) / 64;
    auto tiles = [&](int rows, int cols) {   // about: an expert's last tile is half full in the mean
        const long long full = a.R / rows;
        return (full + (full < a.E ? full : a.E)) * ((columns + cols - 1) / cols);
    };
    if constexpr (!BACK) {
        const bool wide = sizeof(T) == 4;
        const long long slots = row_slots(a.R, a.E, 16), rows = slots < a.R ? slots : a.R, few = rows * ((columns + 15) / 16);
        if (few <= (a.K >= (wide ? 256 : 512) ? (wide ? 1536 : 640) : (wide ? 256 : 128))) return launch_few<T>(a, rows, st);
    }
    const long long middle = tiles(128, 128);
    if constexpr (sizeof(T) == 2) {
        // microseconds: a round of one large tile a unit takes 1.55 a step and 3.5 for its beginning and end, and the last
        // round is paid whole; 512 of the smaller, two a unit, take 1.06 and 1.2, and a quarter of that where they run out
        const double large = (double)((tiles(256, 256) + 255) / 256) * (1.55 * steps + 3.5);
        if (middle > 512 && large <= (middle / 512.0 + 0.25) * (1.06 * steps + 1.2)) return launch_rows<T, BACK, 2, 4, 4, 2, 2, true>(a, st);
    }
    if (middle >= 384) return launch_rows<T, BACK, 2, 2, 2, 2, 2>(a, st);
    if (tiles(64, 128) >= 256) return launch_rows<T, BACK, 2, 2, 1, 2, 2>(a, st);
    return launch_rows<T, BACK, 1, 4, 1, 1, 4>(a, st);
}
template <typename T>
int run_rows(const Args& a, bool back, hipStream_t st) {
    return back ? run_rows_way<T, true>(a, st) : run_rows_way<T, false>(a, st);
}
template <typename T, int WM, int WN, int MB, int NB, int STAGES, bool SPREAD = false>
int launch_weights(const Args& a, hipStream_t st) {
    constexpr int BM = 32 * WM * MB, BN = 32 * WN * NB;
    const long long groups = (long long)((a.K + BN - 1) / BN) * ((a.N + BM - 1) / BM) * (a.slots > 0 ? most_parts(a.R, a.E, a.rows) : a.E);
    if (groups > (1 << 23)) return WTC_ESHAPE;
    hipLaunchKernelGGL((k_product_weights<T, WM, WN, MB, NB, STAGES, SPREAD>), dim3((unsigned)groups), dim3(64 * WM * WN), 0, st,
                       a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}
template <typename T>
int run_weights(const Args& a, bool large, hipStream_t st) {
    int r;
    if constexpr (sizeof(T) == 2)
        r = large ? launch_weights<T, 2, 4, 4, 2, 2, true>(a, st) : launch_weights<T, 2, 2, 2, 2, 2>(a, st);
    else
        r = launch_weights<T, 2, 2, 2, 2, 2>(a, st);
    if (r == WTC_OK && a.slots > 0) {
        const long long blocks = (((long long)a.K + 1) * a.N / 4 + 255) / 256;
        hipLaunchKernelGGL(k_product_join<T>, dim3((unsigned)(blocks < 512 ? blocks : 512), a.E < 4 ? a.E : 4), dim3(256), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? r : WTC_EHIP;
}

}  // namespace product
}  // namespace wtc
