// Attention, backward.  With P = exp(scale Q K^T - lse), delta = rowsum(dO O):
//   dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
//
// Two kernels, each with its results in registers for its whole run, instead
// of one that would have to add dQ into memory from many workgroups in an
// order that changes: dQ by query tiles (3 products a tile: S^T, dP^T, dQ^T),
// dK and dV by key tiles, over the q heads of their group (4 products: S, dP,
// dV^T, dK^T).  P is recomputed in both from the stored lse.  With few tiles
// both are split as the forward pass is, and their partial sums joined.
//
// Bound by the matrix units with the exponentials and roundings between their
// products.  Means of 20 training steps (the fastest up to 18 % less),
// bfloat16, dq and dk/dv: 48 images of 49 to 1024 tokens, 6 heads of 64, 83 and
// 103 us (595 and 635 TFLOP/s of the products each makes); 4 x 4096, 12 heads of
// 64, 320 and 441 us (965, 935); causal 3 x 3500..8192, 16 heads on 4 of 128, 501
// and 717 us (1035, 965) with 26 us of joins; float32 32 x 196, 6 heads on 3 of
// 64, 36 and 44 us (79, 85) with 7 us of joins.
#pragma once

#include "wtc_tok_attn.h"

namespace wtc {
namespace attn {

constexpr int kDqRows = 128;   // queries of a workgroup, 32 a wave
template <typename T>
constexpr int kDqKeys = sizeof(T) == 2 ? 64 : 32;   // keys of a tile
constexpr int kDkvKeys = 128;  // keys of a workgroup, 32 a wave
// Queries of a tile, and whether the wave's 32 rows of V wait in shared memory
// instead of registers.  128 channels of bfloat16 need 64 registers for K and V
// beside 128 for the sums and 32 for S and dP, more than the 256 that leave two
// waves on a vector unit; with V (32 KB) and tiles of 32 queries (33 KB) shared
// memory holds two workgroups as well.
template <typename T, int DP>
constexpr bool kDkvHoldV = sizeof(T) == 2 && DP == 128;
template <typename T, int DP>
constexpr int kDkvRows = sizeof(T) == 2 && !kDkvHoldV<T, DP> ? 64 : 32;

template <typename T, int DP>
__global__ void __launch_bounds__(256, occupancy(kDq, sizeof(T), DP)) k_attn_dq(Args a) {
    constexpr int KEYS = kDqKeys<T>, KB = KEYS / 32, KS = DP / 16, DB = DP / 32;
    using L = Tile<T, DP, KEYS>;
    constexpr int TILE = L::kBytes, LDS = max_of(4 * TILE, 4 * kRowsScratch<float, DP>);
    __shared__ __align__(16) char lds[LDS];   // 2 x (K tile, V tile); then a place to store from
    static_assert(LDS <= 160 * 1024, "shared memory");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % a.Hq, split = blockIdx.x / a.Hq % a.q_splits;
    const Work w = find_work<kDqRows, true>(a, blockIdx.x / a.Hq / a.q_splits, lane);
    if (w.none) return;
    const int row0 = w.tile * kDqRows + wave * 32, row = row0 + (lane & 31);
    const int rows_left = w.len - row0;
    const bool live = row < w.len;
    f32x16 acc[DB] = {};
    auto store = [&] {   // no tile is read any more
        if (rows_left <= 0) return;
        const long long t = w.start + row0;
        if (a.q_splits == 1) {
            store_rows<T, DP>(lds + wave * kRowsScratch<T, DP>, static_cast<T*>(a.dq) + t * a.sdq.token + head * a.sdq.head,
                              a.sdq.token, rows_left, a.D, lane, acc, a.scale);
        } else {
            const long long step = (long long)a.Hq * a.D, n = a.T * step;
            store_rows<float, DP>(lds + wave * kRowsScratch<float, DP>, a.parts + split * n + t * step + head * a.D, step,
                                  rows_left, a.D, lane, acc, a.scale);
        }
    };
    const long long stat = (long long)head * a.T + w.start + min(row, w.len - 1);
    if (w.pad) {
        store();
        return;
    }
    const int kvh = head / a.group, chunks = a.D / 8;
    const char* kbase = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + (long long)w.start * a.sk.token + kvh * a.sk.head);
    const char* vbase = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + (long long)w.start * a.sv.token + kvh * a.sv.head);
    const uint32_t krow = (uint32_t)a.sk.token * sizeof(T), vrow = (uint32_t)a.sv.token * sizeof(T);
    const int keys = a.causal ? min(w.len, (w.tile + 1) * kDqRows) : w.len;
    const int tiles = (keys + KEYS - 1) / KEYS;
    const int begin = (int)((long long)tiles * split / a.q_splits), end = (int)((long long)tiles * (split + 1) / a.q_splits);
    const uint32_t lds0 = lds_address(lds);
    typename L::Load kload, vload;
    auto copy = [&](int j) {
        const int j0 = j * KEYS, there = min(w.len - 1 - j0, KEYS - 1);
        const uint32_t at = lds0 + (uint32_t)(j & 1) * (2 * TILE);
        L::issue(kload, at, kbase + (long long)j0 * krow, krow, there, chunks, wave, lane);
        L::issue(vload, at + TILE, vbase + (long long)j0 * vrow, vrow, there, chunks, wave, lane);
    };
    if (begin < end) copy(begin);

    const float c = a.scale * kLog2e;
    Frag<T> q[KS], g[KS];
    float delta = 0.f;
    const float lse = a.lse[stat];
    {
        const long long t = w.start + min(row, w.len - 1);
        const T* qrow = static_cast<const T*>(a.q) + t * a.sq.token + head * a.sq.head;
        const T* grow = static_cast<const T*>(a.g) + t * a.sg.token + head * a.sg.head;
        const T* orow = static_cast<const T*>(a.o) + t * a.so.token + head * a.so.head;
        row_terms(qrow, a.D, lane, 1.f, q);
        row_terms(grow, a.D, lane, 1.f, g);
        delta = half_dot<T, KS>(grow, orow, a.D, lane);
        // with the bits that were rounded off out: 8 of them alone move dS by as much as its own rounding
        if (sizeof(T) == 2 && a.low)
            delta += half_dot<T, KS>(grow, static_cast<const T*>(a.low) + (t * a.Hq + head) * a.D, a.D, lane);
        delta = both_sum(delta);
        if (split == 0 && live && lane < 32) a.delta[stat] = delta;   // for the other kernel
    }
    const float lse2 = lse * kLog2e;
    const int rlane = L::rows_lane(lane), clane = L::cols_lane(lane), half = L::row_of_half(lane), swap = L::cols_swap(lane);
    const int last = a.causal ? min(w.len - 1, row0 + 31) : w.len - 1;   // last key that any of the wave's queries sees
    f32x16 minus;   // dP starts from -delta
#pragma unroll
    for (int r = 0; r < 16; ++r) minus[r] = -delta;
    for (int j = begin; j < end; ++j) {
        L::commit(kload, lds + (j & 1) * (2 * TILE), wave, lane);
        L::commit(vload, lds + (j & 1) * (2 * TILE) + TILE, wave, lane);
        __syncthreads();   // tile j is there; everyone is done with the other one
        if (j + 1 < end) copy(j + 1);
        const int j0 = j * KEYS;
        if (rows_left <= 0 || (a.causal && j0 > row0 + 31)) continue;
        const char* kt = lds + (j & 1) * (2 * TILE) + rlane;
        const char* kc = lds + (j & 1) * (2 * TILE) + clane;
        const int seen = (a.causal ? min(w.len - 1, row) : w.len - 1) - j0 - half;
        const bool edge = j0 + KEYS - 1 > (a.causal ? min(w.len - 1, row0) : w.len - 1);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if (kb > 0 && j0 + 32 * kb > last) break;   // no pair in this block
            f32x16 s = {}, dp = minus;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                mma(L::rows(kt, 32 * kb, ks), q[ks], s);
                mma(L::rows(kt + TILE, 32 * kb, ks), g[ks], dp);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2));
                s[r] = p * dp[r];
            }
            if (edge) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * kb + L::row_of(r) > seen) s[r] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Frag<T> ds;
                as_terms(s, t, ds);
#pragma unroll
                for (int db = 0; db < DB; ++db) mma(L::cols(kc, swap, 32 * kb, t, db), ds, acc[db]);
            }
        }
    }
    __syncthreads();   // everyone is done with the tiles
    store();
}

template <typename T, int DP>
__global__ void __launch_bounds__(256, occupancy(kDkv, sizeof(T), DP)) k_attn_dkv(Args a) {
    constexpr int ROWS = kDkvRows<T, DP>, KS = DP / 16, DB = DP / 32;
    using L = Tile<T, DP, ROWS>;
    constexpr int TILE = L::kBytes;
    constexpr bool HOLD = kDkvHoldV<T, DP>;
    // 128 channels of float32: 96 registers each for K's and V's terms are 42 more than there are.  Kept as
    // they were loaded they take 64, and the split runs beside the products (4 causal sequences of 500 to 1024,
    // 8 heads: 117 -> 111 us; at 96 channels, which have the registers, 594 -> 640 us for 4 x 2048).
    constexpr bool RAW = sizeof(T) == 4 && DP > 96;
    constexpr int LDS = max_of(4 * TILE + (HOLD ? 4 * KS * 64 * (int)sizeof(Frag<T>) : 0), 4 * kRowsScratch<float, DP>);
    __shared__ __align__(16) char lds[LDS];   // 2 x (Q tile, dO tile), then V of the four waves
    __shared__ __align__(16) float stats[2][2][ROWS];   // 2 x -lse log2(e), over c where S starts from it, and -delta of the tile's queries
    // S starts from -lse log2(e) / c and dP from -delta, which saves their subtraction.  S is then rounded at
    // lse's size: P is off by |lse| log2(e) 2^-24, less than its rounding to bfloat16 (2^-8) up to |lse| = 2^15.
    // Not so in float32 (dk and dv 2.5 times the error)
    constexpr bool START = sizeof(T) == 2;
    static_assert(LDS + 4 * ROWS * 4 <= 160 * 1024, "shared memory");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = blockIdx.x % a.Hk, split = blockIdx.x / a.Hk % a.k_splits;
    const Work w = find_work<kDkvKeys, false>(a, blockIdx.x / a.Hk / a.k_splits, lane);
    if (w.none) return;
    const int key0 = w.tile * kDkvKeys + wave * 32, key = key0 + (lane & 31);
    const int keys_left = w.len - key0;
    const bool live = key < w.len;
    f32x16 ak[DB] = {}, av[DB] = {};
    auto store = [&] {   // no tile is read any more
        if (keys_left <= 0) return;
        const long long t = w.start + key0;
        if (a.k_splits == 1) {
            char* scratch = lds + wave * kRowsScratch<T, DP>;
            store_rows<T, DP>(scratch, static_cast<T*>(a.dk) + t * a.sdk.token + kvh * a.sdk.head, a.sdk.token, keys_left, a.D,
                              lane, ak, a.scale);
            store_rows<T, DP>(scratch, static_cast<T*>(a.dv) + t * a.sdv.token + kvh * a.sdv.head, a.sdv.token, keys_left, a.D,
                              lane, av, 1.f);
        } else {
            const long long n = (long long)a.T * a.Hk * a.D, row = (long long)a.Hk * a.D;
            float* dk = a.parts + 2 * split * n + t * row + kvh * a.D;
            char* scratch = lds + wave * kRowsScratch<float, DP>;
            store_rows<float, DP>(scratch, dk, row, keys_left, a.D, lane, ak, a.scale);
            store_rows<float, DP>(scratch, dk + n, row, keys_left, a.D, lane, av, 1.f);
        }
    };
    static_assert(4 * kRowsScratch<float, DP> <= LDS, "the tiles' place serves for storing");
    if (w.pad) {
        store();
        return;
    }
    const int chunks = a.D / 8;
    const uint32_t qrow = (uint32_t)a.sq.token * sizeof(T), grow = (uint32_t)a.sg.token * sizeof(T);
    const int first = a.causal ? w.tile * kDkvKeys / ROWS : 0;   // the first query tile that sees these keys
    const int per_head = (w.len + ROWS - 1) / ROWS - first, all = per_head * a.group;
    const int begin = (int)((long long)all * split / a.k_splits), end = (int)((long long)all * (split + 1) / a.k_splits);
    if (begin == end) {
        store();
        return;
    }
    const uint32_t lds0 = lds_address(lds);
    // no scale below 2^-100 (a zero one): what it multiplies is then lost beside lse, as it should be
    const float c = copysignf(fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f), a.scale), inv_c = 1.f / c;
    // lse (the first ROWS threads) or delta (the next) of a query of the tile copied last, on its way to
    // shared memory, in the order that a result's registers have the rows in.  It is left as it was loaded
    // until the tile itself is waited for.
    float stat = 0.f;
    int stat_last = 0;
    const bool is_lse = threadIdx.x < ROWS;
    const int stat_row = threadIdx.x % ROWS / 32 * 32 + L::place(threadIdx.x % 32);
    typename L::Load qload, gload;
    int head = kvh * a.group + begin / per_head, j0 = (first + begin % per_head) * ROWS;   // of the next tile to copy
    auto copy = [&](int i) {
        const int last = min(w.len - 1 - j0, ROWS - 1);
        const uint32_t at = lds0 + (uint32_t)(i & 1) * (2 * TILE);
        const T* qp = static_cast<const T*>(a.q) + (long long)(w.start + j0) * a.sq.token + head * a.sq.head;
        const T* gp = static_cast<const T*>(a.g) + (long long)(w.start + j0) * a.sg.token + head * a.sg.head;
        L::issue(qload, at, reinterpret_cast<const char*>(qp), qrow, last, chunks, wave, lane);
        L::issue(gload, at + TILE, reinterpret_cast<const char*>(gp), grow, last, chunks, wave, lane);
        if (threadIdx.x < 2 * ROWS) {
            const long long t = (long long)head * a.T + w.start + j0 + min(stat_row, last);
            stat = (is_lse ? a.lse : a.delta)[t];
            stat_last = last;
        }
        j0 += ROWS;
        if (j0 >= w.len) {
            j0 = first * ROWS;
            ++head;
        }
    };
    int here = j0;   // first query of the tile being worked on
    copy(begin);

    Frag<T> kf[KS], vf[KS];   // with HOLD, V waits in shared memory
    Eight<T> kr[KS], vr[KS];   // with RAW, both are held as they were loaded
    Frag<T>* mine = reinterpret_cast<Frag<T>*>(lds + 4 * TILE) + wave * KS * 64 + lane;   // its place there
    {
        const long long t = w.start + min(key, w.len - 1);
        const T* krow = static_cast<const T*>(a.k) + t * a.sk.token + kvh * a.sk.head;
        const T* vrow = static_cast<const T*>(a.v) + t * a.sv.token + kvh * a.sv.head;
        if constexpr (RAW) {
            load_row(krow, a.D, lane, 1.f, kr);
            load_row(vrow, a.D, lane, 1.f, vr);
        } else {
            row_terms(krow, a.D, lane, 1.f, kf);
            row_terms(vrow, a.D, lane, 1.f, vf);
        }
        if constexpr (HOLD) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mine[64 * ks] = vf[ks];   // read by this lane alone: no barrier
        }
    }
    const int rlane = L::rows_lane(lane), clane = L::cols_lane(lane), swap = L::cols_swap(lane);
    for (int i = begin; i < end; ++i) {
        if (threadIdx.x < 2 * ROWS) {
            // queries past the end: an infinite lse leaves nothing of them
            const float lse = stat_row <= stat_last ? stat * kLog2e : __builtin_inff();
            stats[i & 1][threadIdx.x / ROWS][threadIdx.x % ROWS] = is_lse ? lse * (START ? -inv_c : -1.f) : -stat;
        }
        L::commit(qload, lds + (i & 1) * (2 * TILE), wave, lane);
        L::commit(gload, lds + (i & 1) * (2 * TILE) + TILE, wave, lane);
        __syncthreads();   // tile i is there; everyone is done with the other one
        const int at = here;
        here = j0;
        if (i + 1 < end) copy(i + 1);
        if (keys_left <= 0 || (a.causal && at + ROWS - 1 < key0)) continue;
        const char* qt = lds + (i & 1) * (2 * TILE) + rlane;
        const char* qc = lds + (i & 1) * (2 * TILE) + clane;
        const bool edge = a.causal && at < key0 + 31;   // some of the tile's queries come before some of the keys
#pragma unroll 1
        for (int qb = 0; qb < ROWS / 32; ++qb, qt += L::row_at(32), qc += L::row_at(32)) {
            f32x16 s, dp;
            const float* st = &stats[i & 1][0][32 * qb + 4 * (lane >> 5)];
            if constexpr (START) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = st[8 * (r >> 2) + (r & 3)];
            } else {
                s = f32x16{};
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(L::rows(qt, 0, ks), RAW ? terms_anew<T>(kr[ks]) : kf[ks], s);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 16; ++r) dp[r] = st[ROWS + 8 * (r >> 2) + (r & 3)];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) mma(L::rows(qt + TILE, 0, ks), HOLD ? mine[64 * ks] : RAW ? terms_anew<T>(vr[ks]) : vf[ks], dp);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = __builtin_amdgcn_exp2f(START ? s[r] * c : fmaf(s[r], c, st[8 * (r >> 2) + (r & 3)]));
                dp[r] *= s[r];
            }
            if (edge) {
                const int l = anew(lane), seen = key0 + (l & 31) - at - 32 * qb - L::row_of_half(l);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (L::row_of(r) < seen) s[r] = dp[r] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Frag<T> p, ds;
                as_terms(s, t, p);
                as_terms(dp, t, ds);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    mma(L::cols(qc + TILE, swap, 0, t, db), p, av[db]);
                    mma(L::cols(qc, swap, 0, t, db), ds, ak[db]);
                }
            }
        }
    }
    __syncthreads();   // everyone is done with the tiles
    store();
}

// Gradients from the splits' sums, in their order: `arrays` of them [T, heads,
// D], a split's one after another.  Eight channels a thread.
struct Join {
    const float* parts;
    int splits, arrays, heads, D;
    long long n;   // T heads D
    void* to[2];
    wtc_attn_strides st[2];
};
template <typename T>
__global__ void __launch_bounds__(256) k_attn_join(Join a) {
    const long long step = (long long)gridDim.x * 256 * 8;
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < a.arrays * a.n; i += step) {
        const int which = i >= a.n;
        const long long at = i - which * a.n, row = at / a.D;
        const int c = (int)(at - row * a.D), head = (int)(row % a.heads);
        float sum[8] = {};
        for (int s = 0; s < a.splits; ++s) {
            float x[4], y[4];
            load16(a.parts + s * a.arrays * a.n + i, x);
            load16(a.parts + s * a.arrays * a.n + i + 4, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[j] += x[j];
                sum[4 + j] += y[j];
            }
        }
        T* out = static_cast<T*>(a.to[which]) + row / a.heads * a.st[which].token + head * a.st[which].head + c;
#pragma unroll
        for (int k = 0; k < 8; k += kVec<T>) {
            float v[kVec<T>];
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) v[j] = sum[k + j];
            store16(out + k, v);
        }
    }
}
template <typename T>
void run_join(const Join& j, hipStream_t st) {
    hipLaunchKernelGGL((k_attn_join<T>), dim3(join_groups(j.arrays * j.n / 8)), dim3(256), 0, st, j);
}

template <typename T, int DP>
int run_bwd(const Args& a, hipStream_t st) {
    const long long gq = slots(a.T, a.n_seq, kDqRows) * a.Hq * a.q_splits;
    const long long gk = slots(a.T, a.n_seq, kDkvKeys) * a.Hk * a.k_splits;
    if (gq >= kMaxGroups || gk >= kMaxGroups) return WTC_ESHAPE;
    hipLaunchKernelGGL((k_attn_dq<T, DP>), dim3((unsigned)gq), dim3(256), 0, st, a);
    if (a.q_splits > 1) run_join<T>({a.parts, a.q_splits, 1, a.Hq, a.D, (long long)a.T * a.Hq * a.D, {a.dq, nullptr}, {a.sdq, {}}}, st);
    hipLaunchKernelGGL((k_attn_dkv<T, DP>), dim3((unsigned)gk), dim3(256), 0, st, a);
    if (a.k_splits > 1) run_join<T>({a.parts, a.k_splits, 2, a.Hk, a.D, (long long)a.T * a.Hk * a.D, {a.dk, a.dv}, {a.sdk, a.sdv}}, st);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace attn
}  // namespace wtc
