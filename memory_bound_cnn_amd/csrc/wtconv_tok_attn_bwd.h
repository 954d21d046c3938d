// Attention, backward.  With P = exp(scale Q K^T - lse), delta = rowsum(dO O):
//   dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
//
// Two kernels, each with its results in registers for its whole run, instead
// of one that would have to add dQ into memory from many workgroups in an
// order that changes: dQ by query tiles (3 products a tile: S^T, dP^T, dQ^T),
// dK and dV by key tiles, over the q heads of their group (4 products: S, dP,
// dV^T, dK^T).  P is recomputed in both from the stored lse.
#pragma once

#include "wtc_tok_attn.h"

namespace wtc {
namespace attn {

constexpr int kDqRows = 128;   // queries of a workgroup, 32 a wave
constexpr int kDqKeys = 64;    // keys of a tile
constexpr int kDkvKeys = 128;  // keys of a workgroup, 32 a wave
template <typename T>
constexpr int kDkvRows = sizeof(T) == 2 ? 64 : 32;   // queries of a tile

template <typename T, int DP>
__global__ void __launch_bounds__(256, occupancy(kDq, sizeof(T), DP)) k_attn_dq(Args a) {
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32, TILE = L::bytes(kDqKeys);
    __shared__ __align__(16) char lds[4 * TILE];   // 2 x (K tile, V tile)
    static_assert(4 * TILE <= 160 * 1024, "shared memory");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n_slots = gridDim.x / a.Hq, head = blockIdx.x % a.Hq;
    const int slot = n_slots - 1 - blockIdx.x / a.Hq;   // late tiles have the most keys when causal: they go first
    const Work w = find_work<kDqRows>(a, slot, lane);
    if (w.none) return;
    const int row0 = w.tile * kDqRows + wave * 32, row = row0 + (lane & 31);
    const int rows_left = w.len - row0;
    const bool live = row < w.len;
    T* dq = static_cast<T*>(a.dq) + (long long)(w.start + row) * a.sdq.token + head * a.sdq.head;
    const long long stat = (long long)head * a.T + w.start + min(row, w.len - 1);
    if (w.pad) {
        if (live) {
            f32x16 zero = {};
#pragma unroll
            for (int db = 0; db < DB; ++db) store_tile(dq, db, a.D, lane, zero, 0.f);
        }
        return;
    }
    const int kvh = head / a.group, chunks = a.D * (int)sizeof(T) / 16;
    const char* kbase = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + (long long)w.start * a.sk.token + kvh * a.sk.head);
    const char* vbase = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + (long long)w.start * a.sv.token + kvh * a.sv.head);
    const uint32_t krow = (uint32_t)a.sk.token * sizeof(T), vrow = (uint32_t)a.sv.token * sizeof(T);
    const int keys = a.causal ? min(w.len, (w.tile + 1) * kDqRows) : w.len;
    const int tiles = (keys + kDqKeys - 1) / kDqKeys;
    const uint32_t lds0 = lds_address(lds);
    auto copy = [&](int j) {
        const int j0 = j * kDqKeys, last = min(w.len - 1 - j0, kDqKeys - 1);
        const uint32_t at = lds0 + (uint32_t)(j & 1) * (2 * TILE);
        L::template copy<kDqKeys, 4>(at, kbase + (long long)j0 * krow, krow, last, chunks, wave, lane);
        L::template copy<kDqKeys, 4>(at + TILE, vbase + (long long)j0 * vrow, vrow, last, chunks, wave, lane);
    };
    copy(0);

    const float c = a.scale * kLog2e;
    Frag<T> q[KS], g[KS];
    float delta = 0.f;
    {
        const long long t = w.start + min(row, w.len - 1);
        const T* qrow = static_cast<const T*>(a.q) + t * a.sq.token + head * a.sq.head;
        const T* grow = static_cast<const T*>(a.g) + t * a.sg.token + head * a.sg.head;
        const T* orow = static_cast<const T*>(a.o) + t * a.so.token + head * a.so.head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[ks] = row_terms(qrow, ks, a.D, lane, 1.f);
            g[ks] = row_terms(grow, ks, a.D, lane, 1.f);
            delta += dot(g[ks], row_terms(orow, ks, a.D, lane, 1.f));
        }
        delta = both_sum(delta);
        if (live && lane < 32) a.delta[stat] = delta;   // for the other kernel
    }
    const float lse2 = a.lse[stat] * kLog2e;
    const int rlane = L::rows_lane(lane), clane = L::cols_lane(lane), half = L::row_of_half(lane);
    f32x16 acc[DB] = {};
    for (int j = 0; j < tiles; ++j) {
        dma_wait();
        __syncthreads();   // tile j is there; everyone is done with the other one
        if (j + 1 < tiles) copy(j + 1);
        const int j0 = j * kDqKeys;
        if (rows_left <= 0 || (a.causal && j0 > row0 + 31)) continue;
        const char* kt = lds + (j & 1) * (2 * TILE) + rlane;
        const char* kc = lds + (j & 1) * (2 * TILE) + clane;
        const int limit = a.causal ? min(w.len - 1, row) : w.len - 1;
        const bool edge = j0 + kDqKeys - 1 > (a.causal ? min(w.len - 1, row0) : w.len - 1);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            f32x16 s = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                mma(L::rows(kt, 32 * kb, ks), q[ks], s);
                mma(L::rows(kt + TILE, 32 * kb, ks), g[ks], dp);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2));
                s[r] = p * (dp[r] - delta);
            }
            if (edge) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (j0 + 32 * kb + L::row_of(r) + half > limit) s[r] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Frag<T> ds;
                as_terms(s, t, ds);
#pragma unroll
                for (int db = 0; db < DB; ++db) mma(L::cols(kc, 32 * kb, t, db), ds, acc[db]);
            }
        }
    }
    if (!live) return;
#pragma unroll
    for (int db = 0; db < DB; ++db) store_tile(dq, db, a.D, lane, acc[db], a.scale);
}

template <typename T, int DP>
__global__ void __launch_bounds__(256, occupancy(kDkv, sizeof(T), DP)) k_attn_dkv(Args a) {
    using L = Tile<T, DP>;
    constexpr int KS = DP / 16, DB = DP / 32, ROWS = kDkvRows<T>, TILE = L::bytes(ROWS);
    __shared__ __align__(16) char lds[4 * TILE];   // 2 x (Q tile, dO tile)
    __shared__ __align__(16) float stats[2][2][ROWS];   // 2 x (lse log2(e), delta) of the tile's queries
    static_assert(4 * TILE + 4 * ROWS * 4 <= 160 * 1024, "shared memory");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = blockIdx.x % a.Hk, slot = blockIdx.x / a.Hk;   // early tiles have the most queries when causal
    const Work w = find_work<kDkvKeys>(a, slot, lane);
    if (w.none) return;
    const int key0 = w.tile * kDkvKeys + wave * 32, key = key0 + (lane & 31);
    const int keys_left = w.len - key0;
    const bool live = key < w.len;
    T* dk = static_cast<T*>(a.dk) + (long long)(w.start + key) * a.sdk.token + kvh * a.sdk.head;
    T* dv = static_cast<T*>(a.dv) + (long long)(w.start + key) * a.sdv.token + kvh * a.sdv.head;
    if (w.pad) {
        if (live) {
            f32x16 zero = {};
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                store_tile(dk, db, a.D, lane, zero, 0.f);
                store_tile(dv, db, a.D, lane, zero, 0.f);
            }
        }
        return;
    }
    const int chunks = a.D * (int)sizeof(T) / 16;
    const uint32_t qrow = (uint32_t)a.sq.token * sizeof(T), grow = (uint32_t)a.sg.token * sizeof(T);
    const int first = a.causal ? w.tile * kDkvKeys / ROWS : 0;   // the first query tile that sees these keys
    const int per_head = (w.len + ROWS - 1) / ROWS - first, steps = per_head * a.group;
    const uint32_t lds0 = lds_address(lds);
    float stat = 0.f;   // of the tile copied last, on its way to shared memory
    auto copy = [&](int i) {
        const int head = kvh * a.group + i / per_head, j0 = (first + i % per_head) * ROWS;
        const int last = min(w.len - 1 - j0, ROWS - 1);
        const uint32_t at = lds0 + (uint32_t)(i & 1) * (2 * TILE);
        const T* qp = static_cast<const T*>(a.q) + (long long)(w.start + j0) * a.sq.token + head * a.sq.head;
        const T* gp = static_cast<const T*>(a.g) + (long long)(w.start + j0) * a.sg.token + head * a.sg.head;
        L::template copy<ROWS, 4>(at, reinterpret_cast<const char*>(qp), qrow, last, chunks, wave, lane);
        L::template copy<ROWS, 4>(at + TILE, reinterpret_cast<const char*>(gp), grow, last, chunks, wave, lane);
        if (threadIdx.x < 2 * ROWS) {
            // kept in the order that a result's registers have the rows in
            const int r = threadIdx.x % ROWS / 32 * 32 + L::place(threadIdx.x % 32);
            const long long t = (long long)head * a.T + w.start + j0 + min(r, last);
            // queries past the end: exp2(. - infinity) leaves nothing of them
            stat = threadIdx.x < ROWS ? (r <= last ? a.lse[t] * kLog2e : __builtin_inff()) : a.delta[t];
        }
    };
    copy(0);

    const float c = a.scale * kLog2e;
    Frag<T> kf[KS], vf[KS];
    {
        const long long t = w.start + min(key, w.len - 1);
        const T* krow = static_cast<const T*>(a.k) + t * a.sk.token + kvh * a.sk.head;
        const T* vrow = static_cast<const T*>(a.v) + t * a.sv.token + kvh * a.sv.head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            kf[ks] = row_terms(krow, ks, a.D, lane, 1.f);
            vf[ks] = row_terms(vrow, ks, a.D, lane, 1.f);
        }
    }
    const int rlane = L::rows_lane(lane), clane = L::cols_lane(lane), half = L::row_of_half(lane);
    f32x16 ak[DB] = {}, av[DB] = {};
    for (int i = 0; i < steps; ++i) {
        if (threadIdx.x < 2 * ROWS) stats[i & 1][threadIdx.x / ROWS][threadIdx.x % ROWS] = stat;
        dma_wait();
        __syncthreads();   // tile i is there; everyone is done with the other one
        if (i + 1 < steps) copy(i + 1);
        const int j0 = (first + i % per_head) * ROWS;
        if (keys_left <= 0 || (a.causal && j0 + ROWS - 1 < key0)) continue;
        const char* qt = lds + (i & 1) * (2 * TILE) + rlane;
        const char* qc = lds + (i & 1) * (2 * TILE) + clane;
#pragma unroll
        for (int qb = 0; qb < ROWS / 32; ++qb) {
            f32x16 s = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                mma(L::rows(qt, 32 * qb, ks), kf[ks], s);
                mma(L::rows(qt + TILE, 32 * qb, ks), vf[ks], dp);
            }
            const float* lse = &stats[i & 1][0][32 * qb + 4 * (lane >> 5)];
            const float* del = &stats[i & 1][1][32 * qb + 4 * (lane >> 5)];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int at = 8 * (r >> 2) + (r & 3);
                float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse[at]));
                float ds = p * (dp[r] - del[at]);
                if (a.causal && j0 + 32 * qb + L::row_of(r) + half < key) p = ds = 0.f;
                s[r] = p;
                dp[r] = ds;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Frag<T> p, ds;
                as_terms(s, t, p);
                as_terms(dp, t, ds);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    mma(L::cols(qc + TILE, 32 * qb, t, db), p, av[db]);
                    mma(L::cols(qc, 32 * qb, t, db), ds, ak[db]);
                }
            }
        }
    }
    if (!live) return;
#pragma unroll
    for (int db = 0; db < DB; ++db) {
        store_tile(dk, db, a.D, lane, ak[db], a.scale);
        store_tile(dv, db, a.D, lane, av[db], 1.f);
    }
}

template <typename T, int DP>
int run_bwd(const Args& a, hipStream_t st) {
    const long long gq = slots(a.T, a.n_seq, kDqRows) * a.Hq, gk = slots(a.T, a.n_seq, kDkvKeys) * a.Hk;
    if (gq >= 1LL << 23 || gk >= 1LL << 23) return WTC_ESHAPE;
    hipLaunchKernelGGL((k_attn_dq<T, DP>), dim3((unsigned)gq), dim3(256), 0, st, a);
    hipLaunchKernelGGL((k_attn_dkv<T, DP>), dim3((unsigned)gk), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace attn
}  // namespace wtc
