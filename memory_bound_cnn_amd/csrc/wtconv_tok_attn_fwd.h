// Attention, forward: O = softmax(scale Q K^T) V inside each sequence, one pass
// over the keys with the running maximum and sum of the softmax.
//
// A workgroup of four waves takes one head and 128 queries, 32 a wave; tiles of
// 64 keys and values pass through shared memory, two tiles deep, copied there
// directly from device memory while the tile before is worked on.  Per tile a
// wave computes S^T = K Q^T (rows are keys, columns its queries), so that a lane
// has 32 of the 64 products of one query: the maximum and the sum take one
// exchange between the two halves of the wave, the scale of the running sums is
// the lane's own, and P^T feeds O^T = V^T P^T from the registers it is in.
//
// Where a pack has few query tiles, several workgroups share the keys of one;
// their sums, maxima and sums of exponentials go to a workspace and a second
// kernel joins them.
//
// Bound by the matrix units and, about as long again, the exponentials and
// roundings between the two products.  Means of 20 training steps (the
// fastest up to 18 % less): bfloat16, 48 images of 49 to 1024 tokens, 6 heads of
// 64: 66 us (500 TFLOP/s); 4 x 4096, 12 heads of 64: 253 us (815); causal 3 x
// 3500..8192, 16 heads on 4 of 128: 374 us (925); float32, in six products of
// bfloat16 parts, 32 x 196, 6 heads on 3 of 64: 26 us (71).
#pragma once

#include "wtc_tok_attn.h"

namespace wtc {
namespace attn {

constexpr int kFwdRows = 128;   // queries of a workgroup
template <typename T>
constexpr int kFwdKeys = sizeof(T) == 2 ? 64 : 32;   // keys of a tile

// The running maximum is raised, and the sums rescaled, only when a tile
// exceeds it by more than this many powers of two: P then reaches 2^8 instead
// of 1, far from overflow in 32-bit sums, with the same relative rounding.
constexpr float kRaise = 8.f;

template <typename T, int DP>
__global__ void __launch_bounds__(256, occupancy(kFwd, sizeof(T), DP)) k_attn_fwd(Args a) {
    constexpr int KEYS = kFwdKeys<T>, KB = KEYS / 32, KS = DP / 16, DB = DP / 32;
    using L = Tile<T, DP, KEYS>;
    constexpr int TILE = L::kBytes, LDS = max_of(4 * TILE, 4 * kRowsScratch<float, DP>);
    __shared__ __align__(16) char lds[LDS];   // 2 x (K tile, V tile); then a place to store from
    static_assert(LDS <= 160 * 1024, "shared memory");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % a.Hq, split = blockIdx.x / a.Hq % a.q_splits;
    const Work w = find_work<kFwdRows, true>(a, blockIdx.x / a.Hq / a.q_splits, lane);
    if (w.none) return;
    const int row0 = w.tile * kFwdRows + wave * 32, row = row0 + (lane & 31);   // inside the segment
    const int rows_left = w.len - row0;                                         // <= 0: this wave has none
    const bool live = row < w.len;
    T* out = static_cast<T*>(a.out) + (long long)(w.start + row0) * a.so.token + head * a.so.head;
    char* scratch = lds + wave * kRowsScratch<T, DP>;
    const long long stat = (long long)head * a.T + w.start + row;
    float* lse = a.lse ? a.lse + stat : nullptr;
    // a split's row: the maximum (times c) that its sums are over, and the sum of
    // its exponentials; inf and 0 for a token of no sequence, -inf and 0 where the
    // split has nothing for the row
    auto store_stat = [&](float top, float sum) {
        if (!live || lane >= 32) return;
        a.stat[2 * split * a.row_floats + stat] = top;
        a.stat[(2 * split + 1) * a.row_floats + stat] = sum;
    };
    if (w.pad) {
        if (a.q_splits > 1) {
            store_stat(__builtin_inff(), 0.f);
            return;
        }
        const f32x16 zero[DB] = {};
        store_rows<T, DP>(scratch, out, a.so.token, rows_left, a.D, lane, zero, 0.f);
        if (lse && live && lane < 32) *lse = __builtin_inff();
        return;
    }
    const int kvh = head / a.group, chunks = a.D / 8;
    const char* kbase = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + (long long)w.start * a.sk.token + kvh * a.sk.head);
    const char* vbase = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + (long long)w.start * a.sv.token + kvh * a.sv.head);
    const uint32_t krow = (uint32_t)a.sk.token * sizeof(T), vrow = (uint32_t)a.sv.token * sizeof(T);
    const int keys = a.causal ? min(w.len, (w.tile + 1) * kFwdRows) : w.len;
    const int tiles = (keys + KEYS - 1) / KEYS;
    const int begin = (int)((long long)tiles * split / a.q_splits), end = (int)((long long)tiles * (split + 1) / a.q_splits);
    if (begin == end) {
        store_stat(-__builtin_inff(), 0.f);
        return;
    }
    const uint32_t lds0 = lds_address(lds);
    typename L::Load kload, vload;
    auto copy = [&](int j) {
        const int j0 = j * KEYS, last = min(w.len - 1 - j0, KEYS - 1);
        const uint32_t at = lds0 + (uint32_t)(j & 1) * (2 * TILE);
        L::issue(kload, at, kbase + (long long)j0 * krow, krow, last, chunks, wave, lane);
        L::issue(vload, at + TILE, vbase + (long long)j0 * vrow, vrow, last, chunks, wave, lane);
    };
    copy(begin);

    // a negative scale is taken into Q, so that the largest product is the largest logit
    // (and no scale below 2^-100, a zero one: it must not meet the infinity of a masked product)
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);
    Frag<T> q[KS];
    {
        const T* qrow = static_cast<const T*>(a.q) + (long long)(w.start + min(row, w.len - 1)) * a.sq.token + head * a.sq.head;
        row_terms(qrow, a.D, lane, a.scale < 0.f ? -1.f : 1.f, q);
    }
    f32x16 o[DB] = {};
    const int rlane = L::rows_lane(lane), clane = L::cols_lane(lane), half = L::row_of_half(lane), swap = L::cols_swap(lane);
    float m = -__builtin_inff(), mc = 0.f, l = 0.f;   // mc = m c, finite
    for (int j = begin; j < end; ++j) {
        L::commit(kload, lds + (j & 1) * (2 * TILE), wave, lane);
        L::commit(vload, lds + (j & 1) * (2 * TILE) + TILE, wave, lane);
        __syncthreads();   // tile j is there; everyone is done with the other one
        if (j + 1 < end) copy(j + 1);
        const int j0 = j * KEYS;
        if (rows_left <= 0 || (a.causal && j0 > row0 + 31)) continue;   // nothing of this tile for this wave
        const char* kt = lds + (j & 1) * (2 * TILE) + rlane;
        const char* vt = lds + (j & 1) * (2 * TILE) + TILE + clane;
        // waves in a product go before waves in a softmax, whose vector work then
        // runs beside it (4 x 4096 tokens, 12 heads of 64: 246 -> 239 us)
        __builtin_amdgcn_s_setprio(1);
        f32x16 s[KB] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) mma(L::rows(kt, 32 * kb, ks), q[ks], s[kb]);
        __builtin_amdgcn_s_setprio(0);
        const int seen = (a.causal ? min(w.len - 1, row) : w.len - 1) - j0 - half;   // last key of the tile that this query sees
        const bool edge = j0 + KEYS - 1 > (a.causal ? min(w.len - 1, row0) : w.len - 1);
        if (edge) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * kb + L::row_of(r) > seen) s[kb][r] = -__builtin_inff();
        }
        float top = s[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
        top = both_max(top);
        // raised where a lane's tile is above its maximum by more than kRaise powers of two
        if (__builtin_amdgcn_ballot_w64((top - m) * c > kRaise || m == -__builtin_inff())) {
            const bool first = m == -__builtin_inff();
            m = fmaxf(m, top);
            const float next = m == -__builtin_inff() ? 0.f : m * c;
            const float alpha = first ? 0.f : __builtin_amdgcn_exp2f(mc - next);
            mc = next;
            l *= alpha;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] *= alpha;
        }
        float sum = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[kb][r] = __builtin_amdgcn_exp2f(fmaf(s[kb][r], c, -mc));
                sum += s[kb][r];
            }
        l += sum;
        __builtin_amdgcn_s_setprio(2);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Frag<T> p;
                as_terms(s[kb], t, p);
#pragma unroll
                for (int db = 0; db < DB; ++db) mma(L::cols(vt, swap, 32 * kb, t, db), p, o[db]);
            }
        __builtin_amdgcn_s_setprio(0);
    }
    l = both_sum(l);
    if (a.q_splits > 1) {
        store_stat(m == -__builtin_inff() ? m : mc, l);
        __syncthreads();   // everyone is done with the tiles
        if (rows_left <= 0) return;
        const long long step = (long long)a.Hq * a.D, n = a.T * step;
        store_rows<float, DP>(lds + wave * kRowsScratch<float, DP>, a.parts + split * n + (w.start + row0) * step + head * a.D,
                              step, rows_left, a.D, lane, o, 1.f);
        return;
    }
    const float inv = 1.f / l;
    if (lse && live && lane < 32) *lse = (mc + log2f(l)) * kLn2;
    __syncthreads();   // everyone is done with the tiles
    if (rows_left <= 0) return;
    store_rows<T, DP>(scratch, out, a.so.token, rows_left, a.D, lane, o, inv);
    if constexpr (sizeof(T) == 2) {
        if (a.low) {
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[db][r] = o[db][r] * inv - as_stored<T>(o[db][r] * inv);
            store_rows<T, DP>(scratch, static_cast<T*>(a.low) + ((long long)(w.start + row0) * a.Hq + head) * a.D,
                              (long long)a.Hq * a.D, rows_left, a.D, lane, o, 1.f);
        }
    }
}

// The splits' outputs joined: each weighed by 2^(its maximum - the largest one),
// over the sum of the sums so weighed.  Eight channels a thread.
template <typename T>
__global__ void __launch_bounds__(256) k_attn_join_out(Args a) {
    const int units = a.D / 8;
    const long long rows = (long long)a.T * a.Hq, n = rows * a.D, step = (long long)gridDim.x * 256;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < rows * units; i += step) {
        const long long row = i / units, t = row / a.Hq;
        const int c = (int)(i - row * units) * 8, head = (int)(row - t * a.Hq);
        const float* stat = a.stat + (long long)head * a.T + t;
        float top = -__builtin_inff(), sum = 0.f, o[8] = {};
        for (int s = 0; s < a.q_splits; ++s) top = fmaxf(top, stat[2 * s * a.row_floats]);
        for (int s = 0; s < a.q_splits; ++s) {
            const float l = stat[(2 * s + 1) * a.row_floats];
            if (l == 0.f) continue;   // nothing for this row, and nothing stored where the split has no keys
            const float weight = __builtin_amdgcn_exp2f(stat[2 * s * a.row_floats] - top);
            sum = fmaf(weight, l, sum);
            float x[4], y[4];
            load16(a.parts + s * n + row * a.D + c, x);
            load16(a.parts + s * n + row * a.D + c + 4, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j] = fmaf(weight, x[j], o[j]);
                o[4 + j] = fmaf(weight, y[j], o[4 + j]);
            }
        }
        const bool pad = top == __builtin_inff() && sum == 0.f;   // a token of no sequence
        const float inv = pad ? 0.f : 1.f / sum;
        if (a.lse && c == 0) a.lse[(long long)head * a.T + t] = pad ? top : (top + log2f(sum)) * kLn2;
        T* out = static_cast<T*>(a.out) + t * a.so.token + head * a.so.head + c;
#pragma unroll
        for (int k = 0; k < 8; k += kVec<T>) {
            float v[kVec<T>], low[kVec<T>];
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) {
                v[j] = o[k + j] * inv;
                low[j] = v[j] - as_stored<T>(v[j]);
            }
            store16(out + k, v);
            if (sizeof(T) == 2 && a.low) store16(static_cast<T*>(a.low) + row * a.D + c + k, low);
        }
    }
}

template <typename T, int DP>
int run_fwd(const Args& a, hipStream_t st) {
    const long long grid = slots(a.T, a.n_seq, kFwdRows) * a.Hq * a.q_splits;
    if (grid >= kMaxGroups) return WTC_ESHAPE;
    hipLaunchKernelGGL((k_attn_fwd<T, DP>), dim3((unsigned)grid), dim3(256), 0, st, a);
    if (a.q_splits > 1)
        hipLaunchKernelGGL((k_attn_join_out<T>), dim3(join_groups((long long)a.T * a.Hq * a.D / 8)), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace attn
}  // namespace wtc
