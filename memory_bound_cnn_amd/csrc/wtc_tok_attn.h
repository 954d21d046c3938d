// Building blocks of the attention kernels (wtconv_tok_attn_*.hip).
//
// Products run on the matrix cores as 32 x 32 tiles over 16 terms.  A lane
// holds, of an A tile, row (lane % 32), and of a B tile, column (lane % 32),
// at the eight terms of its half of the wave (h = lane / 32); of a result, 16
// values of column (lane % 32), register r being row 8 (r / 4) + 4 h + r % 4.
// Any assignment of terms to (h, i) serves as long as A and B agree, and that
// is what lets a result feed the next product without moving between lanes:
// registers 8 s .. 8 s + 7 of a result are, as a B tile, the terms
//   16 s + 4 h + {0, 1, 2, 3} and 16 s + 8 + 4 h + {0, 1, 2, 3}     ("turned" order)
// and the A tile of that product is read from shared memory in this order.
// bfloat16 takes one v_mfma_f32_32x32x16_bf16 a tile (32 cycles).  A float32
// is the sum of three bfloat16 (8 of its 24 bits each, split exactly), and its
// product six of theirs: the three left out are below 2^-24 of it, so this is
// float32's own precision in 192 cycles, where the float32 instructions take
// 512 (4 sequences of 2048 tokens, 12 heads of 64: forward, dq, dk and dv 425,
// 608 and 832 us with those, 251, 382 and 512 so).
#pragma once

#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Eight terms of a lane.
template <typename T>
struct Frag;
template <>
struct Frag<uint16_t> {
    u32x4 v;
};
template <>
struct Frag<float> {
    u32x4 v[3];   // high, middle and low parts
};

__device__ __forceinline__ void mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x16& c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c,
                                                0, 0, 0);
}
__device__ __forceinline__ void mma(const Frag<float>& a, const Frag<float>& b, f32x16& c) {
    auto part = [&](int i, int j) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.v[i]),
                                                    __builtin_bit_cast(bf16x8, b.v[j]), c, 0, 0, 0);
    };
    part(0, 2);
    part(2, 0);
    part(1, 1);
    part(0, 1);
    part(1, 0);
    part(0, 0);
}

// Two float32 to the pairs of their parts; each difference is exact.
__device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = bf16x2_rne(a, b);
    a -= __builtin_bit_cast(float, hi << 16);
    b -= __builtin_bit_cast(float, hi & 0xFFFF0000u);
    mid = bf16x2_rne(a, b);
    a -= __builtin_bit_cast(float, mid << 16);
    b -= __builtin_bit_cast(float, mid & 0xFFFF0000u);
    lo = bf16x2_rne(a, b);
}
__device__ __forceinline__ Frag<float> split8(const f32x4& x, const f32x4& y) {
    Frag<float> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h, m, l;
        if (i < 2)
            split(x[2 * i], x[2 * i + 1], h, m, l);
        else
            split(y[2 * i - 4], y[2 * i - 3], h, m, l);
        f.v[0][i] = h;
        f.v[1][i] = m;
        f.v[2][i] = l;
    }
    return f;
}

// Registers 8 s .. 8 s + 7 of a result as the terms of a B tile.  bfloat16:
// rounded to nearest even; the sums stay in 32 bits, and the tile's values
// reach them with the same 8 bits as the tensors they are multiplied with.
__device__ __forceinline__ void as_terms(const f32x16& c, int s, Frag<uint16_t>& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = bf16x2_rne(c[8 * s + 2 * i], c[8 * s + 2 * i + 1]);
}
__device__ __forceinline__ void as_terms(const f32x16& c, int s, Frag<float>& f) {
    f = split8(f32x4{c[8 * s], c[8 * s + 1], c[8 * s + 2], c[8 * s + 3]},
               f32x4{c[8 * s + 4], c[8 * s + 5], c[8 * s + 6], c[8 * s + 7]});
}

// A tile of ROWS rows in shared memory: groups of 1024 bytes (kGroup whole
// rows of 16-bit channels, what one copying instruction moves), 32 bytes
// between groups; float32 has three such parts, one after another.
//   Lane l of an A tile stands for row place(l) of 32, not for row l: place()
// sends the bits of l to bits of the row so that lanes next to each other read
// different banks (256 bytes wide), rows() and cols() alike, and every read of
// a tile is one register plus a constant: place(a + b) = place(a) + place(b)
// where a and b share no bit, and row_at() likewise.  Results whose rows are
// rows of the tile have them in that order.
//   Bits 0 and 1 of l are the four rows of 64 bytes that cols() reads at once:
// they step by 64 bytes or more.  Bit 2 is the wave's half in cols().  Bits 0
// to 3 are what rows() reads at once, 16 bytes a lane; bit 3 steps by 256
// bytes, so rows with that bit set have their 16-byte chunks swapped in pairs
// (kSwap).
template <typename T, int DP, int ROWS>
struct Tile {
    static constexpr int kParts = sizeof(T) == 2 ? 1 : 3;
    static constexpr int kRowBytes = (DP == 96 ? 128 : DP) * 2;
    static constexpr int kChunks = kRowBytes / 16;     // of 8 channels; a power of two
    static constexpr int kGroup = 1024 / kRowBytes;    // rows of a group: 4, 8 or 16
    static constexpr int kStride = 1024 + 32;
    static constexpr int kSwap = kRowBytes == 256 ? 1 : kRowBytes == 128 ? 2 : 4;   // a bit of the row
    static constexpr int kPart = ROWS / kGroup * kStride;
    static constexpr int kBytes = kParts * kPart;

    // The row bits that bits 0 .. 4 of l go to.  Rows of 64 bytes: the group is
    // bit 4 of the row; 128: bits 3 and 4; 256: bits 2 to 4.
    static constexpr __host__ __device__ int place(int l) {
        constexpr int to[3][5] = {{0, 1, 4, 2, 3}, {0, 4, 3, 1, 2}, {3, 4, 2, 0, 1}};
        constexpr int k = kRowBytes == 64 ? 0 : kRowBytes == 128 ? 1 : 2;
        int r = 0;
        for (int b = 0; b < 5; ++b) r |= ((l >> b) & 1) << to[k][b];
        return r;
    }
    static constexpr __host__ __device__ int row_at(int r) { return r / kGroup * kStride + r % kGroup * kRowBytes; }

    // Rows j0 .. j0 + ROWS - 1 of a matrix on their way into the tile, which
    // commit() ends: a barrier then makes them visible.  Rows past `last`
    // repeat row `last`, chunks past the head's channels its last chunk, so
    // that nothing outside the sequence is read (those places meet zeros or are
    // not used).  `base` points at row j0, `dst` is the tile's byte address in
    // shared memory, `chunks` the head's channels / 8.  The workgroup has four
    // waves.  bfloat16 is copied by the memory system; float32 passes through
    // registers, where it is split, once for all the waves that read it.
    static constexpr int kUnits = sizeof(T) == 2 ? 1 : (ROWS * kChunks + 255) / 256;   // of 8 channels, a thread
    struct Load {
        f32x4 v[kUnits][2];
    };
    static __device__ __forceinline__ void issue(Load& load, uint32_t dst, const char* base, uint32_t row_bytes, int last,
                                                 int chunks, int wave, int lane) {
        if constexpr (sizeof(T) == 2) {
            constexpr int CALLS = ROWS / kGroup / 4;
            static_assert(ROWS % (kGroup * 4) == 0, "whole groups");
            const int r = lane / kChunks;   // of the group
            const uint32_t c = (uint32_t)min((lane % kChunks) ^ (r & kSwap ? 1 : 0), chunks - 1) * 16u;
            if (last >= ROWS - 1) {
                const uint32_t off = (uint32_t)r * row_bytes + c;
#pragma unroll
                for (int i = 0; i < CALLS; ++i) {
                    const int g = wave * CALLS + i;
                    dma(dst + (uint32_t)(g * kStride), base + (size_t)(uint32_t)(g * kGroup) * row_bytes, off);
                }
            } else {
#pragma unroll
                for (int i = 0; i < CALLS; ++i) {
                    const int g = wave * CALLS + i;
                    dma(dst + (uint32_t)(g * kStride), base, (uint32_t)min(g * kGroup + r, last) * row_bytes + c);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int u = 256 * i + 64 * wave + lane;   // past the last row: not committed
                const char* p = base + (uint32_t)min(u / kChunks, last) * row_bytes +
                                (uint32_t)min(u % kChunks, chunks - 1) * 32u;
                load.v[i][0] = *reinterpret_cast<const f32x4*>(p);
                load.v[i][1] = *reinterpret_cast<const f32x4*>(p + 16);
            }
        }
    }
    static __device__ __forceinline__ void commit(const Load& load, char* tile, int wave, int lane) {
        if constexpr (sizeof(T) == 2) {
            // the builtin tells the compiler that its own loads are done as well: it then adds no wait for them in a
            // loop, where it would also be one for the copies.  It knows nothing of the copies, hence the other.
            __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int u = 256 * i + 64 * wave + lane, r = u / kChunks;
                if (ROWS * kChunks % 256 != 0 && u >= ROWS * kChunks) break;
                const Frag<float> f = split8(load.v[i][0], load.v[i][1]);
                char* p = tile + row_at(r) + (((u % kChunks) ^ (r & kSwap ? 1 : 0)) << 4);
#pragma unroll
                for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4*>(p + k * kPart) = f.v[k];
            }
        }
    }
    // 16 bytes a lane from base + off to 1024 consecutive bytes at dst.  A scalar register that a vector instruction
    // wrote may be an address five instructions later; the compiler sees to that outside of asm only.
    static __device__ __forceinline__ void dma(uint32_t dst, const char* base, uint32_t off) {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(off), "s"(base)
                     : "m0", "memory");
    }

    // The lane's part of the addresses that rows() and cols() read.
    static __device__ __forceinline__ int rows_lane(int lane) {
        const int r = place(lane & 31);
        return row_at(r) + (((lane >> 5) * 16) ^ (r & kSwap ? 16 : 0));
    }
    static __device__ __forceinline__ int cols_lane(int lane) {
        return row_at(place(4 * (lane >> 5) + ((lane & 15) >> 2))) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    }

    // Terms 16 ks + 8 h .. + 7 of row r0 + place(lane % 32), r0 a multiple of
    // 32: an A tile whose rows are rows of the matrix.  p = tile + rows_lane().
    static __device__ __forceinline__ Frag<T> rows(const char* p, int r0, int ks) {
        p += row_at(r0) + 32 * ks;
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            f.v = *reinterpret_cast<const u32x4*>(p);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) f.v[k] = *reinterpret_cast<const u32x4*>(p + k * kPart);
        }
        return f;
    }

    // Rows r0 + place(16 s + the turned order), of column 32 db + lane % 32: an
    // A tile whose rows are columns of the matrix.  p = tile + cols_lane(), and
    // swap = cols_swap(), to the other chunk of a pair, for the rows of l's bit 3.
    // 16 lanes read 4 rows of 16 columns and get them transposed, 4 rows of a
    // column each.
    static __device__ __forceinline__ int cols_swap(int lane) { return lane & 2 ? -16 : 16; }
    static __device__ __forceinline__ u32x4 cols_part(const char* p, int swap, int s) {
        u32x4 v;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(lds_char*)(p + k * swap + row_at(place(16 * s + 8 * k))));
            const u32x2 u = __builtin_bit_cast(u32x2, t);
            v[2 * k] = u[0];
            v[2 * k + 1] = u[1];
        }
        return v;
    }
    static __device__ __forceinline__ Frag<T> cols(const char* p, int swap, int r0, int s, int db) {
        p += row_at(r0) + 64 * db;
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            f.v = cols_part(p, swap, s);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) f.v[k] = cols_part(p + k * kPart, swap, s);
        }
        return f;
    }

    // Row of register r of a result whose rows are rows of the tile (32 of them): + 4 h's part.
    static constexpr __host__ __device__ int row_of(int r) { return place(8 * (r >> 2) + (r & 3)); }
    static __device__ __forceinline__ int row_of_half(int lane) { return place(4) * (lane >> 5); }
};

// v, but what is derived from it is not kept in registers over a loop: a
// register too many there is stored away, and its reload waits for every copy
// that is on its way.
__device__ __forceinline__ int anew(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(lds_char*)p; }

// 8 channels from c on of a row of D in device memory; zeros from D on.  Read
// with no branch, so that the loads of a row are on their way together.
template <typename T>
struct Eight {
    u32x4 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* row, int c) {
    Eight<T> x;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.u[i] = reinterpret_cast<const u32x4*>(row + c)[i];
    return x;
}

// Terms 16 ks + 8 h .. + 7, ks < KS, of one row (D > 16 KS - 32 channels, the
// others zero), times `sign` (+1 or -1): B tiles whose columns are rows of the
// matrix.
template <typename T, int KS>
__device__ __forceinline__ void load_row(const T* row, int D, int lane, float sign, Eight<T> (&x)[KS]) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int c = 16 * ks + 8 * (lane >> 5);
        x[ks] = load_eight(row, ks < KS - 2 || c < D ? c : 0);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int c = 16 * ks + 8 * (lane >> 5);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            if (ks >= KS - 2 && c >= D) x[ks].u[i] = u32x4{0u, 0u, 0u, 0u};
            if (sign < 0.f) x[ks].u[i] ^= sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
        }
    }
}
template <typename T>
__device__ __forceinline__ Frag<T> terms_of(const Eight<T>& x) {
    if constexpr (sizeof(T) == 2)
        return Frag<T>{x.u[0]};
    else
        return split8(__builtin_bit_cast(f32x4, x.u[0]), __builtin_bit_cast(f32x4, x.u[1]));
}
template <typename T, int KS>
__device__ __forceinline__ void row_terms(const T* row, int D, int lane, float sign, Frag<T> (&f)[KS]) {
    Eight<T> x[KS];
    load_row(row, D, lane, sign, x);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) f[ks] = terms_of<T>(x[ks]);
}
// The same kept as they were loaded, and split anew at each use.
template <typename T>
__device__ __forceinline__ Frag<T> terms_anew(Eight<T> x) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) asm volatile("" : "+v"(x.u[i]));
    return terms_of<T>(x);
}

// The lane's half of the terms of a . b, rows of D > 16 KS - 32 channels in
// device memory.
template <typename T, int KS>
__device__ __forceinline__ float half_dot(const T* a, const T* b, int D, int lane) {
    Eight<T> x[KS], y[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int c = 16 * ks + 8 * (lane >> 5), at = ks < KS - 2 || c < D ? c : 0;
        x[ks] = load_eight(a, at);
        y[ks] = load_eight(b, at);
    }
    float v = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t p = x[ks].u[i][j], q = y[ks].u[i][j];
                if constexpr (sizeof(T) == 2) {
                    part = fmaf(__builtin_bit_cast(float, p << 16), __builtin_bit_cast(float, q << 16), part);
                    part = fmaf(__builtin_bit_cast(float, p & 0xFFFF0000u), __builtin_bit_cast(float, q & 0xFFFF0000u), part);
                } else {
                    part = fmaf(__builtin_bit_cast(float, p), __builtin_bit_cast(float, q), part);
                }
            }
        v += ks < KS - 2 || 16 * ks + 8 * (lane >> 5) < D ? part : 0.f;
    }
    return v;
}

// The value of the lane with the same column in the other half, joined with
// this one's: both halves get the maximum or the sum.
__device__ __forceinline__ float both_max(float v) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                     false, false);
    const uint32_t x = r[0], y = r[1];
    return fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float both_sum(float v) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                     false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Stores a wave's 32 rows from the result tiles of a transposed output (lane:
// row lane % 32, channels 32 db + 8 (r / 4) + 4 h + r % 4), times `factor`:
// rows 0 .. rows - 1 of D channels, `stride` elements apart.  They pass through
// shared memory, a place of the wave's own (`at`, kRowsScratch bytes that
// nothing else uses now), so that a store has whole rows of 16-byte chunks
// instead of 8 bytes of 32 rows each.  The 8-byte writes of bfloat16 rows on
// their way in are the only accesses that meet a bank twice: 53 cycles for a
// wave's 32 rows of 64 channels (SQ_LDS_BANK_CONFLICT counts them once in dq,
// twice in the forward pass with out_low and in dk and dv), float32's none in 128.
template <typename T, int DP>
constexpr int kScratchRow = DP * (int)sizeof(T) + 16;   // 16 bytes more: rows begin in different banks
template <typename T, int DP>
constexpr int kRowsScratch = 32 * kScratchRow<T, DP>;

template <typename T, int DP>
__device__ __forceinline__ void store_rows(char* at, T* out, long long stride, int rows, int D, int lane,
                                           const f32x16 (&c)[DP / 32], float factor) {
    constexpr int ROW = kScratchRow<T, DP>, CH = DP * (int)sizeof(T) / 16;
    asm volatile("" ::: "memory");
    char* p = at + (lane & 31) * ROW + (lane >> 5) * 4 * (int)sizeof(T);
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 v = f32x4{c[db][4 * g], c[db][4 * g + 1], c[db][4 * g + 2], c[db][4 * g + 3]} * factor;
            char* to = p + (32 * db + 8 * g) * (int)sizeof(T);
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<u32x2*>(to) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
            else
                *reinterpret_cast<f32x4*>(to) = v;
        }
    asm volatile("" ::: "memory");   // a wave's own accesses to shared memory stay in order
#pragma unroll
    for (int i = 0; i < 32 * CH / 64; ++i) {
        const int u = 64 * i + lane, r = u / CH, k = u % CH;
        const u32x4 v = *reinterpret_cast<const u32x4*>(at + r * ROW + 16 * k);
        if (r < rows && k * kVec<T> < D) *reinterpret_cast<u32x4*>(out + r * stride + k * kVec<T>) = v;
    }
}

constexpr int max_of(int a, int b) { return a > b ? a : b; }

// Workgroups (of four waves, one on each vector unit) that the registers of a
// compute unit hold at least.
enum Kernel { kFwd, kDq, kDkv };
constexpr int occupancy(Kernel k, int elem, int dp) {
    if (elem == 4) return dp <= 64 ? 2 : 1;
    return dp > 64 ? 2 : dp > 32 && k != kFwd ? 3 : 4;
}

constexpr long long kMaxGroups = 1LL << 23;   // workgroups of a launch: 2^31 threads

struct Args {
    const void *q, *k, *v, *o, *g;
    const int* cu;
    void *out, *dq, *dk, *dv;
    void* low;   // what was rounded off the output, [T, Hq, D] bfloat16, or null
    float *lse, *delta;
    int q_splits, k_splits;   // of a query tile's keys, of a key tile's queries; with several, their results:
    float* parts;             // sums [split][T, heads, D] (dk and dv: [split][2][T, heads, D])
    float* stat;              // forward: maximum c, log2, and sum of exp2, [split][2][row_floats]
    long long row_floats;
    int T, n_seq, Hq, Hk, group, D, causal;
    float scale;
    wtc_attn_strides sq, sk, sv, so, sg, sdq, sdk, sdv;
};

// The segment and the tile of SIZE rows that a workgroup works on.  Segments
// are the tokens before the first sequence, the sequences, and the tokens
// after the last one.  Up to 64 segments a wave holds one in each lane and
// hands out the tiles with the most work first, so that long ones do not start
// when the chip is running empty: by the length of their sequence, or when
// causal by the number of keys (of queries) that the tile itself meets.  Both
// orders count the work in tiles: with w(L) = the tiles that come before all
// those of L tiles' work, the slot's L is found by bisection, with no plan on
// the host.  Measured against the order of the sequences (forward, dq, dk and
// dv): 48 images of 49 to 1024 tokens, 6 heads of 64 channels, 65 / 85 / 104 ->
// 56 / 78 / 87 us; 4 causal sequences of 2000 to 4096, 8 heads of 96, 129 / 165
// / 204 -> 104 / 136 / 175; equal lengths the same within 3 %.
//   More segments: segment s may use the slots from floor(start / SIZE) + s on.
// That leaves ceil(length / SIZE) slots at least to each, and a slot's segment
// is found by searching cu_seqlens itself, 63 segments at a time.
struct Work {
    int start, len, tile;
    bool pad;    // tokens of no sequence
    bool none;   // a slot that no tile has
};
__device__ __forceinline__ int bound_of(const Args& a, int s) {
    if (s <= 0) return 0;
    if (s >= a.n_seq + 2) return a.T;
    return min(max(a.cu[s - 1], 0), a.T);
}

// Sum and maximum over the wave of values that are not negative, the same in every lane.
template <typename F>
__device__ __forceinline__ int wave_join(int v, const F& f) {
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));   // row_shr 1, 2, 4, 8
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));   // row_bcast 15 into rows 1 and 3
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));   // row_bcast 31 into rows 2 and 3
    return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ int wave_sum(int v) {
    return wave_join(v, [](int x, int y) { return x + y; });
}
__device__ __forceinline__ int wave_max(int v) {
    return wave_join(v, [](int x, int y) { return max(x, y); });
}

// LATE: when causal, a sequence's late tiles have the most work (its queries
// do); otherwise its early ones (its keys do).
template <int SIZE, bool LATE>
__device__ __forceinline__ Work find_work(const Args& a, int slot, int lane) {
    const int segments = a.n_seq + 2;
    Work w;
    if (segments <= 64) {
        const int start = bound_of(a, lane), next = __shfl_down(start, 1);
        const int len = max((lane < 63 ? next : a.T) - start, 0);   // 0 past the last one
        const bool pad = lane == 0 || lane == segments - 1;
        const int tiles = (len + SIZE - 1) / SIZE, real = pad ? 0 : tiles;
        auto before = [&](int L) {   // tiles of more than L tiles' work
            return wave_sum(real > L ? (a.causal ? real - L : real) : 0);
        };
        int lo = 0, hi = wave_max(real), above = 0;   // the slot's work is in lo + 1 .. hi; above = before(hi)
        const int all = before(0);
        int at;
        if (slot < all) {
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2, n = before(mid);
                if (n > slot) {
                    lo = mid;
                } else {
                    hi = mid;
                    above = n;
                }
            }
            int k = slot - above;   // among the tiles of hi tiles' work
            if (a.causal) {
                w.tile = hi - 1;
            } else {
                w.tile = k % hi;
                k /= hi;
            }
            const uint64_t these = __builtin_amdgcn_ballot_w64(a.causal ? real >= hi : real == hi);
            const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(these >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)these, 0));
            at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(((these >> lane) & 1) && rank == k) | (1ull << 63));
            if (a.causal && !LATE) w.tile = __builtin_amdgcn_readlane(real, at) - hi;
        } else {   // the tokens of no sequence
            const int first = __builtin_amdgcn_readlane(tiles, 0);
            w.tile = slot - all;
            at = w.tile < first ? 0 : segments - 1;
            if (at != 0) w.tile -= first;
        }
        w.start = __builtin_amdgcn_readlane(start, at);
        w.len = __builtin_amdgcn_readlane(len, at);
        w.pad = at == 0 || at == segments - 1;
    } else {
        int lo = 0, hi = segments;   // the segment is in lo .. hi - 1
        for (;;) {
            const int step = (hi - lo + 62) / 63, s = lo + lane * step;
            const int b = bound_of(a, min(s, hi));   // where the lane's segment starts
            const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(s < hi && b / SIZE + s <= slot));
            const int at = n > 0 ? n - 1 : 0;
            lo += at * step;
            hi = min(hi, lo + step);
            if (step == 1) {   // the segment's bounds are two lanes' own
                w.start = __builtin_amdgcn_readlane(b, at);
                w.len = max(__builtin_amdgcn_readlane(b, at + 1) - w.start, 0);
                break;
            }
        }
        w.tile = slot - (w.start / SIZE + lo);
        w.pad = lo == 0 || lo == segments - 1;
    }
    w.none = w.tile < 0 || (long long)w.tile * SIZE >= w.len;
    return w;
}
inline long long slots(long long T, int n_seq, int size) { return T / size + n_seq + 2; }

// workgroups of 256 for a join of splits, which strides over what is left
inline unsigned join_groups(long long threads) {
    const long long groups = (threads + 255) / 256;
    return (unsigned)(groups < 8192 ? groups : 8192);
}

}  // namespace attn
}  // namespace wtc
