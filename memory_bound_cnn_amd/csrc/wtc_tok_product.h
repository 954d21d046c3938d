// Building blocks of the experts' products (wtconv_tok_product*.hip): tiles of
// matrices in shared memory and their products on the matrix cores.
//
// A workgroup makes a tile of the output, rows i by columns j (consecutive in
// memory), as 32 x 32 blocks.  The matrix instruction's A operand is the one
// with the columns and its B operand the one with the rows, so that a lane owns
// one row of the output (i = lane % 32) and register r is column
// 8 (r / 4) + 4 h + r % 4, h = lane / 32: four consecutive ones at a time.
//   An operand lies in memory with its terms (what is summed over) along the
// rows or across them:
//   Along   a row of the tile is a step's terms of a row (or column) of the
//           output; a lane reads 16 bytes of its row.
//   Across  a row of the tile is one term, its 16-byte chunks are rows (columns)
//           of the output; bfloat16 is read with the transposing instruction,
//           float32 a value at a time.
// A step takes 128 bytes of terms.  Tiles are copied by the memory system 1024
// consecutive bytes of shared memory at a time, and the chunks of a row are
// permuted on that way so that reads meet no bank twice.
#pragma once

#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"
#include "wtc_tok_segment.h"

namespace wtc {
namespace product {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

// A lane's eight terms of a read; those of the two halves of a wave are a step of the matrix instruction.
// A float32 is the sum of three bfloat16 (8 of its 24 bits each, split exactly), and its product six of theirs:
// the three left out are below 2^-24 of it, so this is float32's own precision in 192 cycles a block, where the
// float32 instructions take 512.
constexpr int kRead = 16;
constexpr int kStepBytes = 128;
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
// Eight terms as they lie in memory.
template <typename T>
struct Eight {
    u32x4 u[sizeof(T) / 2];
};
__device__ __forceinline__ Frag<uint16_t> frag(const Eight<uint16_t>& x) { return {x.u[0]}; }
__device__ __forceinline__ Frag<float> frag(const Eight<float>& x) {
    Frag<float> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = x.u[i / 2][2 * i % 4], q = x.u[i / 2][2 * i % 4 + 1];
        float a = __builtin_bit_cast(float, p), b = __builtin_bit_cast(float, q);
        const uint32_t hi = bf16x2_rne(a, b);
        a -= __builtin_bit_cast(float, hi << 16);   // each difference is exact
        b -= __builtin_bit_cast(float, hi & 0xFFFF0000u);
        const uint32_t mid = bf16x2_rne(a, b);
        a -= __builtin_bit_cast(float, mid << 16);
        b -= __builtin_bit_cast(float, mid & 0xFFFF0000u);
        f.v[0][i] = hi;
        f.v[1][i] = mid;
        f.v[2][i] = bf16x2_rne(a, b);
    }
    return f;
}
__device__ __forceinline__ void mma(const u32x4& a, const u32x4& b, f32x16& c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ void mma(const u32x4& a, const u32x4& b, f32x4& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Sums of products.  Those of float32's lower parts are apart: they are 2^-8 of the others and less, so that their six-fold
// number of additions does not round the whole.
template <typename T, typename V>
struct Sum {
    V v = {};
    __device__ __forceinline__ V all() const { return v; }
};
template <typename V>
struct Sum<float, V> {
    V v = {}, low = {};
    __device__ __forceinline__ V all() const { return v + low; }
};
template <typename V>
__device__ __forceinline__ void mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, Sum<uint16_t, V>& c) {
    mma(a.v, b.v, c.v);
}
template <typename V>
__device__ __forceinline__ void mma(const Frag<float>& a, const Frag<float>& b, Sum<float, V>& c) {
    mma(a.v[0], b.v[2], c.low);   // the smallest first
    mma(a.v[2], b.v[0], c.low);
    mma(a.v[1], b.v[1], c.low);
    mma(a.v[0], b.v[0], c.v);
    mma(a.v[0], b.v[1], c.low);
    mma(a.v[1], b.v[0], c.low);
}

__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(lds_char*)p; }

// 16 bytes a lane from base + off to 1024 consecutive bytes at dst.  A scalar register that a vector instruction
// wrote may be an address five instructions later; the compiler sees to that outside of asm only.
__device__ __forceinline__ void copy1024(uint32_t dst, const char* base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(off), "s"(base)
                 : "m0", "memory");
}

// v, but what is derived from it is not kept in registers over a loop.
__device__ __forceinline__ int anew(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// N rows (or columns) of an operand whose terms lie along its rows, a step's 128 bytes of terms.
template <typename T, int N, int WAVES>
struct Along {
    static constexpr int kBytes = N * kStepBytes, kCopies = kBytes / 1024 / WAVES, kChunks = kStepBytes / 16;
    static_assert(kBytes % (1024 * WAVES) == 0, "whole copies");
    // 16 lanes read a chunk of 16 rows: those rows' chunks that share banks, 256 bytes apart, are exchanged
    static constexpr __host__ __device__ int turn(int row) { return (row * kStepBytes / 256) & (kChunks - 1); }
    uint32_t off[kCopies];   // bytes from the operand's first row to the lane's part of each copy
    static __device__ __forceinline__ int row_at(int i, int wave, int lane) {
        return (wave * kCopies + i) * (64 / kChunks) + lane / kChunks;
    }
    static __device__ __forceinline__ int unit_at(int row, int lane) { return (lane % kChunks) ^ turn(row); }   // the chunk
    // rows past `last` repeat it
    __device__ __forceinline__ void place(uint32_t row_bytes, int last, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int r = row_at(i, wave, lane);
            off[i] = (uint32_t)min(r, last) * row_bytes + unit_at(r, lane) * 16;
        }
    }
    // base: the step's first term of the operand's first row; chunks: of terms that are there, if fewer than a step's
    __device__ __forceinline__ void copy(uint32_t dst, const char* base, int chunks, int wave, int lane) const {
        dst += wave * (kCopies * 1024);
        if (chunks >= kChunks) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) copy1024(dst + i * 1024, base, off[i]);
        } else {
            lane = anew(lane);
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                copy1024(dst + i * 1024, base,
                         off[i] - (uint32_t)max(unit_at(row_at(i, wave, lane), lane) - chunks + 1, 0) * 16);
        }
    }
    // The wave's i-th copy of a step that has all its terms.
    __device__ __forceinline__ void copy_one(int i, uint32_t dst, const char* base, int wave) const {
        copy1024(dst + (wave * kCopies + i) * 1024, base, off[i]);
    }
    // Zeros to the chunks of terms that are not there.
    __device__ static __forceinline__ void clear(char* tile, int chunks) {
        for (int u = threadIdx.x; u < N * kChunks; u += 64 * WAVES)
            if (((u % kChunks) ^ turn(u / kChunks)) >= chunks) *reinterpret_cast<u32x4*>(tile + u * 16) = u32x4{0u, 0u, 0u, 0u};
    }
    __device__ static __forceinline__ int lane_part(int lane) { return (lane & 31) * kStepBytes; }
    // Terms 16 at + 8 h .. of row r0 + lane % 32, r0 a multiple of 32
    __device__ static __forceinline__ Eight<T> read(const char* tile, int part, int r0, int at, int lane) {
        constexpr int UNITS = (int)sizeof(T) / 2;
        Eight<T> x;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int unit = (UNITS * (2 * at + (lane >> 5)) + k) ^ turn(lane & 31);
            x.u[k] = *reinterpret_cast<const u32x4*>(tile + part + r0 * kStepBytes + unit * 16);
        }
        return x;
    }
};

// The same of an operand whose terms lie across: a row of the tile is one term
// with N of the output's rows (or columns).
template <typename T, int N, int WAVES>
struct Across {
    static constexpr int kRow = N * (int)sizeof(T), kChunks = kRow / 16;
    static constexpr int kTerms = kStepBytes / (int)sizeof(T);
    static constexpr int kBytes = kTerms * kRow, kCopies = kBytes / 1024 / WAVES;
    static constexpr int kRowsEach = 1024 / kRow > 0 ? 1024 / kRow : 1;
    static_assert(kBytes % (1024 * WAVES) == 0 && 1024 % kRow == 0 && kRow >= 256, "whole copies, and chunks to permute");
    // the permutation of a row's chunks: bfloat16 by 64 bytes, with the four terms of one
    // transposing read; float32 by 128 bytes, with the halves of the wave
    static __device__ __forceinline__ int turn(int term) {
        return sizeof(T) == 2 ? (term & 3) << 2 : ((term >> 3) & 1) << 3;
    }
    uint32_t off[kCopies];   // bytes from the step's first term of the operand's first row (column)
    static __device__ __forceinline__ int term_at(int i, int wave, int lane) {
        return (wave * kCopies + i) * kRowsEach + lane / kChunks;
    }
    __device__ __forceinline__ void place(uint32_t row_bytes, int last_chunk, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int t = term_at(i, wave, lane);
            off[i] = (uint32_t)t * row_bytes + (uint32_t)min((lane % kChunks) ^ turn(t), last_chunk) * 16;
        }
    }
    // base: the step's first term of the operand's first row (column); last: the last term that is there
    __device__ __forceinline__ void copy(uint32_t dst, const char* base, uint32_t row_bytes, int last, int wave, int lane) const {
        dst += wave * (kCopies * 1024);
        if (last >= kTerms - 1) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) copy1024(dst + i * 1024, base, off[i]);
        } else {
            lane = anew(lane);
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                copy1024(dst + i * 1024, base, off[i] - (uint32_t)max(term_at(i, wave, lane) - last, 0) * row_bytes);
        }
    }
    __device__ __forceinline__ void copy_one(int i, uint32_t dst, const char* base, int wave) const {
        copy1024(dst + (wave * kCopies + i) * 1024, base, off[i]);
    }
    // Zeros to the terms from `there` on.
    __device__ static __forceinline__ void clear(char* tile, int there) {
        for (int b = there * kRow + (int)threadIdx.x * 16; b < kBytes; b += 64 * WAVES * 16)
            *reinterpret_cast<u32x4*>(tile + b) = u32x4{0u, 0u, 0u, 0u};
    }
    // The lane's part: of the terms it reads first, and its column's.
    __device__ static __forceinline__ int lane_part(int lane) {
        if constexpr (sizeof(T) == 2) return (8 * (lane >> 5) + ((lane & 15) >> 2)) * kRow + (lane & 3) * 8;
        return 8 * (lane >> 5) * kRow + (lane & 3) * 4;
    }
    // Terms 16 at + 8 h .. of row (column) r0 + lane % 32
    __device__ static __forceinline__ Eight<T> read(const char* tile, int part, int r0, int at, int lane) {
        Eight<T> x;
        if constexpr (sizeof(T) == 2) {
            const int c = (r0 / 8 + ((lane >> 4) & 1) * 2) ^ turn((lane & 15) >> 2);   // the last bit is in `part`
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4*)(lds_char*)(tile + part + (16 * at + 4 * k) * kRow + c * 16));
                const u32x2 u = __builtin_bit_cast(u32x2, t);
                x.u[0][2 * k] = u[0];
                x.u[0][2 * k + 1] = u[1];
            }
        } else {
            const int c = (r0 / 4 + ((lane & 31) >> 2)) ^ turn(8 * (lane >> 5));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x.u[i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(tile + part + (16 * at + i) * kRow + c * 16);
        }
        return x;
    }
};

// ------------------------------------------------------------------ work
// Segment s = 0 .. E + 1 of the rows: those before the first expert's, the experts', those after the last's.
__device__ __forceinline__ int segment_begin(const int* cu, int E, int R, int s) {
    if (s <= 0) return 0;
    if (s >= E + 2) return R;
    return min(max(cu[s - 1], 0), R);
}
// Segment s may use the tiles from floor(begin / SIZE) + s on, which leaves it
// ceil(rows / SIZE) at least; or, where there are fewer rows than that, a tile is
// numbered by its first row (BY_ROW).  Whose a tile is, is found by searching cu,
// 63 segments at a time.  count = 0: a tile of none.
template <int SIZE, bool BY_ROW = false>
__device__ __forceinline__ Rows find_rows(const int* cu, int E, int R, int slot, int lane) {
    int lo = 0, hi = E + 2, b, e;   // the segment is in lo .. hi - 1
    for (;;) {
        const int step = (hi - lo + 62) / 63, s = lo + lane * step, begin = segment_begin(cu, E, R, min(s, hi));
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(s < hi && (BY_ROW ? begin : begin / SIZE + s) <= slot)), k = n > 0 ? n - 1 : 0;
        lo += k * step;
        hi = min(hi, lo + step);
        if (step == 1) {   // the segment's bounds are two lanes' own
            b = __builtin_amdgcn_readlane(begin, k);
            e = __builtin_amdgcn_readlane(begin, k + 1);
            break;
        }
    }
    const int tile = BY_ROW ? ((slot - b) % SIZE == 0 ? (slot - b) / SIZE : -1) : slot - (b / SIZE + lo);
    return rows_of<SIZE>(lo == 0 || lo == E + 1 ? -1 : lo - 1, b, e, tile);
}
inline long long row_slots(long long R, int E, int size) { return R / size + E + 2; }

// The number of a workgroup, counted so that those of one XCD (every eighth)
// are next to each other.
__device__ __forceinline__ int spread(int id, int all) {
    const int each = all / 8, more = all % 8, x = id % 8;
    return x * each + min(x, more) + id / 8;
}

// ------------------------------------------------------------------ output
// Stores 32 rows by 32 NB columns of a wave from its blocks (see above) through
// shared memory (`at`, kStoreBytes of the wave's own), so that a store has whole
// rows of 16-byte chunks.  Rows `rows` and more, and columns `columns` and more,
// are not there.
template <typename T, int NB>
constexpr int kStoreRow = 32 * NB * (int)sizeof(T) + 16;
template <typename T, int NB>
constexpr int kStoreBytes = 32 * kStoreRow<T, NB>;

// Elements at .. at + 3 (a multiple of four) of an aligned row.
__device__ __forceinline__ void load_four(const uint16_t* p, int at, float (&v)[4]) {
    const u32x2 u = *reinterpret_cast<const u32x2*>(p + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t e = u[i];
        v[2 * i] = __builtin_bit_cast(float, e << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, e & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load_four(const float* p, int at, float (&v)[4]) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(p + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u[i];
}

template <typename T, int NB, typename S>
__device__ __forceinline__ void store_block(char* at, T* out, long long stride, int rows, int columns, int lane,
                                            const S (&sums)[NB]) {
    constexpr int ROW = kStoreRow<T, NB>, CH = 32 * NB * (int)sizeof(T) / 16;
    asm volatile("" ::: "memory");
    char* p = at + (lane & 31) * ROW + (lane >> 5) * 4 * (int)sizeof(T);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const f32x16 c = sums[nb].all();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 v = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
            char* to = p + (32 * nb + 8 * g) * (int)sizeof(T);
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<u32x2*>(to) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
            else
                *reinterpret_cast<f32x4*>(to) = v;
        }
    }
    asm volatile("" ::: "memory");   // a wave's own accesses to shared memory stay in order
#pragma unroll
    for (int i = 0; i < 32 * CH / 64; ++i) {
        const int u = 64 * i + lane, r = u / CH, k = u % CH;
        const u32x4 v = *reinterpret_cast<const u32x4*>(at + r * ROW + 16 * k);
        if (r < rows && k * kVec<T> < columns) *reinterpret_cast<u32x4*>(out + r * stride + k * kVec<T>) = v;
    }
    asm volatile("" ::: "memory");
}

}  // namespace product
}  // namespace wtc
