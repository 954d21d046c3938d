// Rows held in the registers of a group of lanes, for the norms: the groups'
// shapes, their sums, and the join of the rows' partial sums of a parameter's
// gradient.
#pragma once

#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace {

// Sum (or maximum) over the G lanes of a row; every lane gets it.  `red`: one
// float per wave for groups wider than a wave (all threads of the workgroup
// call it together).
template <int G, bool MAX>
__device__ __forceinline__ float group_reduce(float v, float* red) {
#pragma unroll
    for (int o = 1; o < (G < 64 ? G : 64); o <<= 1) {
        const float other = __shfl_xor(v, o);
        v = MAX ? fmaxf(v, other) : v + other;
    }
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();   // the previous use of `red` is over
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < G / 64; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
    }
    return v;
}

// Parameters of channels c .. c + V - 1 of C, zero past the last one.
template <int V>
__device__ __forceinline__ void load_weight(const float* w, int C, int c, float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
        float part[4];
        load_part(w + c + k, C - c - k, part);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[k + j] = part[j];
    }
}

// The sums of n records' W floats, in a fixed order: 32 threads of a column take
// every 32nd record, then their sums are joined.  The first C go to dw, the others to db.
__global__ void __launch_bounds__(1024) k_row_join(const float* __restrict__ parts, int n, int W,
                                                   float* __restrict__ dw, int C, float* __restrict__ db) {
    __shared__ float sums[32][33];
    const int col = threadIdx.x & 31, part = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
    float v = 0.f;
    if (c < W) {
#pragma unroll 8
        for (int p = part; p < n; p += 32) v += parts[(size_t)p * W + c];
    }
    sums[part][col] = v;
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (part < o) sums[part][col] += sums[part + o][col];
        __syncthreads();
    }
    if (part == 0 && c < W) (c < C ? dw + c : db + (c - C))[0] = sums[0][col];
}

// The group of G lanes and the NV vectors per lane for a row of n 16-byte
// vectors: the first of these shapes, in the order of G * NV, that holds it.
// Where two have the same G * NV the wider group stands here (longer runs of
// consecutive addresses).  Those marked `many` leave no lane idle in rows of 24,
// 48 and 96 vectors, and are for forward passes of kManyVectors and more, as
// bfloat16 (without, with the residual): 65536 x 192 9.5 and 16.5 us, 11.4 and
// 17.0 without them, 25088 x 384 8.4 and 13.3, 9.9 and 13.4; but 49 x 768 4.0
// and 5.4, 3.7 and 4.5 without.  Around kManyVectors, 192 channels in a graph:
// 5461 rows (2^17 vectors) 3.8 and 5.2, 3.3 and 4.0 without, 8192 rows 3.5 and
// 4.6, 3.6 and 4.6, 10922 rows 4.1 and 5.8, 4.3 and 5.6, 21845 rows 5.3 and 8.5,
// 5.8 and 7.8, 87381 rows 11.9 and 24.7, 13.4 and 24.8: the two meet between 2^17
// and 2^18 without a residual, and with one do not differ by more than 0.8 us
// from there on.  Nor for the backward pass, whose registers they
// fill: 22.2 us, 18.2 without them, and 18.0, 15.2.
struct RowShape {
    int G, NV;
    bool many;
};
constexpr long long kManyVectors = 1 << 17;
constexpr RowShape kRowShapes[] = {{2, 1, false},    {4, 1, false},    {8, 1, false},   {16, 1, false}, {8, 3, true},
                                   {32, 1, false},   {16, 3, true},    {64, 1, false},  {32, 3, true},  {64, 2, false},
                                   {64, 3, false},   {64, 4, false},   {256, 2, false}, {256, 3, false}, {256, 4, false},
                                   {1024, 2, false}, {1024, 3, false}, {1024, 4, false}};
constexpr int kRowShapeCount = (int)(sizeof(kRowShapes) / sizeof(kRowShapes[0]));
static_assert(1024 * 4 * kVec<float> >= WTC_RMS_MAX_C && 1024 * 2 * kVec<uint16_t> >= WTC_RMS_MAX_C, "the longest row");

int row_shape(int C, int dtype, long long forward_rows) {
    const int V = dtype == WTC_BF16 ? kVec<uint16_t> : kVec<float>;
    const bool many = forward_rows * ((C + V - 1) / V) >= kManyVectors;
    int i = 0;
    while (kRowShapes[i].G * kRowShapes[i].NV * V < C || (kRowShapes[i].many && !many)) ++i;
    return i;
}

// f<T, G, NV>() for shape number `at`; shapes past the longest row of T are
// not compiled.
template <typename T, int I = 0, typename F>
void row_dispatch(int at, const F& f) {
    if (at == I) f.template operator()<T, kRowShapes[I].G, kRowShapes[I].NV>();
    if constexpr (I + 1 < kRowShapeCount)
        if constexpr (kRowShapes[I].G * kRowShapes[I].NV * kVec<T> < WTC_RMS_MAX_C) row_dispatch<T, I + 1>(at, f);
}

// Workgroups of a backward pass over rows, each with one record of its sums.
int row_parts(long long rows, int C, int dtype) {
    const int G = kRowShapes[row_shape(C, dtype, 0)].G, rpb = (G > 256 ? G : 256) / G;
    // a row to a workgroup: fewer, whose records of C floats are much of the traffic
    const long long blocks = (rows + rpb - 1) / rpb, most = G > 64 ? kRmsMaxParts / 2 : kRmsMaxParts;
    return (int)(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace wtc
