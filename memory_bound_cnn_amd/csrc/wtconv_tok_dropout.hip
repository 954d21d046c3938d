// Dropout with the residual's addition and no stored mask:
//   y[i] = r[i] + (bits[i] >= least ? x[i] 65536 / (65536 - least) : 0).
//
// bits[i] comes from the counter-based generator Philox 4x32-10 (Salmon et
// al., 2011): one counter gives 128 bits, which serve eight elements of 16
// bits each, one 16-byte vector of bfloat16.  Ten rounds are 20 products of
// 32 x 32 bits, which run at a quarter of the vector rate: with 32 bits for
// each element they alone would take longer than the 6 bytes an element moves
// (bfloat16 with a residual).  The bound is device memory, 3 N e bytes with a
// residual and 2 N e without.  Means of 20 training steps: 100663296 bfloat16 109
// and 76 us (5.5 and 5.3 TB/s), 50331648 float32 114 and 69 (5.3 and 5.9).
#include <hip/hip_runtime.h>

#include "wtc_tok_device.h"
#include "wtc_tok_internal.h"

namespace wtc {
namespace {

constexpr int kGroup = 8;   // elements of one counter

struct Words {
    uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t block, uint64_t offset, uint64_t seed) {
    Words c = {{(uint32_t)block, (uint32_t)(block >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)}};
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)c.w[0] * 0xD2511F53u, q = (uint64_t)c.w[2] * 0xCD9E8D57u;
        c = {{(uint32_t)(q >> 32) ^ c.w[1] ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ c.w[3] ^ k1, (uint32_t)p}};
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

template <typename T, bool RES>
__global__ void __launch_bounds__(256) k_dropout(long long n, uint32_t least, float scale, const T* x, const T* r,
                                                 const unsigned long long* rng, T* y) {
    constexpr int V = kVec<T>;
    const uint64_t seed = rng[0], offset = rng[1];
    const long long groups = (n + kGroup - 1) / kGroup, step = (long long)gridDim.x * 256;
    for (long long g = (long long)blockIdx.x * 256 + threadIdx.x; g < groups; g += step) {
        const long long i0 = g * kGroup;
        const int left = (int)min((long long)kGroup, n - i0);
        float v[kGroup / V][V], res[kGroup / V][V];
#pragma unroll
        for (int k = 0; k < kGroup / V; ++k) {
            load_part(x + i0 + k * V, left - k * V, v[k]);
            if constexpr (RES) load_part(r + i0 + k * V, left - k * V, res[k]);
        }
        const Words b = philox((uint64_t)g, offset, seed);
#pragma unroll
        for (int k = 0; k < kGroup / V; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = k * V + j;
                const uint32_t bits = (b.w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                const float kept = bits >= least ? v[k][j] * scale : 0.f;
                v[k][j] = RES ? kept + res[k][j] : kept;
            }
            store_part(y + i0 + k * V, left - k * V, v[k]);
        }
    }
}

template <typename T>
void dropout_t(long long n, unsigned least, const void* x, const void* r, const unsigned long long* rng, void* y,
               hipStream_t st) {
    // one counter a thread, up to a launch of 2^31 threads; fewer that go on to the next (100663296 bfloat16
    // with a residual and without) take 109 and 72.5 us with 8192 workgroups, 103 and 69.5 so
    const long long blocks = (n + 256 * kGroup - 1) / (256 * kGroup), cap = 1 << 23;
    const dim3 grid((unsigned)(blocks < cap ? blocks : cap)), block(256);
    const float scale = least < 65536u ? 65536.f / (float)(65536u - least) : 0.f;
    const T *xp = static_cast<const T*>(x), *rp = static_cast<const T*>(r);
    if (r)
        hipLaunchKernelGGL((k_dropout<T, true>), grid, block, 0, st, n, least, scale, xp, rp, rng, static_cast<T*>(y));
    else
        hipLaunchKernelGGL((k_dropout<T, false>), grid, block, 0, st, n, least, scale, xp, rp, rng, static_cast<T*>(y));
}

}  // namespace

int launch_dropout(long long n, int dtype, unsigned least, const void* x, const void* r,
                   const unsigned long long* rng, void* y, void* stream) {
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (dtype == WTC_BF16)
        dropout_t<uint16_t>(n, least, x, r, rng, y, st);
    else
        dropout_t<float>(n, least, x, r, rng, y, st);
    return hipGetLastError() == hipSuccess ? WTC_OK : WTC_EHIP;
}

}  // namespace wtc
