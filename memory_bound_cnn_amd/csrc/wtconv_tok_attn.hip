// Launchers of the attention kernels: arguments and the storage type.
#include "wtc_tok_attn.h"

namespace wtc {
namespace attn {

int fwd_bf16(const Args& a, hipStream_t st);
int fwd_fp32(const Args& a, hipStream_t st);
int bwd_bf16(const Args& a, hipStream_t st);
int bwd_fp32(const Args& a, hipStream_t st);

namespace {
Args args_of(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const int* cu) {
    Args a = {};
    a.q = q; a.k = k; a.v = v; a.cu = cu;
    a.T = (int)d->T; a.n_seq = d->n_seq; a.Hq = d->Hq; a.Hk = d->Hk; a.group = d->Hq / d->Hk; a.D = d->D;
    a.causal = d->causal; a.scale = d->scale;
    a.sq = d->q; a.sk = d->k; a.sv = d->v; a.so = d->o; a.sg = d->g; a.sdq = d->dq; a.sdk = d->dk; a.sdv = d->dv;
    return a;
}

// Splits of a key tile's queries.  With few key tiles (few heads of k and v, a
// short pack), or causal ones, whose first have twice the mean tile's queries,
// one workgroup a tile leaves most of the chip waiting for the longest: several
// share it where there are fewer than kWanted tiles (twice as many causal
// ones: 512 workgroups run at once), with kLeast query tiles each at the pack's
// mean length.  Their sums cost 8 bytes written and read a channel and split.
// Measured, dk and dv with their join: causal 3 sequences of 3500 to 8192
// tokens, 16 heads on 4 of 128 channels (552 tiles), 843 us in 4, 795 in 2;
// causal 4 of 2000 to 4096, 8 heads of 96 (800 tiles), 164 us whole, 198 in 2;
// float32 32 of 196, 6 heads on 3 of 64 (192 tiles), 56 us whole, 53 in 2, 60
// in 3.
constexpr int kWanted = 512, kWantedCausal = 1100, kLeast = 6, kMostSplits = 16;
int dkv_splits(const wtc_attn_desc* d) {
    if (d->T == 0 || d->n_seq == 0) return 1;
    const long long mean = (d->T + d->n_seq - 1) / d->n_seq, rows = d->dtype == WTC_BF16 ? 64 : 32;
    const long long tiles = (mean + 127) / 128 * d->n_seq * d->Hk, wanted = d->causal ? kWantedCausal : kWanted;
    const long long steps = (mean + rows - 1) / rows * (d->Hq / d->Hk) / (d->causal ? 2 : 1);
    long long s = (wanted + tiles / 2) / tiles;
    if (s > steps / kLeast) s = steps / kLeast;
    return (int)(s < 1 ? 1 : s > kMostSplits ? kMostSplits : s);
}
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t delta_bytes(const wtc_attn_desc* d) { return align256((size_t)d->Hq * (size_t)d->T * sizeof(float)); }
}  // namespace
}  // namespace attn

size_t attn_backward_bytes(const wtc_attn_desc* d) {
    const int s = attn::dkv_splits(d);
    return attn::delta_bytes(d) + (s > 1 ? sizeof(float) * 2 * s * (size_t)d->T * d->Hk * d->D : 0);
}

int launch_attn_forward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const int* cu, void* out,
                        float* lse, void* out_low, void* stream) {
    attn::Args a = attn::args_of(d, q, k, v, cu);
    a.out = out;
    a.lse = lse;
    a.low = out_low;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? attn::fwd_bf16(a, st) : attn::fwd_fp32(a, st);
}

int launch_attn_backward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const void* out,
                         const float* lse, const void* out_low, const void* dout, const int* cu, void* dq, void* dk, void* dv,
                         void* workspace, void* stream) {
    attn::Args a = attn::args_of(d, q, k, v, cu);
    a.o = out;
    a.g = dout;
    a.low = const_cast<void*>(out_low);
    a.lse = const_cast<float*>(lse);
    a.delta = static_cast<float*>(workspace);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + attn::delta_bytes(d));
    a.splits = attn::dkv_splits(d);
    a.dq = dq; a.dk = dk; a.dv = dv;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? attn::bwd_bf16(a, st) : attn::bwd_fp32(a, st);
}

}  // namespace wtc
