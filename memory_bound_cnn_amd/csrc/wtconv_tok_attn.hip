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

// Splits of a tile's other side.  With few tiles (few heads, a short pack), or
// causal ones, whose longest have twice the mean tile's work, one workgroup a
// tile leaves most of the chip waiting for the longest: several share it, as
// many as keep their number within `wanted`, with kLeast tiles of the other side
// each at the pack's mean length.  Partial results cost 8 bytes written and read
// a channel and split.  Measured, with the joins, bfloat16, whole and split:
//   8192 tokens, 1 head of 64 (64 tiles): forward 112 us, 39 in 8; dq 129, 48
//   2 x 2000..2048, 6 of 64 (192 tiles): forward 35.3 us, 32.9 in 2; dq 41.5, 41.8
//   3 x 1024, 12 of 64 (288 tiles): forward 26.2 us, 30.9 in 2; dq 34.6, 39.4
//   causal 2 x 3100, 8 on 2 of 64 (400 tiles): forward 52 us, 45 in 2; dq 63, 53
//   causal 4096, 16 of 128 (512 tiles): forward 103 us, 104 in 2; dq 134, 148
//   causal 3 x 3500..8192, 16 on 4 of 128 (552 key tiles): dk and dv 843 us in 4, 795 in 2
//   causal 4 x 2000..4096, 8 of 96 (800 key tiles): dk and dv 164 us, 198 in 2
// Around kWantedCausalKeys (split in 2 up to 575 key tiles), the backward pass:
//   causal 8192, 9 to 12 of 128 (576, 640, 704, 768): 605, 633, 663, 688 us, 584, 624, 681, 720 in 2
//   causal 4 x 3000, 6 and 7 of 96 (576, 672): 188, 199 us, 207, 229 in 2
//   causal 8 x 2048, 5 of 64 (640): 111 us, 131 in 2; 4 x 4096, 5 of 64 (640): 204, 204
// The lengths themselves are on the device: the rule knows their mean, with empty
// sequences counted.  One of 8192 tokens and one head takes 43 us forward and 95
// backward alone, but 113 and 331 beside 63 empty ones, 15 of one token or 61 of
// 64, where it is not split.
constexpr int kWanted = 512, kWantedCausal = 820, kWantedCausalKeys = 1150, kLeast = 6, kMostSplits = 16;
int splits_of(const wtc_attn_desc* d, int wanted, int heads, int together) {
    if (d->T == 0 || d->n_seq == 0) return 1;
    const long long mean = (d->T + d->n_seq - 1) / d->n_seq, rows = d->dtype == WTC_BF16 ? 64 : 32;
    const long long tiles = (mean + 127) / 128 * d->n_seq * heads;
    const long long steps = (mean + rows - 1) / rows * together / (d->causal ? 2 : 1);
    const long long s = wanted / tiles < steps / kLeast ? wanted / tiles : steps / kLeast;
    return (int)(s < 1 ? 1 : s > kMostSplits ? kMostSplits : s);
}
// of a query tile's keys (forward, dq)
int query_splits(const wtc_attn_desc* d) { return splits_of(d, d->causal ? kWantedCausal : kWanted, d->Hq, 1); }
// of a key tile's queries, the heads' of its group (dk, dv)
int key_splits(const wtc_attn_desc* d) {
    return splits_of(d, d->causal ? kWantedCausalKeys : kWanted, d->Hk, d->Hq / d->Hk);
}
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t row_floats(const wtc_attn_desc* d) { return align256((size_t)d->Hq * (size_t)d->T * sizeof(float)); }
size_t part_bytes(const wtc_attn_desc* d, int splits, int heads) {
    return splits > 1 ? sizeof(float) * splits * (size_t)d->T * heads * d->D : 0;
}
}  // namespace
}  // namespace attn

// the splits' outputs, and the maximum and the sum of their rows
size_t attn_forward_bytes(const wtc_attn_desc* d) {
    const int s = attn::query_splits(d);
    return s > 1 ? 2 * s * attn::row_floats(d) + attn::part_bytes(d, s, d->Hq) : 0;
}
// delta, then the splits' sums of dq, whose place those of dk and dv take afterwards
size_t attn_backward_bytes(const wtc_attn_desc* d) {
    const size_t q = attn::part_bytes(d, attn::query_splits(d), d->Hq);
    const size_t kv = 2 * attn::part_bytes(d, attn::key_splits(d), d->Hk);
    return attn::row_floats(d) + (q > kv ? q : kv);
}

int launch_attn_forward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const int* cu, void* out,
                        float* lse, void* out_low, void* workspace, void* stream) {
    attn::Args a = attn::args_of(d, q, k, v, cu);
    a.out = out;
    a.lse = lse;
    a.low = out_low;
    a.q_splits = attn::query_splits(d);
    a.row_floats = (long long)(attn::row_floats(d) / sizeof(float));
    a.stat = static_cast<float*>(workspace);
    a.parts = a.stat + (workspace ? 2 * a.q_splits * a.row_floats : 0);
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
    a.parts = a.delta + attn::row_floats(d) / sizeof(float);
    a.q_splits = attn::query_splits(d);
    a.k_splits = attn::key_splits(d);
    a.dq = dq; a.dk = dk; a.dv = dv;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? attn::bwd_bf16(a, st) : attn::bwd_fp32(a, st);
}

}  // namespace wtc
