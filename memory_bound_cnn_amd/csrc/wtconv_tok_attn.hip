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
}  // namespace
}  // namespace attn

int launch_attn_forward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const int* cu, void* out,
                        float* lse, void* stream) {
    attn::Args a = attn::args_of(d, q, k, v, cu);
    a.out = out;
    a.lse = lse;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? attn::fwd_bf16(a, st) : attn::fwd_fp32(a, st);
}

int launch_attn_backward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const void* out,
                         const float* lse, const void* dout, const int* cu, void* dq, void* dk, void* dv,
                         float* delta, void* stream) {
    attn::Args a = attn::args_of(d, q, k, v, cu);
    a.o = out;
    a.g = dout;
    a.lse = const_cast<float*>(lse);
    a.delta = delta;
    a.dq = dq; a.dk = dk; a.dv = dv;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return d->dtype == WTC_BF16 ? attn::bwd_bf16(a, st) : attn::bwd_fp32(a, st);
}

}  // namespace wtc
