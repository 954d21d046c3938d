// Attention kernels for bfloat16 activations: one instance for each multiple of 32 channels of
// a head (heads of 8, 16, .. channels take the next one, their missing terms zero).
#include "wtconv_tok_attn_bwd.h"
#include "wtconv_tok_attn_fwd.h"

namespace wtc {
namespace attn {

int fwd_bf16(const Args& a, hipStream_t st) {
    if (a.D <= 32) return run_fwd<uint16_t, 32>(a, st);
    if (a.D <= 64) return run_fwd<uint16_t, 64>(a, st);
    if (a.D <= 96) return run_fwd<uint16_t, 96>(a, st);
    return run_fwd<uint16_t, 128>(a, st);
}

int bwd_bf16(const Args& a, hipStream_t st) {
    if (a.D <= 32) return run_bwd<uint16_t, 32>(a, st);
    if (a.D <= 64) return run_bwd<uint16_t, 64>(a, st);
    if (a.D <= 96) return run_bwd<uint16_t, 96>(a, st);
    return run_bwd<uint16_t, 128>(a, st);
}

}  // namespace attn
}  // namespace wtc
