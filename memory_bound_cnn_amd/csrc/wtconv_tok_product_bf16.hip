// The experts' products for bfloat16.
#include <hip/hip_runtime.h>

#include "wtc_tok_product_launch.h"

namespace wtc {
namespace product {

int rows_bf16(const Args& a, bool back, hipStream_t st) { return run_rows<uint16_t>(a, back, st); }
int weights_bf16(const Args& a, bool large, hipStream_t st) { return run_weights<uint16_t>(a, large, st); }

}  // namespace product
}  // namespace wtc
