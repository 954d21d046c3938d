// The experts' products for float32.
#include <hip/hip_runtime.h>

#include "wtc_tok_product_launch.h"

namespace wtc {
namespace product {

int rows_fp32(const Args& a, bool back, hipStream_t st) { return run_rows<float>(a, back, st); }
int weights_fp32(const Args& a, bool large, hipStream_t st) { return run_weights<float>(a, large, st); }

}  // namespace product
}  // namespace wtc
