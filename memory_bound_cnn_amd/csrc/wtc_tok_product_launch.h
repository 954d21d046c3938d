// What the experts' products' launches pass on to the files of each type.
#pragma once

#include "wtc_tok_product_kernels.h"

namespace wtc {
namespace product {

int rows_bf16(const Args& a, bool back, hipStream_t st);
int rows_fp32(const Args& a, bool back, hipStream_t st);
int weights_bf16(const Args& a, bool large, hipStream_t st);
int weights_fp32(const Args& a, bool large, hipStream_t st);

}  // namespace product
}  // namespace wtc
