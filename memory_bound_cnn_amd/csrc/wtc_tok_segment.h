// Tiles of an expert's rows: shared by the kernels of the products and the CPU
// tests, which compile it on the host.
#pragma once

#include "wtc_numeric.h"

namespace wtc {
namespace product {

// The rows of a tile: at most a tile's number of one expert's, or of no expert's (before the first's, after the last's).
struct Rows {
    int expert;   // -1: rows of none
    int start, count;
};
// Tile number `tile` of rows b .. e - 1, 0 <= b and e < 2^31 in any order; count = 0 if there is none of that number.
// With bounds in no order the number may be that of any other segment's, and its first row beyond 2^31.
template <int SIZE>
WTC_HD Rows rows_of(int expert, int b, int e, int tile) {
    if (tile < 0 || tile > (e - b) / SIZE || e <= b) return {expert, b, 0};
    const int start = tile * SIZE, left = e - b - start;
    return {expert, b + start, left < SIZE ? left : SIZE};
}

}  // namespace product
}  // namespace wtc
