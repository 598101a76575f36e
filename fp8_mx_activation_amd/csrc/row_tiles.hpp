// How many tiles an expert's rows make: plain C++, for kernels and host tests.
#pragma once

#include <stdint.h>

namespace mxq {

constexpr int kAllRows = 0;  // in the place of a tile's rows: one tile of all

// Up to 2^31 - 2^16 rows (MXQ_MAX_MATMUL_ROWS) and 2^15 rows a tile the sum
// stays within 32 bits; one tile of all rows must not be a sum with a large TM.
template <int TM>
constexpr int32_t row_tiles(int32_t count) {
  static_assert(TM >= 0 && TM <= (1 << 15), "the sum fits 32 bits");
  if constexpr (TM == kAllRows)
    return count > 0 ? 1 : 0;
  else
    return (count + TM - 1) / TM;
}

}  // namespace mxq
