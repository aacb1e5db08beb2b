// row_grid.cuh -- how many CTAs (clusters, teams' CTAs) a norm kernel's rows
// are spread over.  Host arithmetic only: plain C++, no CUDA headers.
#pragma once

#include <cstdint>

namespace hq {

// One unit a row while `most` units run at the same time, else as many as
// that, rounded down to whole steps of `apart`: unit u takes rows u, u + grid,
// ..., and with rows that start between 16-byte boundaries those must lie a
// multiple of `apart` rows apart.  `apart` units at least where the device (or
// the share of it that the process may use) runs fewer at once: units do not
// wait for one another, the rest run after the first.  Never more units than
// rows: each writes its own partial row.
inline int64_t row_grid(int64_t rows, int64_t most, int64_t apart) {
  if (most < apart) most = apart;
  return rows <= most ? rows : most / apart * apart;
}

}  // namespace hq
