// Tables of a rotation (see rotary.cu) and the checks shared by the calls on pages.
#pragma once

#include <stdint.h>

#include "../../include/evict.h"

namespace evict {

struct RotaryTable {
  alignas(16) uint64_t freq[EVICT_HEAD_DIM / 2];   // turns per position, as a fraction of 2^64
  alignas(8) uint8_t axis[EVICT_HEAD_DIM / 2];
  int half;                            // pairs that turn
  int adjacent;
  int n_axes;
  float scale;
};

int check_pages(const evict_pages* pages);
// Two of a tensor's batch x heads x m rows share an element: no output may have that.
bool rows_overlap(const evict_rows& x, int batch, int m);

}  // namespace evict

struct evict_rotary {
  evict::RotaryTable t;
};
