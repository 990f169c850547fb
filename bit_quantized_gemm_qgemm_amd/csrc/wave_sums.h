// Sums over the lanes of a wave by moves between lanes (VALU; a shuffle through LDS
// takes several times as long).
#pragma once

#include "qgemm_common.h"

namespace qgemm {
namespace {

// x of the lane that a DPP control names, 0 where it names none or the row is
// masked out.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int moved_int(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}

// Inclusive sums: by shifts of 1, 2, 4 and 8 within a row of 16, then the last lane
// of a row to the next one (rows 1 and 3) and lane 31 to the upper half.
__device__ __forceinline__ int int_sums_of_wave(int x) {
  x += moved_int<0x111>(x);
  x += moved_int<0x112>(x);
  x += moved_int<0x114>(x);
  x += moved_int<0x118>(x);
  x += moved_int<0x142, 0xa>(x);
  x += moved_int<0x143, 0xc>(x);
  return x;
}

}  // namespace
}  // namespace qgemm
