// Layout of a chunk plan (int32 words), shared by the host planner and the
// kernels:
//   [0] magic  [1] CTAs  [2] units  [3] joins
//   lists at 8:  first unit of every CTA's list, CTAs + 1 entries
//   units: 12 words  {q0, ntok, pos0, kvh,  kv0, t0, t1, twin,  part, 0, 0, 0}
//          query tokens q0.. of one request, at positions pos0.. in it; keys
//          [t0, t1) of the request, whose position 0 is flat position kv0;
//          part: first partial row, -1: the rows are final
//   joins: 8 words   {q0, rows, kvh, part, count, 0, 0, 0}
//          `count` partials of `rows` rows each, back to back from `part`
#pragma once

#include <stdint.h>

namespace psa {

constexpr int32_t kChunkMagic = 0x50534343;
constexpr int32_t kChunkTile = 128;  // keys per tile

struct ChunkPlanView {
  int64_t lists, units, joins, len;
#ifdef __CUDACC__
  __host__ __device__
#endif
  ChunkPlanView(int32_t n_ctas, int32_t n_units, int32_t n_joins) {
    lists = 8;
    units = (lists + n_ctas + 1 + 3) / 4 * 4;
    joins = units + 12 * int64_t(n_units);
    len = joins + 8 * int64_t(n_joins);
  }
};

}  // namespace psa
