// ragged.cuh — rows of a ragged batch: which sequence a packed row belongs to, and where.
//
// Sequence b owns rows [row_start[b], row_start[b+1]) and they are its last positions.
#pragma once
#include "common.cuh"

namespace hs2 {

// n[k] = number of entries of row_start[0 .. batch] that are <= r0 + k, by one warp: every
// lane gets all of them. One round of independent loads per 32 entries (a binary search
// would chain its loads).
template <int TOK>
HS2_DEVI void warp_rows_at_most(const int32_t* row_start, int batch, int r0, int (&n)[TOK]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < TOK; ++k) n[k] = 0;
  for (int j = lane; j <= batch; j += 32) {
    const int v = row_start[j];
#pragma unroll
    for (int k = 0; k < TOK; ++k) n[k] += v <= r0 + k;
  }
#pragma unroll
  for (int k = 0; k < TOK; ++k) n[k] = __reduce_add_sync(0xffffffffu, n[k]);
}

struct RowPlace {
  int b;    // sequence, or -1: the row is outside every sequence
  int pos;  // its position; -1: the sequence's length or rows are out of range
};
// Place of row r given n_le, the number of row_start entries <= r: the last sequence that starts at or
// before r owns it (those before it that start there too have no rows).
HS2_DEVI RowPlace row_place(const int32_t* row_start, const int32_t* seq_len, int batch, int max_pages, int r, int n_le) {
  RowPlace p{n_le - 1, -1};
  if (p.b < 0 || p.b >= batch) {
    p.b = -1;
    return p;
  }
  const int r0 = row_start[p.b], n = row_start[p.b + 1] - r0, t = seq_len[p.b];
  if (r < r0 || n <= 0 || (uint32_t)(r - r0) >= (uint32_t)n) return p;  // a descending row_start
  if (t >= n && t <= max_pages * kPage) p.pos = t - n + (r - r0);
  return p;
}

}  // namespace hs2
