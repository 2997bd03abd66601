// ragged.cuh — rows of a ragged batch: which sequence a packed row belongs to, and where.
//
// Sequence b owns rows [row_start[b], row_start[b+1]) and they are its last positions.
#pragma once
#include "common.cuh"

namespace hs2 {

// Whether any sequence's rows are not within [0, n_rows), or a start falls, by one warp: what the
// rows themselves cannot see, where no row of theirs exists.
HS2_DEVI bool warp_bad_starts(const int32_t* row_start, int batch, int n_rows) {
  bool bad = false;
  for (int b = threadIdx.x & 31; b < batch; b += 32) {
    const int r0 = row_start[b], r1 = row_start[b + 1];
    bad |= r1 != r0 && (r1 < r0 || r0 < 0 || r1 > n_rows);
  }
  return __any_sync(0xffffffffu, bad);
}

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
HS2_DEVI RowPlace row_place(const int32_t* row_start, const int32_t* seq_len, int batch, int max_pages, int n_rows,
                            int r, int n_le) {
  RowPlace p{n_le - 1, -1};
  if (p.b < 0 || p.b >= batch) {
    p.b = -1;
    return p;
  }
  const int r0 = row_start[p.b], r1 = row_start[p.b + 1], t = seq_len[p.b];
  if (r0 < 0 || r1 > n_rows) return p;  // rows that do not exist
  if (r < r0 || r >= r1) return p;      // a descending row_start
  const int n = r1 - r0;
  if (t >= n && t <= (long long)max_pages * kPage) p.pos = t - n + (r - r0);
  return p;
}

}  // namespace hs2
