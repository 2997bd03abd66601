// pages.cu — the books of a page pool: growing, freeing and forking sequences, compaction.
//
// A pool's pages are numbered alike in every cache that shares its block table. The books are
// a reference count per page and a stack of free pages. What a call takes or returns is
// decided by prefix sums in a fixed order (sequence, then entry; or page), never by the order
// in which atomics land, so tables, counts and stack are the same on every run.
//
// Bound by latency: the books of a pool of 10^4..10^5 pages are a few hundred KB, so a call
// is one or two short launches with few dependent rounds of loads, and every launch overlaps
// the end of the one before it (programmatic dependent launch). Only the copies (a forked
// sequence's partial page, the pages that compaction moves) are bandwidth.
// Measured: fork, grow and free of 64 branches of 16 sequences (4K to 16K keys, two caches) 19 us together,
// of 8 branches 14; compaction that moves half of what is left of 64 sequences (540 MB read and
// written) 101 us, 0.80 of the copy bandwidth.
#include <cooperative_groups.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "kernels.h"

namespace hs2 {

namespace cg = cooperative_groups;

namespace {

constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;  // CTAs of the clusters that scan all pages
constexpr int kGone = -(1 << 30);  // ref of a page whose last reference the running free call took

HS2_DEVI int pages_of(int t) { return (t + kPage - 1) / kPage; }
HS2_DEVI bool good_len(int t, int max_pages) { return t >= 0 && t <= max_pages * kPage; }

}  // namespace

// ---------------------------------------------------------------------------- grow
// One block. Sequences in chunks of 1024: a prefix sum of the pages each needs, then a warp
// per sequence writes its entries. A batch of one chunk is summed once.
__global__ void __launch_bounds__(kPagesThreads) pages_grow_kernel(const PagesArgs a) {
  __shared__ int sums[33], base[kPagesThreads], need_s[kPagesThreads], from[kPagesThreads];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nf = *a.n_free;
  int old = 0, add = 0;  // this thread's sequence of the chunk
  auto need_of = [&](int b, bool flag) -> int {
    if (b >= a.batch) return -1;
    old = a.seq_len[b], add = a.n_new[b];
    if (add < 0 || !good_len(old, a.max_pages) || add > a.max_pages * kPage - old) {
      if (flag) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      return -1;
    }
    return pages_of(old + add) - pages_of(old);
  };
  long long all = 0;
  int need = -1, at = 0, total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPagesThreads) {
    need = need_of(b0 + threadIdx.x, true);
    at = block_prefix(max(need, 0), sums, total);
    all += total;
  }
  if (nf < 0 || nf > a.num_pages || all > nf) {
    if (threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    return;
  }
  int taken = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPagesThreads) {
    if (a.batch > kPagesThreads) {
      need = need_of(b0 + threadIdx.x, false);
      at = block_prefix(max(need, 0), sums, total);
    }
    base[threadIdx.x] = taken + at;
    need_s[threadIdx.x] = need;
    from[threadIdx.x] = pages_of(old);
    if (need >= 0) a.seq_len[b0 + threadIdx.x] = old + add;
    __syncthreads();
    const int nb = min(kPagesThreads, a.batch - b0);
    for (int i = warp; i < nb; i += kPagesThreads / 32)
      for (int j = lane; j < need_s[i]; j += 32) {
        const int page = a.free_list[nf - 1 - base[i] - j];
        a.bt[(size_t)(b0 + i) * a.max_pages + from[i] + j] = page;
        if (page >= 0 && page < a.num_pages) a.ref[page] = 1;
        else flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
      }
    taken += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.n_free = nf - taken;
}

cudaError_t launch_pages_grow(const PagesArgs& a, cudaStream_t s) {
  return launch_pdl(pages_grow_kernel, dim3(1), dim3(kPagesThreads), 0, s, a);
}

// ---------------------------------------------------------------------------- free
// One cluster. Every entry takes a reference down; the one that took a page's last marks the page by
// an addition, and one that found none left (a bad table) gives it back: additions commute, so
// the counts come out the same in any order. (By compare-and-swap the branches of a page retried
// against each other: 24 us for 64 branches of 64 to 256 pages, four to a page, now 9.) Then each block
// counts and pushes its slice of the marked pages, in page order. A warp takes 128 entries of a
// row at a time, four a lane, so that their atomics are in flight together.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)
    pages_free_kernel(const PagesArgs a) {
  constexpr int E = 4;
  __shared__ int sums[33], found;
  cg::cluster_group cl = cg::this_cluster();
  griddep_launch_dependents();
  griddep_wait();
  const int rank = (int)cl.block_rank();
  const int nf = *a.n_free;
  const int warp = rank * (kPagesThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int per_row = (a.max_pages + 32 * E - 1) / (32 * E);
  for (long long item = warp; item < (long long)a.batch * per_row; item += kPagesCluster * (kPagesThreads / 32)) {
    const int b = (int)(item / per_row), j0 = (int)(item % per_row) * 32 * E + lane;
    if (a.drop[b] == 0) continue;
    const int t = a.seq_len[b];
    if (!good_len(t, a.max_pages)) {
      if (lane == 0 && item % per_row == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      continue;
    }
    const int np = pages_of(t);
    int page[E], was[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = j0 + 32 * e;
      page[e] = j < np ? a.bt[(size_t)b * a.max_pages + j] : -1;
      if (j < np && (page[e] < 0 || page[e] >= a.num_pages)) {
        flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        page[e] = -1;
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) was[e] = page[e] >= 0 ? atomicSub(&a.ref[page[e]], 1) : 2;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (was[e] == 1) {
        atomicAdd(&a.ref[page[e]], kGone);
      } else if (was[e] <= 0) {
        atomicAdd(&a.ref[page[e]], 1);
        flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
      }
    }
  }
  cl.sync();
  const int per = (a.num_pages + kPagesCluster - 1) / kPagesCluster;
  const int p0 = min(a.num_pages, rank * per), p1 = min(a.num_pages, p0 + per);
  int mine = 0, total;
  for (int p = p0 + threadIdx.x; p < p1; p += kPagesThreads) mine += __ldcg(&a.ref[p]) == kGone;
  (void)block_prefix(mine, sums, total);
  if (threadIdx.x == 0) found = total;
  cl.sync();
  int at = nf, all = 0;
  for (int k = 0; k < kPagesCluster; ++k) {
    const int f = *cl.map_shared_rank(&found, k);
    if (k < rank) at += f;
    all += f;
  }
  for (int c0 = p0; c0 < p1 && total > 0; c0 += kPagesThreads) {
    const int p = c0 + threadIdx.x;
    const bool gone = p < p1 && __ldcg(&a.ref[p]) == kGone;
    int here;
    const int i = at + block_prefix(gone, sums, here);
    if (gone) {
      a.ref[p] = 0;
      if (i >= 0 && i < a.num_pages) a.free_list[i] = p;
      else flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    }
    at += here;
  }
  if (rank == 0 && threadIdx.x == 0) *a.n_free = min(nf + all, a.num_pages);
  cl.sync();  // no block leaves while its count may be read
}

cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t s) {
  return launch_pdl(pages_free_kernel, dim3(kPagesCluster), dim3(kPagesThreads), 0, s, a);
}

// ---------------------------------------------------------------------------- fork
// First launch, one block: lengths, and the page of its own that a branch's partial page takes
// (at its entry of the branch's table, -1 where it takes none).
__global__ void __launch_bounds__(kPagesThreads) pages_fork_plan_kernel(const PagesArgs a) {
  __shared__ int sums[33];
  griddep_launch_dependents();
  griddep_wait();
  const int nf = *a.n_free;
  auto len_of = [&](int c, bool flag) -> int {
    if (c >= a.n_child) return 0;
    const int p = a.src[c];
    if (p < -1 || p >= a.batch) {
      if (flag) flag_error(a.dev_err, HS2_DEV_BAD_INDEX);
      return 0;
    }
    if (p < 0) return 0;
    const int t = a.seq_len[p];
    if (!good_len(t, a.max_pages)) {
      if (flag) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      return 0;
    }
    return t;
  };
  int all = 0, total = 0, len = 0, at = 0;
  for (int c0 = 0; c0 < a.n_child; c0 += kPagesThreads) {
    len = len_of(c0 + threadIdx.x, true);
    at = block_prefix(len % kPage != 0, sums, total);
    all += total;
  }
  const bool fits = nf >= 0 && nf <= a.num_pages && all <= nf;
  if (!fits && threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
  int taken = 0;
  for (int c0 = 0; c0 < a.n_child; c0 += kPagesThreads) {
    const int c = c0 + threadIdx.x;
    if (a.n_child > kPagesThreads) {  // else the sum above was this chunk's
      len = len_of(c, false);
      at = block_prefix(len % kPage != 0, sums, total);
    }
    const int t = fits ? len : 0, i = taken + at;
    const bool own = t % kPage != 0;
    if (c < a.n_child) {
      a.child_len[c] = t;
      if (own) {
        const int page = a.free_list[nf - 1 - i];
        const bool ok = page >= 0 && page < a.num_pages;
        if (ok) a.ref[page] = 1;
        else flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        a.child_table[(size_t)c * a.max_pages + t / kPage] = ok ? page : -1;
      }
    }
    taken += total;
  }
  if (threadIdx.x == 0 && fits && taken > 0) *a.n_free = nf - taken;
}

// Second launch, grid (branches, slabs of a page): the rest of the branch's table (slab 0) and
// the filled rows of the source's last page.
__global__ void __launch_bounds__(256) pages_fork_copy_kernel(const PagesArgs a, const PageSlabs sl) {
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x, p = a.src[c], t = a.child_len[c];
  const int full = t / kPage, rest = t % kPage;
  int32_t* child = a.child_table + (size_t)c * a.max_pages;
  const int32_t* par = a.bt + (size_t)max(p, 0) * a.max_pages;
  int slab = blockIdx.y;
  if (slab == 0) {
    for (int j = threadIdx.x; j < a.max_pages; j += blockDim.x) {
      if (j == full && rest > 0) continue;
      int page = -1;
      if (j < full) {
        page = par[j];
        if (page < 0 || page >= a.num_pages || __ldcg(&a.ref[page]) <= 0) {  // out of range, or a free page
          flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
          page = -1;
        } else {
          atomicAdd(&a.ref[page], 1);
        }
      }
      child[j] = page;
    }
  }
  if (rest == 0) return;
  const int to = child[full], of = par[full];
  if (to < 0) return;  // flagged by the plan
  if (of < 0 || of >= a.num_pages || __ldcg(&a.ref[of]) <= 0) {  // as above
    if (slab == 0 && threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    return;
  }
  int k = 0;
  while (k < sl.n && slab >= sl.Hkv[k]) slab -= sl.Hkv[k++];
  if (k >= sl.n) return;
  const PageSlab s = sl.s[k];
  const uint8_t* from = s.base + ((size_t)of * sl.Hkv[k] + slab) * s.slab_bytes;
  uint8_t* dst = s.base + ((size_t)to * sl.Hkv[k] + slab) * s.slab_bytes;
  const int bytes = s.row_bytes ? rest * s.row_bytes : (int)s.slab_bytes;  // a multiple of 4
  const int vec = bytes / 16;
  if (((uintptr_t)from & 15) == 0 && ((uintptr_t)dst & 15) == 0) {
    for (int i = threadIdx.x; i < vec; i += blockDim.x)
      reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(from)[i];
    for (int i = vec * 4 + threadIdx.x; i < bytes / 4; i += blockDim.x)
      reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(from)[i];
  } else {
    for (int i = threadIdx.x; i < bytes / 4; i += blockDim.x)
      reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(from)[i];
  }
}

cudaError_t launch_pages_fork(const PagesArgs& a, const PageSlabs& sl, cudaStream_t s) {
  const cudaError_t e = launch_pdl(pages_fork_plan_kernel, dim3(1), dim3(kPagesThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  int slabs = 0;
  for (int k = 0; k < sl.n; ++k) slabs += sl.Hkv[k];
  return launch_pdl(pages_fork_copy_kernel, dim3(a.n_child, slabs), dim3(256), 0, s, a, sl);
}

// ---------------------------------------------------------------------------- compact
// First launch, one cluster: every block takes a slice of the pages. From the blocks' counts of
// referenced pages come L and the ranks of its holes (free pages below L) and movers
// (referenced pages from L on); the i-th mover goes to the i-th hole. The lists, by page whether it is
// free (-1) and a mover's rank, and the free list are written; references and tables follow with the copies.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)
    pages_compact_plan_kernel(const PagesArgs a) {
  __shared__ int sums[33], live_s, hole_s, mover_s;
  cg::cluster_group cl = cg::this_cluster();
  griddep_launch_dependents();
  griddep_wait();
  const int rank = (int)cl.block_rank();
  const int per = (a.num_pages + kPagesCluster - 1) / kPagesCluster;
  const int p0 = min(a.num_pages, rank * per), p1 = min(a.num_pages, p0 + per);
  const int half = a.num_pages / 2;
  int32_t* src = a.moves + 4;
  int32_t* dst = src + half;
  int32_t* rank_of = dst + half;
  int mine = 0, total;
  for (int p = p0 + threadIdx.x; p < p1; p += kPagesThreads) mine += a.ref[p] > 0;
  (void)block_prefix(mine, sums, total);
  if (threadIdx.x == 0) live_s = total;
  cl.sync();
  int L = 0;
  for (int k = 0; k < kPagesCluster; ++k) L += *cl.map_shared_rank(&live_s, k);
  // the slice's pages below L, then those from L on
  const int cut = min(max(L, p0), p1);
  int below = 0;
  if (cut == p1) {
    below = total;
  } else if (cut > p0) {
    mine = 0;
    for (int p = p0 + threadIdx.x; p < cut; p += kPagesThreads) mine += a.ref[p] > 0;
    (void)block_prefix(mine, sums, below);
  }
  if (threadIdx.x == 0) hole_s = cut - p0 - below, mover_s = total - below;
  cl.sync();
  int hole_at = 0, mover_at = 0, n_moves = 0;
  for (int k = 0; k < kPagesCluster; ++k) {
    const int h = *cl.map_shared_rank(&hole_s, k), m = *cl.map_shared_rank(&mover_s, k);
    if (k < rank) hole_at += h, mover_at += m;
    n_moves += m;
  }
  for (int c0 = p0; c0 < p1; c0 += kPagesThreads) {
    const int p = c0 + threadIdx.x;
    const bool in = p < p1, live = in && a.ref[p] > 0, low = p < L;
    int here;
    // of one chunk the holes lie below L and the movers do not: one sum with the two in halves
    const int r = block_prefix(in && low && !live ? 1 : live && !low ? 1 << 16 : 0, sums, here);
    const int hi = hole_at + (r & 0xffff), mi = mover_at + (r >> 16);
    hole_at += here & 0xffff;
    mover_at += here >> 16;
    if (in && low && !live) dst[hi] = p;
    if (live && !low) src[mi] = p;
    if (in) rank_of[p] = live ? (low ? 0 : mi) : -1;
    if (in) a.free_list[a.num_pages - 1 - p] = low ? -1 : p;
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.moves[0] = n_moves;
    a.moves[1] = L;
    *a.n_free = a.num_pages - L;
  }
  cl.sync();  // no block leaves while its counts may be read
}

// Second launch: the moved pages' arrays in pieces of 8 KB, their references, and the tables.
// Sources are >= L and destinations < L, so no page is both and the copies need no order.
constexpr int kMovePiece = 8192;
__global__ void __launch_bounds__(256) pages_move_kernel(const PagesArgs a, const PageSlabs sl) {
  griddep_launch_dependents();
  griddep_wait();
  const int half = a.num_pages / 2;
  const int n_moves = a.moves[0], L = a.moves[1];
  const int32_t* src = a.moves + 4;
  const int32_t* dst = src + half;
  const int32_t* rank_of = dst + half;
  int pieces = 0;
  for (int k = 0; k < sl.n; ++k) pieces += (int)((sl.s[k].slab_bytes * sl.Hkv[k] + kMovePiece - 1) / kMovePiece);
  for (long long x = blockIdx.x; x < (long long)n_moves * pieces; x += gridDim.x) {
    const int m = (int)(x / pieces);
    int piece = (int)(x % pieces), k = 0;
    const int of = src[m], to = dst[m];
    long long bytes = sl.s[0].slab_bytes * sl.Hkv[0];
    while (piece >= (int)((bytes + kMovePiece - 1) / kMovePiece)) {
      piece -= (int)((bytes + kMovePiece - 1) / kMovePiece);
      ++k;
      bytes = sl.s[k].slab_bytes * sl.Hkv[k];
    }
    const long long o = (long long)piece * kMovePiece;
    const int len = (int)min((long long)kMovePiece, bytes - o);
    const uint8_t* f = sl.s[k].base + of * bytes + o;
    uint8_t* d = sl.s[k].base + to * bytes + o;
    if (len == kMovePiece && (((uintptr_t)f | (uintptr_t)d) & 15) == 0) {
      uint4 v[kMovePiece / 16 / 256];
#pragma unroll
      for (int i = 0; i < kMovePiece / 16 / 256; ++i) v[i] = reinterpret_cast<const uint4*>(f)[threadIdx.x + 256 * i];
#pragma unroll
      for (int i = 0; i < kMovePiece / 16 / 256; ++i) reinterpret_cast<uint4*>(d)[threadIdx.x + 256 * i] = v[i];
    } else {
      for (int i = threadIdx.x; i < len / 4; i += 256)
        reinterpret_cast<uint32_t*>(d)[i] = reinterpret_cast<const uint32_t*>(f)[i];
    }
    if (piece == 0 && k == 0 && threadIdx.x == 0) {
      a.ref[to] = a.ref[of];
      a.ref[of] = 0;
    }
  }
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  for (int b = warp; b < a.batch; b += gridDim.x * 8) {
    const int t = a.seq_len[b];
    if (!good_len(t, a.max_pages)) {
      if (lane == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      continue;
    }
    for (int j = lane; j < pages_of(t); j += 32) {
      int32_t* e = a.bt + (size_t)b * a.max_pages + j;
      const int page = *e;
      const int r = page >= 0 && page < a.num_pages ? rank_of[page] : -1;
      if (r < 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
      else if (page >= L) *e = dst[r];
    }
  }
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PageSlabs& sl, cudaStream_t s) {
  const cudaError_t e = launch_pdl(pages_compact_plan_kernel, dim3(kPagesCluster), dim3(kPagesThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_move_kernel, dim3(152 * 8), dim3(256), 0, s, a, sl);
}

}  // namespace hs2
