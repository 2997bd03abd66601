// pages.cu — the books of a page pool: growing, freeing and forking sequences, compaction.
//
// A pool's pages are numbered alike in every cache that shares its block table. The books are
// a reference count per page and a stack of free pages. What a call takes or returns is
// decided by prefix sums in a fixed order (sequence, then entry; or page), never by the order
// in which atomics land, so tables, counts and stack are the same on every run.
//
// Bound by latency: the books of a pool of 10^4..10^5 pages are a few hundred KB, so a call
// is one or two short launches with few dependent rounds of loads. Only the copies (a forked
// sequence's partial page, the pages that compaction moves) are bandwidth.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace hs2 {

namespace cg = cooperative_groups;

namespace {

constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;  // CTAs of the clusters that scan all pages
constexpr int kGone = -1;         // ref of a page whose last reference the running free call took

// Exclusive prefix sum over the block (all threads call it); `total` is the block's sum.
HS2_DEVI int block_prefix(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int k = 0; k < (int)(blockDim.x >> 5); ++k) {
    if (k < warp) before += warp_sums[k];
    total += warp_sums[k];
  }
  return before + x - v;
}

HS2_DEVI int pages_of(int t) { return (t + kPage - 1) / kPage; }
HS2_DEVI bool good_len(int t, int max_pages) { return t >= 0 && t <= max_pages * kPage; }

}  // namespace

// ---------------------------------------------------------------------------- grow
// One block. Sequences in chunks of 1024: a prefix sum of the pages each needs, then a warp
// per sequence writes its entries.
__global__ void __launch_bounds__(kPagesThreads) pages_grow_kernel(const PagesArgs a) {
  __shared__ int sums[32], base[kPagesThreads], need_s[kPagesThreads], from[kPagesThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nf = *a.n_free;
  auto need_of = [&](int b, int& first, bool flag) -> int {
    first = 0;
    if (b >= a.batch) return -1;
    const int old = a.seq_len[b], add = a.n_new[b];
    if (add < 0 || !good_len(old, a.max_pages) || add > a.max_pages * kPage - old) {
      if (flag) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      return -1;
    }
    first = pages_of(old);
    return pages_of(old + add) - first;
  };
  long long all = 0;
  int first, total;
  for (int b0 = 0; b0 < a.batch; b0 += kPagesThreads) {
    const int need = need_of(b0 + threadIdx.x, first, true);
    (void)block_prefix(max(need, 0), sums, total);
    all += total;
  }
  if (nf < 0 || nf > a.num_pages || all > nf) {
    if (threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    return;
  }
  int taken = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPagesThreads) {
    const int need = need_of(b0 + threadIdx.x, first, false);
    const int at = block_prefix(max(need, 0), sums, total);
    base[threadIdx.x] = taken + at;
    need_s[threadIdx.x] = need;
    from[threadIdx.x] = first;
    __syncthreads();
    const int nb = min(kPagesThreads, a.batch - b0);
    for (int i = warp; i < nb; i += kPagesThreads / 32)
      for (int j = lane; j < need_s[i]; j += 32) {
        const int page = a.free_list[nf - 1 - base[i] - j];
        a.bt[(size_t)(b0 + i) * a.max_pages + from[i] + j] = page;
        if (page >= 0 && page < a.num_pages) a.ref[page] = 1;
        else flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
      }
    if (need >= 0) a.seq_len[b0 + threadIdx.x] += a.n_new[b0 + threadIdx.x];
    taken += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.n_free = nf - taken;
}

cudaError_t launch_pages_grow(const PagesArgs& a, cudaStream_t s) {
  pages_grow_kernel<<<1, kPagesThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- free
// One cluster. References go down by compare-and-swap, so that a page without one is seen; a
// page that loses its last is marked. Then each block counts and pushes its slice of the
// marked pages, in page order.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)
    pages_free_kernel(const PagesArgs a) {
  __shared__ int sums[32], found;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int nf = *a.n_free;
  const int warp = rank * (kPagesThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  for (int b = warp; b < a.batch; b += kPagesCluster * (kPagesThreads / 32)) {
    if (a.drop[b] == 0) continue;
    const int t = a.seq_len[b];
    if (!good_len(t, a.max_pages)) {
      if (lane == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      continue;
    }
    for (int j = lane; j < pages_of(t); j += 32) {
      const int page = a.bt[(size_t)b * a.max_pages + j];
      bool ok = page >= 0 && page < a.num_pages;
      if (ok) {
        int cur = atomicAdd(&a.ref[page], 0);
        while (true) {
          if (cur <= 0) {
            ok = false;
            break;
          }
          const int seen = atomicCAS(&a.ref[page], cur, cur == 1 ? kGone : cur - 1);
          if (seen == cur) break;
          cur = seen;
        }
      }
      if (!ok) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    }
  }
  cl.sync();
  const int per = ((a.num_pages + kPagesCluster - 1) / kPagesCluster + 3) & ~3;
  const int p0 = min(a.num_pages, rank * per), p1 = min(a.num_pages, p0 + per);
  int mine = 0;
  for (int p = p0 + threadIdx.x; p < p1; p += kPagesThreads) mine += __ldcg(&a.ref[p]) == kGone;
  int total;
  (void)block_prefix(mine, sums, total);
  if (threadIdx.x == 0) found = total;
  cl.sync();
  int at = nf, all = 0;
  for (int k = 0; k < kPagesCluster; ++k) {
    const int f = *cl.map_shared_rank(&found, k);
    if (k < rank) at += f;
    all += f;
  }
  cl.sync();  // every block has read the counts
  for (int c0 = p0; c0 < p1; c0 += kPagesThreads) {
    const int p = c0 + threadIdx.x;
    const bool gone = p < p1 && __ldcg(&a.ref[p]) == kGone;
    const int i = at + block_prefix(gone, sums, total);
    if (gone) {
      a.ref[p] = 0;
      if (i >= 0 && i < a.num_pages) a.free_list[i] = p;
      else flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    }
    at += total;
  }
  if (rank == 0 && threadIdx.x == 0) *a.n_free = min(nf + all, a.num_pages);
}

cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t s) {
  pages_free_kernel<<<kPagesCluster, kPagesThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- fork
// First launch, one block: lengths, and the page of its own that a branch's partial page takes
// (at its entry of the branch's table, -1 where it takes none).
__global__ void __launch_bounds__(kPagesThreads) pages_fork_plan_kernel(const PagesArgs a) {
  __shared__ int sums[32];
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
  int all = 0, total;
  for (int c0 = 0; c0 < a.n_child; c0 += kPagesThreads) {
    const int t = len_of(c0 + threadIdx.x, true);
    (void)block_prefix(t % kPage != 0, sums, total);
    all += total;
  }
  const bool fits = nf >= 0 && nf <= a.num_pages && all <= nf;
  if (!fits && threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
  int taken = 0;
  for (int c0 = 0; c0 < a.n_child; c0 += kPagesThreads) {
    const int c = c0 + threadIdx.x;
    const int t = fits ? len_of(c, false) : 0;
    const bool own = t % kPage != 0;
    const int i = taken + block_prefix(own, sums, total);
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
  if (threadIdx.x == 0 && taken > 0) *a.n_free = nf - taken;
  griddep_launch_dependents();
}

// Second launch, grid (branches, slabs of a page): the rest of the branch's table (slab 0) and
// the filled rows of the source's last page.
__global__ void __launch_bounds__(256) pages_fork_copy_kernel(const PagesArgs a, const PageSlabs sl) {
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
  if (of < 0 || of >= a.num_pages) {
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
  pages_fork_plan_kernel<<<1, kPagesThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int slabs = 0;
  for (int k = 0; k < sl.n; ++k) slabs += sl.Hkv[k];
  return launch_pdl(pages_fork_copy_kernel, dim3(a.n_child, slabs), dim3(256), 0, s, a, sl);
}

// ---------------------------------------------------------------------------- compact
// First launch, one cluster: every block takes a slice of the pages; holes (free pages below
// L) and movers (referenced pages from L on) get their ranks from the blocks' counts, the
// i-th mover goes to the i-th hole, and the books and the block table follow.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)
    pages_compact_plan_kernel(const PagesArgs a) {
  __shared__ int sums[32], count[2];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int per = (a.num_pages + kPagesCluster - 1) / kPagesCluster;
  const int p0 = min(a.num_pages, rank * per), p1 = min(a.num_pages, p0 + per);
  const int half = a.num_pages / 2;
  int32_t* src = a.moves + 4;
  int32_t* dst = src + half;
  int32_t* map = dst + half;
  int mine = 0, total;
  for (int p = p0 + threadIdx.x; p < p1; p += kPagesThreads) mine += a.ref[p] > 0;
  (void)block_prefix(mine, sums, total);
  if (threadIdx.x == 0) count[0] = total;
  cl.sync();
  int L = 0;
  for (int k = 0; k < kPagesCluster; ++k) L += *cl.map_shared_rank(&count[0], k);
  // holes and movers of this slice: a slice's pages below L, then those from L on
  const int cut = min(max(L, p0), p1);
  int holes = 0, movers = 0;
  for (int p = p0 + threadIdx.x; p < p1; p += kPagesThreads) {
    const bool live = a.ref[p] > 0;
    holes += !live && p < cut;
    movers += live && p >= cut;
  }
  int nh, nm;
  (void)block_prefix(holes, sums, nh);
  (void)block_prefix(movers, sums, nm);
  cl.sync();  // count[0] has been read
  if (threadIdx.x == 0) count[0] = nh, count[1] = nm;
  cl.sync();
  int hole_at = 0, mover_at = 0, n_moves = 0;
  for (int k = 0; k < kPagesCluster; ++k) {
    const int h = *cl.map_shared_rank(&count[0], k), m = *cl.map_shared_rank(&count[1], k);
    if (k < rank) hole_at += h, mover_at += m;
    n_moves += m;
  }
  for (int c0 = p0; c0 < p1; c0 += kPagesThreads) {
    const int p = c0 + threadIdx.x;
    const bool live = p < p1 && a.ref[p] > 0;
    const bool hole = p < p1 && !live && p < L, mover = live && p >= L;
    const int hi = hole_at + block_prefix(hole, sums, total);
    hole_at += total;
    const int mi = mover_at + block_prefix(mover, sums, total);
    mover_at += total;
    if (hole) dst[hi] = p;
    if (mover) src[mi] = p;
    if (p < p1 && p >= L) {
      if (!live) map[p] = -1;
      a.free_list[a.num_pages - 1 - p] = p;
    }
    if (p < p1 && p < L) a.free_list[a.num_pages - 1 - p] = -1;
  }
  cl.sync();
  const int tid = rank * kPagesThreads + threadIdx.x;
  for (int i = tid; i < n_moves; i += kPagesCluster * kPagesThreads) {
    const int from = __ldcg(src + i), to = __ldcg(dst + i);
    map[from] = to;
    a.ref[to] = a.ref[from];
    a.ref[from] = 0;
  }
  if (tid == 0) {
    a.moves[0] = n_moves;
    *a.n_free = a.num_pages - L;
  }
  cl.sync();
  const int warp = tid >> 5, lane = tid & 31;
  for (int b = warp; b < a.batch; b += kPagesCluster * (kPagesThreads / 32)) {
    const int t = a.seq_len[b];
    if (!good_len(t, a.max_pages)) {
      if (lane == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      continue;
    }
    for (int j = lane; j < pages_of(t); j += 32) {
      int32_t* e = a.bt + (size_t)b * a.max_pages + j;
      const int page = *e;
      if (page < 0 || page >= a.num_pages) {
        flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
      } else if (page >= L) {
        const int to = __ldcg(map + page);
        if (to < 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        else *e = to;
      }
    }
  }
  griddep_launch_dependents();
}

// Second launch: the moved pages' arrays. Sources are >= L and destinations < L, so no page is
// both and the copies need no order.
__global__ void __launch_bounds__(256) pages_move_kernel(const PagesArgs a, const PageSlabs sl) {
  griddep_wait();
  const int half = a.num_pages / 2;
  const int n_moves = a.moves[0];
  const int32_t* src = a.moves + 4;
  const int32_t* dst = src + half;
  for (int m = blockIdx.x; m < n_moves; m += gridDim.x) {
    const int of = src[m], to = dst[m];
    for (int k = 0; k < sl.n; ++k) {
      const long long bytes = sl.s[k].slab_bytes * sl.Hkv[k];
      const uint8_t* f = sl.s[k].base + of * bytes;
      uint8_t* d = sl.s[k].base + to * bytes;
      if (bytes % 16 == 0 && ((uintptr_t)f & 15) == 0) {
        for (long long i = threadIdx.x; i < bytes / 16; i += blockDim.x)
          reinterpret_cast<uint4*>(d)[i] = reinterpret_cast<const uint4*>(f)[i];
      } else {
        for (long long i = threadIdx.x; i < bytes / 4; i += blockDim.x)
          reinterpret_cast<uint32_t*>(d)[i] = reinterpret_cast<const uint32_t*>(f)[i];
      }
    }
  }
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PageSlabs& sl, cudaStream_t s) {
  pages_compact_plan_kernel<<<kPagesCluster, kPagesThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_move_kernel, dim3(152 * 8), dim3(256), 0, s, a, sl);
}

}  // namespace hs2
