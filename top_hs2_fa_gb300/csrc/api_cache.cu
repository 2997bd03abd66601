// api_cache.cu — the extern "C" boundary of the paged-cache operators: rows in and out, chunk
// attention, pages. Validation and launches as in api.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/hs2.h"
#include "api_util.h"
#include "kernels.h"

using namespace hs2::api;

namespace {

size_t elem_bytes(hs2_dtype t) { return t == HS2_F32 ? 4 : 2; }

hs2_status kv_rows(const hs2_kv* kv, const void* k_rows, const void* v_rows, hs2_dtype row_dtype, int64_t row_stride,
                   const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream, bool write) {
  if (!valid_kv(kv, false) || !row_start || n_rows < 0) return HS2_ERR_ARG;
  if (kv->v && !valid_kv(kv, true)) return HS2_ERR_ARG;
  if (row_dtype != HS2_F32 && row_dtype != HS2_BF16) return HS2_ERR_ARG;
  if (n_rows == 0) return HS2_OK;
  if (!k_rows || !aligned16(k_rows) || (kv->v && (!v_rows || !aligned16(v_rows)))) return HS2_ERR_ARG;
  if (row_stride < (int64_t)kv->Hkv * kv->d || row_stride * elem_bytes(row_dtype) % 16 != 0) return HS2_ERR_ARG;
  if (kv->Hkv > 65535) return HS2_ERR_UNSUPPORTED;  // grid y
  hs2::RowsArgs a{};
  a.k = const_cast<void*>(kv->k);
  a.v = const_cast<void*>(kv->v);
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.k_sf = const_cast<uint8_t*>(kv->k_sf);
  a.v_sf = const_cast<uint8_t*>(kv->v_sf);
  a.bt = kv->block_table;
  a.seq_len = kv->seq_len;
  a.batch = kv->batch;
  a.num_pages = kv->num_pages;
  a.max_pages = kv->max_pages;
  a.Hkv = kv->Hkv;
  a.k_rows = k_rows;
  a.v_rows = v_rows;
  a.row_stride = row_stride;
  a.row_start = row_start;
  a.n_rows = n_rows;
  a.dev_err = dev_err;
  const cudaError_t e = hs2::launch_kv_rows(a, kv->d, kv->dtype, write, row_dtype == HS2_F32, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 152;
  }
  return std::min(n, 512);  // the merge's blocks hold the list of cut units, one per CTA at most
}

// Which kernels a call runs, by the rows (tokens times G) that share a KV head's keys.
struct ChunkCuts {
  int narrow;  // the narrow kernel takes sequences of up to this many rows, 0: none
  bool wide;   // the wide kernel takes the rest
};

// The narrow kernel reads the cache's codes and converts each once per 64 rows. The wide one runs
// at the tensor pipe's rate, 256 rows at a time, but FP8 / FP4 pages are expanded to bf16 for it. Each
// plan costs about 20 us whatever it holds. `top` rows are the most a sequence can have. d = 128,
// FP8 where nothing else is said; FP4 is within 4 %:
//   bf16: no expansion. Single tokens of 8 rows take 25 us narrow, 29 wide (8 sequences), 94 and 107
//     (256), 477 and 480 (64 long ones); 8 sequences of 8 to 160 rows 67 with both, 40 wide, 64 long
//     ones 603 and 590.
//   up to 256 rows: one sequence of 256 rows and 32K keys 68 narrow, 95 wide; at 512 rows 98 and 95;
//     8 sequences of 8K to 16K keys with 256 rows 143 and 134, with 512 rows 247 and 166 (FP4). So
//     one sequence alone sets the border; the rule does not count sequences, and several lose 6 % there.
//   few rows times keys: 5 sequences of 32 to 352 rows over 1K to 6K keys 35 narrow, 39 wide, 55 both;
//     one of 512 rows and 2K keys 31 and 35, and 16K keys 62 and 56.
//   little to expand: 12 sequences of 32 to 22400 rows over 1K to 6K keys 132 wide, 161 both; 9 of up
//     to 512 rows (110 MB expanded) 68 and 84; 16 of up to 800 rows and 16K keys (520 MB) 229 and
//     212; 64 of up to 800 rows (8 GB) 2998 and 2191.
constexpr long long kFewExpanded = 256LL << 20;
ChunkCuts chunk_cuts(long long top, int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t, int w) {
  const int all = 0x7fffffff;
  const long long keys = w > 0 ? std::min<long long>(max_t, (long long)max_n + w) : max_t;
  if (kv->dtype == HS2_BF16) return top <= 64 ? ChunkCuts{all, false} : ChunkCuts{0, true};
  if (top <= 256 || (long long)n_rows * Hq * keys <= 1LL << 24) return {all, false};
  const long long expanded = kv->batch * keys * kv->Hkv * kv->d * 4;  // bytes, K and V
  return {expanded <= kFewExpanded ? 0 : 256, true};
}

// Workspace of hs2_fa_chunk: the plans of the two kernels with their parts, and the expanded
// pages of a quantised cache.
struct ChunkLayout {
  int n_plans;
  hs2::ChunkPlan plan[2];  // narrow, wide, or both; pointers after bind()
  bool narrow[2];
  size_t off[2][7], off_exp[4];
  int exp_seqs, exp_pages_seq;
  size_t off_ek, off_ev, off_params, total;
  long long tiles;  // an upper bound of a plan's tiles
};

// Most rows of a sequence, as the declared sizes have it.
long long chunk_top(int n_rows, int Hq, const hs2_kv* kv, int max_n) {
  return (long long)std::min(max_n, n_rows) * (Hq / kv->Hkv);
}

// `most_pages` bounds the expanded pages further.
ChunkLayout chunk_layout(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t, int w, ChunkCuts cut,
                         long long most_pages) {
  ChunkLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  if (kv->dtype != HS2_F32 && n_rows > 0 && max_n > 0 && max_t > 0) {
    const int G = Hq / kv->Hkv;
    const long long top = chunk_top(n_rows, Hq, kv, max_n);
    auto add = [&](bool narrow, int tile_rows, int lo, int hi) {
      hs2::ChunkPlan& p = L.plan[L.n_plans];
      L.narrow[L.n_plans] = narrow;
      p.ctas = sm_count();
      p.tile_rows = tile_rows;
      p.min_rows = lo;
      p.max_rows = hi;
      p.snap = 2;
      const long long units = (long long)kv->Hkv * ((long long)n_rows * G / tile_rows + std::min(kv->batch, n_rows));
      p.max_units = (int)std::min<long long>(units, 1 << 30);
      L.tiles = std::max(L.tiles, units * (max_t / 128 + 2));
      size_t* o = L.off[L.n_plans++];
      o[0] = take(16);
      o[1] = take(4 * (size_t)p.ctas);
      o[2] = take(4 * (size_t)p.ctas);
      o[6] = take(4 * (size_t)p.ctas);
      o[3] = take(48 * (size_t)p.max_units);
      o[4] = take(2 * (size_t)p.ctas * tile_rows * 8);
      o[5] = take(2 * (size_t)p.ctas * tile_rows * kv->d * 4);
      return &p;
    };
    if (cut.narrow > 0) {
      const long long few = std::min<long long>(top, cut.narrow);
      add(true, few <= 16 ? 16 : few <= 32 ? 32 : 64, 0, cut.narrow);
    }
    if (cut.wide) {
      hs2::ChunkPlan* p = add(false, 256, cut.narrow, 0x7fffffff);
      p->expand = low_precision(kv);
      if (p->expand) {
        L.exp_seqs = (int)std::min<long long>(kv->batch, (long long)n_rows * G / (cut.narrow + 1));
        L.exp_pages_seq = cdiv(max_t, 64);
        if (w > 0) L.exp_pages_seq = (int)std::min<long long>(L.exp_pages_seq, ((long long)max_n + w) / 64 + 2);
        const long long pages = std::min((long long)L.exp_seqs * L.exp_pages_seq, most_pages);
        if (pages * kv->Hkv * 64 > 0x7fffffff) L.tiles = 1LL << 40;  // beyond a tensor map's rows
        p->max_exp_pages = (int)std::min<long long>(pages, 0x7fffffff);
        for (int i = 0; i < 3; ++i) L.off_exp[i] = take(4 * (size_t)L.exp_seqs);
        L.off_exp[3] = take(4);
        const size_t rows = (size_t)pages * kv->Hkv * 64;
        L.off_ek = take(rows * kv->d * 2);
        L.off_ev = take(rows * kv->d * 2);
        L.off_params = take(rows / 64 * 8);
      }
    }
  }
  L.total = std::max<size_t>(off, 256);
  return L;
}

ChunkLayout chunk_layout(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t, int w) {
  const ChunkCuts cut = chunk_cuts(chunk_top(n_rows, Hq, kv, max_n), n_rows, Hq, kv, max_n, max_t, w);
  return chunk_layout(n_rows, Hq, kv, max_n, max_t, w, cut, 1LL << 60);
}

// What this call and every call with fewer rows, tokens or keys needs, whichever kernels those run:
// narrower units are more, and a call that splits its sequences may expand fewer pages than a
// smaller one that does not.
size_t chunk_bytes(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t, int w) {
  const long long any = 1LL << 60;
  const ChunkCuts cut = chunk_cuts(chunk_top(n_rows, Hq, kv, max_n), n_rows, Hq, kv, max_n, max_t, w);
  size_t need = chunk_layout(n_rows, Hq, kv, max_n, max_t, w, cut, any).total;
  for (int rows = 16; rows <= 64; rows *= 2) {
    const int n = std::min(max_n, std::max(1, rows / (Hq / kv->Hkv)));
    need = std::max(need, chunk_layout(n_rows, Hq, kv, n, max_t, w, {0x7fffffff, false}, any).total);
  }
  if (cut.wide) {
    const long long few = kFewExpanded / (256LL * kv->Hkv * kv->d) + 2LL * kv->batch;
    need = std::max(need, chunk_layout(n_rows, Hq, kv, max_n, max_t, w, {0, true}, few).total);
  }
  return need;
}

void bind(ChunkLayout& L, char* ws) {
  for (int i = 0; i < L.n_plans; ++i) {
    hs2::ChunkPlan& p = L.plan[i];
    p.head = (int32_t*)(ws + L.off[i][0]);
    p.cta_first = (int32_t*)(ws + L.off[i][1]);
    p.cuts = (int32_t*)(ws + L.off[i][2]);
    p.cta_begin = (int32_t*)(ws + L.off[i][6]);
    p.units = (int32_t*)(ws + L.off[i][3]);
    p.part_ml = (float*)(ws + L.off[i][4]);
    p.part_o = (float*)(ws + L.off[i][5]);
    if (p.expand) {
      p.exp_seq = (int32_t*)(ws + L.off_exp[0]);
      p.exp_base = (int32_t*)(ws + L.off_exp[1]);
      p.exp_page = (int32_t*)(ws + L.off_exp[2]);
      p.exp_head = (int32_t*)(ws + L.off_exp[3]);
    }
  }
}

bool valid_pages(const hs2_pages* p) { return p && p->ref && p->free_list && p->n_free && p->num_pages >= 1; }
// a sequence's entries; the bound keeps sums of 1024 sequences' pages within 32 bits
bool valid_table(int batch, int max_pages) { return batch >= 1 && max_pages >= 1 && max_pages <= (1 << 20); }

hs2::PagesArgs pages_args(const hs2_pages* p, int32_t* dev_err) {
  hs2::PagesArgs a{};
  a.ref = p->ref;
  a.free_list = p->free_list;
  a.n_free = p->n_free;
  a.num_pages = p->num_pages;
  a.dev_err = dev_err;
  return a;
}

// The caches of one table: their arrays, and the table itself.
bool page_caches(const hs2_pages* pages, int n_caches, const hs2_kv* kvs, hs2::PagesArgs* a, hs2::PageSlabs* sl) {
  if (!valid_pages(pages) || !kvs || n_caches < 1 || n_caches > hs2::kMaxPageCaches) return false;
  sl->n = 0;
  auto add = [&](const void* base, int Hkv, long long slab_bytes, int row_bytes) {
    hs2::PageSlab& s = sl->s[sl->n];
    s.base = (uint8_t*)const_cast<void*>(base);
    s.slab_bytes = slab_bytes;
    s.row_bytes = row_bytes;
    sl->Hkv[sl->n++] = Hkv;
  };
  for (int c = 0; c < n_caches; ++c) {
    const hs2_kv* kv = &kvs[c];
    if (valid_latent(kv) ? low_precision(kv) : !valid_kv(kv, false) || (kv->v && !valid_kv(kv, true))) return false;
    if (kv->num_pages != pages->num_pages || kv->block_table != kvs[0].block_table || kv->seq_len != kvs[0].seq_len ||
        kv->batch != kvs[0].batch || kv->max_pages != kvs[0].max_pages)
      return false;
    const int row = kv->dtype == HS2_F32 ? 4 * kv->d : kv->dtype == HS2_BF16 ? 2 * kv->d
                                                   : kv->dtype == HS2_FP8_E4M3 ? kv->d : kv->d / 2;
    for (int side = 0; side < (kv->v ? 2 : 1); ++side) {
      add(side ? kv->v : kv->k, kv->Hkv, 64LL * row, row);
      if (kv->dtype == HS2_FP4_E2M1) add(side ? kv->v_sf : kv->k_sf, kv->Hkv, 64LL * (kv->d / 16), kv->d / 16);
      if (low_precision(kv)) add(side ? kv->v_scale : kv->k_scale, kv->Hkv, 4, 0);
    }
  }
  if (!valid_table(kvs[0].batch, kvs[0].max_pages)) return false;
  a->bt = const_cast<int32_t*>(kvs[0].block_table);
  a->seq_len = const_cast<int32_t*>(kvs[0].seq_len);
  a->batch = kvs[0].batch;
  a->max_pages = kvs[0].max_pages;
  return true;
}

}  // namespace

extern "C" {

hs2_status hs2_kv_write(const hs2_kv* kv, const void* k_rows, const void* v_rows, hs2_dtype row_dtype,
                        int64_t row_stride, const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream) {
  return kv_rows(kv, k_rows, v_rows, row_dtype, row_stride, row_start, n_rows, dev_err, stream, true);
}

hs2_status hs2_kv_read(const hs2_kv* kv, void* k_rows, void* v_rows, hs2_dtype row_dtype, int64_t row_stride,
                       const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream) {
  return kv_rows(kv, k_rows, v_rows, row_dtype, row_stride, row_start, n_rows, dev_err, stream, false);
}

size_t hs2_fa_chunk_workspace(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t, int w) {
  if (!kv || kv->batch < 1 || kv->Hkv < 1 || Hq < 1 || n_rows < 0 || max_n < 0 || max_t < 0 || w < 0 ||
      (kv->d != 64 && kv->d != 128))
    return 0;
  if (Hq % kv->Hkv != 0 || !pow2_le32(Hq / kv->Hkv)) return 0;
  return chunk_bytes(n_rows, Hq, kv, max_n, max_t, w);
}

hs2_status hs2_fa_chunk(const void* q, const int32_t* row_start, int n_rows, int max_n, int Hq, const hs2_kv* kv,
                        int max_t, int w, float scale, const float* sink, void* o, hs2_dtype o_dtype, float* lse,
                        void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream) {
  if (!valid_kv(kv, true) || !row_start || n_rows < 0 || Hq < 1 || Hq % kv->Hkv != 0) return HS2_ERR_ARG;
  if (!pow2_le32(Hq / kv->Hkv)) return HS2_ERR_UNSUPPORTED;
  if (max_n < 0 || max_n > max_t || (long long)max_t > (long long)kv->max_pages * 64 || w < 0) return HS2_ERR_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return HS2_ERR_ARG;
  if (o_dtype != HS2_F32 && o_dtype != HS2_BF16) return HS2_ERR_ARG;
  if (n_rows == 0 || max_n == 0) return HS2_OK;
  if (!q || !aligned16(q) || !o || !aligned16(o)) return HS2_ERR_ARG;
  if (Hq > 65535 || (kv->max_pages > (1 << 24))) return HS2_ERR_UNSUPPORTED;
  ChunkLayout L = chunk_layout(n_rows, Hq, kv, max_n, max_t, w);
  // 32-bit tile counts and pool rows; grid y
  if (L.tiles > 1LL << 30 || (long long)kv->num_pages * kv->Hkv * 64 > 0x7fffffff - 64 || kv->Hkv > 65535)
    return HS2_ERR_UNSUPPORTED;
  if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < L.total) return HS2_ERR_ARG;
  hs2::ChunkArgs a{};
  a.q = q;
  a.row_start = row_start;
  a.n_rows = n_rows;
  a.max_n = max_n;
  a.max_t = max_t;
  a.batch = kv->batch;
  a.Hq = Hq;
  a.Hkv = kv->Hkv;
  a.G = Hq / kv->Hkv;
  while ((1 << a.log2G) < a.G) ++a.log2G;
  a.k = kv->k;
  a.v = kv->v;
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.k_sf = kv->k_sf;
  a.v_sf = kv->v_sf;
  a.bt = kv->block_table;
  a.seq_len = kv->seq_len;
  a.num_pages = kv->num_pages;
  a.max_pages = kv->max_pages;
  a.w = w >= max_t ? 0 : w;  // a window that hides nothing
  a.scale_log2 = scale * 1.4426950408889634f;
  a.sink = sink;
  a.o = o;
  a.o_bf16 = o_dtype == HS2_BF16;
  a.lse = lse;
  a.dev_err = dev_err;
  cudaStream_t s = (cudaStream_t)stream;
  if (kv->dtype == HS2_F32) {
    const cudaError_t e = hs2::launch_chunk_cc(a, kv->d, s);
    return e == cudaSuccess ? HS2_OK : cuda_fail(e);
  }
  char* ws = (char*)workspace;
  bind(L, ws);
  // every tensor map before the first launch, so that an error launches nothing
  CUtensorMap map[2][3];
  const uint64_t pool_rows = (uint64_t)kv->num_pages * kv->Hkv * 64;
  for (int i = 0; i < L.n_plans; ++i) {
    const hs2::ChunkPlan& p = L.plan[i];
    bool ok;
    if (L.narrow[i] && low_precision(kv)) {
      const uint32_t row = kv->dtype == HS2_FP8_E4M3 ? kv->d : kv->d / 2;
      ok = encode_2d_bytes(&map[i][1], kv->k, row, pool_rows, 64) && encode_2d_bytes(&map[i][2], kv->v, row, pool_rows, 64);
    } else {
      const uint64_t rows = p.expand ? (uint64_t)p.max_exp_pages * kv->Hkv * 64 : pool_rows;
      ok = encode_2d_bf16(&map[i][1], p.expand ? ws + L.off_ek : kv->k, kv->d, rows, 64) &&
           encode_2d_bf16(&map[i][2], p.expand ? ws + L.off_ev : kv->v, kv->d, rows, 64);
    }
    ok = ok && encode_3d_bf16(&map[i][0], q, kv->d, (uint64_t)Hq, (uint64_t)n_rows, a.G,
                              (L.narrow[i] ? p.tile_rows : 128) / a.G);
    if (!ok) return HS2_ERR_ARG;
  }
  cudaError_t e = hs2::launch_chunk_plan(a, L.plan, L.n_plans, s);
  for (int i = 0; i < L.n_plans && e == cudaSuccess; ++i) {
    const hs2::ChunkPlan& p = L.plan[i];
    if (L.narrow[i]) {
      e = hs2::launch_chunk_narrow(map[i][0], map[i][1], map[i][2], a, p, kv->d, kv->dtype, s);
      continue;
    }
    float2* params = p.expand ? (float2*)(ws + L.off_params) : nullptr;
    if (p.expand)
      e = hs2::launch_chunk_expand(a, p, kv->d, kv->dtype, ws + L.off_ek, ws + L.off_ev, params, L.exp_seqs,
                                   L.exp_pages_seq, s);
    if (e == cudaSuccess) e = hs2::launch_chunk_wide(map[i][0], map[i][1], map[i][2], a, p, params, kv->d, s);
  }
  if (e == cudaSuccess) e = hs2::launch_chunk_merge(a, L.plan, L.n_plans, kv->d, s);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

hs2_status hs2_pages_grow(const hs2_pages* pages, int32_t* block_table, int32_t* seq_len, const int32_t* n_new,
                          int batch, int max_pages, int32_t* dev_err, void* stream) {
  if (!valid_pages(pages) || !block_table || !seq_len || !n_new || batch < 0 || max_pages < 1) return HS2_ERR_ARG;
  if (batch == 0) return HS2_OK;
  if (!valid_table(batch, max_pages)) return HS2_ERR_UNSUPPORTED;
  hs2::PagesArgs a = pages_args(pages, dev_err);
  a.bt = block_table;
  a.seq_len = seq_len;
  a.n_new = n_new;
  a.batch = batch;
  a.max_pages = max_pages;
  const cudaError_t e = hs2::launch_pages_grow(a, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

hs2_status hs2_pages_free(const hs2_pages* pages, const int32_t* block_table, const int32_t* seq_len,
                          const int32_t* drop, int batch, int max_pages, int32_t* dev_err, void* stream) {
  if (!valid_pages(pages) || !block_table || !seq_len || !drop || batch < 0 || max_pages < 1) return HS2_ERR_ARG;
  if (batch == 0) return HS2_OK;
  if (!valid_table(batch, max_pages)) return HS2_ERR_UNSUPPORTED;
  hs2::PagesArgs a = pages_args(pages, dev_err);
  a.bt = const_cast<int32_t*>(block_table);
  a.seq_len = const_cast<int32_t*>(seq_len);
  a.drop = drop;
  a.batch = batch;
  a.max_pages = max_pages;
  const cudaError_t e = hs2::launch_pages_free(a, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

hs2_status hs2_pages_fork(const hs2_pages* pages, int n_caches, const hs2_kv* kvs, const int32_t* src, int n_child,
                          int32_t* child_table, int32_t* child_len, int32_t* dev_err, void* stream) {
  hs2::PagesArgs a{};
  hs2::PageSlabs sl;
  if (!valid_pages(pages) || !src || !child_table || !child_len || n_child < 0) return HS2_ERR_ARG;
  a = pages_args(pages, dev_err);
  if (!page_caches(pages, n_caches, kvs, &a, &sl)) return HS2_ERR_ARG;
  if (n_child == 0) return HS2_OK;
  int slabs = 0;
  for (int k = 0; k < sl.n; ++k) slabs += sl.Hkv[k];
  if (slabs > 65535) return HS2_ERR_UNSUPPORTED;  // grid y
  a.src = src;
  a.n_child = n_child;
  a.child_table = child_table;
  a.child_len = child_len;
  const cudaError_t e = hs2::launch_pages_fork(a, sl, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

size_t hs2_pages_compact_workspace(const hs2_pages* pages) {
  if (!pages || pages->num_pages < 1) return 0;
  return align256(4 * (4 + 2 * (size_t)(pages->num_pages / 2) + (size_t)pages->num_pages));
}

hs2_status hs2_pages_compact(const hs2_pages* pages, int n_caches, const hs2_kv* kvs, void* workspace,
                             size_t ws_bytes, int32_t* dev_err, void* stream) {
  hs2::PagesArgs a{};
  hs2::PageSlabs sl;
  if (!valid_pages(pages)) return HS2_ERR_ARG;
  a = pages_args(pages, dev_err);
  if (!page_caches(pages, n_caches, kvs, &a, &sl)) return HS2_ERR_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < hs2_pages_compact_workspace(pages)) return HS2_ERR_ARG;
  a.moves = (int32_t*)workspace;
  const cudaError_t e = hs2::launch_pages_compact(a, sl, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

}  // extern "C"
