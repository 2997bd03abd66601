// api_latent.cu — the extern "C" boundary of latent attention and of the rows that are rotated on
// their way into a cache. Validation and launches as in api.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/hs2.h"
#include "api_util.h"
#include "kernels.h"

using namespace hs2::api;

namespace {

int elem_bytes(hs2_dtype t) { return t == HS2_F32 ? 4 : 2; }
bool row_type(hs2_dtype t) { return t == HS2_F32 || t == HS2_BF16; }
// a row array's base and a stride of it: 16-byte loads
bool rows16(const void* p, int64_t stride, hs2_dtype t) { return p && aligned16(p) && stride * elem_bytes(t) % 16 == 0; }

// Bounds on strides and counts that keep products within 64 bits.
constexpr int64_t kMaxStride = 1LL << 31;

bool valid_rot(const hs2_rot* r, int d) {
  return r && r->table && aligned16(r->table) && r->n_pos >= 1 && r->dim >= 32 && r->dim <= d && r->dim % 32 == 0 &&
         (r->pairs == 0 || r->pairs == 1);
}
hs2::RotTable rot_table(const hs2_rot* r) { return {r->table, r->n_pos, r->dim, r->pairs}; }

hs2::RowsArgs rows_args(const hs2_kv* kv, const int32_t* row_start, int n_rows, int32_t* dev_err) {
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
  a.row_start = row_start;
  a.n_rows = n_rows;
  a.dev_err = dev_err;
  return a;
}

hs2_status latent_rows(const hs2_kv* kv, const void* c_rows, int64_t c_stride, const void* r_rows, int64_t r_stride,
                       hs2_dtype row_dtype, const int32_t* row_start, int n_rows, hs2::LatentRowsArgs& z, bool write,
                       int32_t* dev_err, void* stream) {
  z.rows = rows_args(kv, row_start, n_rows, dev_err);
  z.c_rows = c_rows;
  z.r_rows = r_rows;
  z.c_stride = c_stride;
  z.r_stride = r_stride;
  const cudaError_t e = hs2::launch_latent_rows(z, kv->d - hs2::kLatentRot, kv->dtype == HS2_F32, row_dtype == HS2_F32,
                                                write, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

// The checks that the reading and the writing of latent rows share; HS2_OK with *go = false: nothing to do.
hs2_status check_latent_rows(const hs2_kv* kv, const void* c_rows, int64_t c_stride, const void* r_rows,
                             int64_t r_stride, hs2_dtype row_dtype, const int32_t* row_start, int n_rows, bool* go) {
  *go = false;
  if (!valid_latent(kv) || !row_start || n_rows < 0 || !row_type(row_dtype)) return HS2_ERR_ARG;
  if (low_precision(kv)) return HS2_ERR_UNSUPPORTED;
  if (n_rows == 0) return HS2_OK;
  if (!rows16(c_rows, c_stride, row_dtype) || !rows16(r_rows, r_stride, row_dtype)) return HS2_ERR_ARG;
  if (c_stride < kv->d - hs2::kLatentRot || r_stride < hs2::kLatentRot || c_stride > kMaxStride || r_stride > kMaxStride)
    return HS2_ERR_ARG;
  *go = true;
  return HS2_OK;
}

// What the two attention forms take alike.
bool valid_attention(int n_rows, int max_n, int max_t, float scale, hs2_dtype o_dtype) {
  return n_rows >= 0 && max_n >= 0 && max_n <= max_t && std::isfinite(scale) && scale > 0.f && row_type(o_dtype);
}
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 152;
  }
  return std::min(n, 512);  // the merge's blocks hold the list of cut units, one per CTA at most
}

// Calls with few keys cut no unit, and there is nothing to merge: a unit's few tiles take a CTA no longer than
// its parts take the merge. With up to `own` keys and no more sequences than a warp has lanes and 16 units a CTA
// there is no planning kernel either, every CTA finds its units itself; other calls plan, and cut none up to
// `planned` keys. us on the device:
//   absorbed, planned, cut and whole: 4 single tokens of 16 heads over 256 keys 19.2 and 17.0, 64 of them 20.2
//     and 19.1; over 500 keys 19.6 and 20.9, 16 sequences of 3 tokens of 32 heads 24.7 and 27.2.
//   absorbed, planned (whole by length) and own: 8 chunks of 100 of 32 heads over 500 keys 43.4 and 39.4, over 700
//     48.7 and 47.9.
//   expanded, planned, cut and whole: 3 prompts of 64 tokens, 16 heads, over 256 keys 15.0 and 12.5, over 500 15.8
//     and 15.2; 16 of 100 28.0 and 24.4; one of 128 tokens over 700 keys 17.3 and 18.9.
//   expanded, cut and own: one of 128 tokens over 1000 keys 17.6 and 17.2, 3 of 64 18.2 and 17.8, 16 of 400 of
//     32 heads 119 and 92. With up to 4 units a CTA instead of 16 these over 500 keys 77.9, not 71.4.
// Where a sequence has one unit (absorbed, up to 128 rows) every CTA finds its range of the line itself: planned and
// not, 16 single tokens of 16 heads over 2000 keys 23.1 and 18.8, 8 of 128 heads over 8000 46.9 and 40.8, 128 of 16
// over 500 25.3 and 23.7; of pairs with up to 32 sequences (64 single tokens of 128 heads over 300 keys 26.7 and
// 29.8, and 128 over 4000 159 and 165: whole units fit there; but 33 over 2000 46.1 and 42.7). Up to `planned` keys
// the units stay whole (4 single tokens of 16 heads over 256 keys 13.3, as ranges 15.2; over 512 17.0 and 15.4).
struct Whole {
  int planned, own;
};
constexpr Whole kWholeAbsorbed{256, 512}, kWholeExpanded{512, 1024};
// What being cut costs a CTA, in tiles (chunk_plan.cu has the figures).
constexpr int kCutAbsorbed = 4, kCutExpanded = 8;

// Workspace of an attention call: the plan and the parts of cut units.
struct Layout {
  hs2::ChunkPlan plan;  // pointers after bind()
  size_t off[8], total;
  long long tiles;  // an upper bound
};

// `heads` units beside one another per sequence, of G rows a token, parts of dv channels; one: a sequence has one
// unit at most.
Layout layout(int n_rows, int heads, int G, int batch, int tile_rows, int ctas, int dv, int max_t, Whole whole,
              int cut_tiles, bool one) {
  Layout L{};
  size_t at = 0;
  auto take = [&](int i, size_t bytes) { L.off[i] = at, at = align256(at + bytes); };
  hs2::ChunkPlan& p = L.plan;
  p.ctas = ctas;
  p.tile_rows = tile_rows;
  p.max_rows = 0x7fffffff;
  p.cut_tiles = cut_tiles;
  const long long units = heads * ((long long)n_rows * G / tile_rows + std::min(batch, n_rows));
  p.max_units = (int)std::min<long long>(units, 1 << 30);
  L.tiles = units * (max_t / 128 + 2);
  const bool own = max_t <= (one ? whole.planned : whole.own) && batch <= hs2::kOwnPlanSeqs &&
                   units <= hs2::kOwnPlanUnits * (long long)ctas;
  p.own = own ? 1 : one && batch <= hs2::line_seqs(tile_rows == 128) ? 2 : 0;
  // ranges differ by a unit at most: with 2 a prompt's by a third (16384 tokens of 16 heads 981 us)
  p.snap = own || (p.own == 0 && max_t <= whole.planned) ? 0 : 32;
  if (p.own == 1) p.ctas = std::max(1, (int)std::min<long long>(units, ctas));  // no more CTAs than there can be units
  take(0, 16);
  take(1, 4 * (size_t)ctas);
  take(2, 4 * (size_t)ctas);
  take(6, 4 * (size_t)ctas);
  take(3, 48 * (size_t)p.max_units);
  take(4, 2 * (size_t)ctas * tile_rows * 8);
  take(5, 2 * (size_t)ctas * tile_rows * dv * 4);
  take(7, 8 * (size_t)std::min<long long>(units, hs2::kOwnPlanUnits * (long long)ctas));
  L.total = std::max<size_t>(at, 256);
  return L;
}
void bind(Layout& L, char* ws) {
  hs2::ChunkPlan& p = L.plan;
  p.head = (int32_t*)(ws + L.off[0]);
  p.cta_first = (int32_t*)(ws + L.off[1]);
  p.cuts = (int32_t*)(ws + L.off[2]);
  p.cta_begin = (int32_t*)(ws + L.off[6]);
  p.units = (int32_t*)(ws + L.off[3]);
  p.order = p.own ? nullptr : (int2*)(ws + L.off[7]);
  p.part_ml = (float*)(ws + L.off[4]);
  p.part_o = (float*)(ws + L.off[5]);
}

// Rows of a unit of the absorbed form: the least width that holds a sequence's; 128 by pairs of CTAs.
int chunk_width(long long top) { return top <= 16 ? 16 : top <= 32 ? 32 : top <= 64 ? 64 : 128; }
Layout chunk_layout(int n_rows, int Hq, const hs2_kv* kv, int width, int max_t, long long top) {
  const int sms = sm_count();
  return layout(n_rows, 1, Hq, kv->batch, width, width == 128 ? std::max(1, sms / 2) : sms, kv->d - hs2::kLatentRot, max_t,
                kWholeAbsorbed, kCutAbsorbed, top <= width);
}

// A unit of the expanded form is 256 tokens of a head.
Layout prefill_layout(int n_rows, int Hq, int batch, int max_t) {
  return layout(n_rows, Hq, 1, batch, 256, sm_count(), hs2::kLatentValue, max_t, kWholeExpanded, kCutExpanded, false);
}

bool heads_supported(int Hq) { return Hq <= 128 && (Hq & (Hq - 1)) == 0; }

hs2::ChunkArgs chunk_args(const void* q, const int32_t* row_start, int n_rows, int max_n, int max_t, int batch, int Hq,
                          float scale, void* o, hs2_dtype o_dtype, float* lse, int32_t* dev_err) {
  hs2::ChunkArgs a{};
  a.q = q;
  a.row_start = row_start;
  a.n_rows = n_rows;
  a.max_n = max_n;
  a.max_t = max_t;
  a.batch = batch;
  a.Hq = Hq;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.o = o;
  a.o_bf16 = o_dtype == HS2_BF16;
  a.lse = lse;
  a.dev_err = dev_err;
  return a;
}

}  // namespace

extern "C" {

hs2_status hs2_kv_write_rot(const hs2_kv* kv, const void* k_rows, int64_t k_stride, const void* v_rows, int64_t v_stride,
                            hs2_dtype row_dtype, const int32_t* row_start, int n_rows, const hs2_rot* rot, const void* q,
                            int64_t q_stride, int Hq, void* q_out, int64_t q_out_stride, int32_t* dev_err, void* stream) {
  if (!valid_kv(kv, false) || (kv->v && !valid_kv(kv, true))) return HS2_ERR_ARG;
  if (!row_start || n_rows < 0 || !row_type(row_dtype) || !valid_rot(rot, kv->d)) return HS2_ERR_ARG;
  if (Hq < 0) return HS2_ERR_ARG;
  if (n_rows == 0) return HS2_OK;
  if ((Hq > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr)) return HS2_ERR_ARG;
  const int64_t row = (int64_t)kv->Hkv * kv->d, q_row = (int64_t)Hq * kv->d;
  if (!rows16(k_rows, k_stride, row_dtype) || k_stride < row || k_stride > kMaxStride) return HS2_ERR_ARG;
  if (kv->v && (!rows16(v_rows, v_stride, row_dtype) || v_stride < row || v_stride > kMaxStride)) return HS2_ERR_ARG;
  const hs2_dtype q_type = kv->dtype == HS2_F32 ? HS2_F32 : HS2_BF16;
  if (q && (!rows16(q, q_stride, row_dtype) || q_stride < q_row || q_stride > kMaxStride ||
            !rows16(q_out, q_out_stride, q_type) || q_out_stride < q_row || q_out_stride > kMaxStride))
    return HS2_ERR_ARG;
  if (q && q == q_out && (q_type != row_dtype || q_stride != q_out_stride)) return HS2_ERR_ARG;
  if (kv->Hkv > 65535 || Hq > 65535) return HS2_ERR_UNSUPPORTED;
  hs2::RotRowsArgs z{};
  z.rows = rows_args(kv, row_start, n_rows, dev_err);
  z.rows.k_rows = k_rows;
  z.rows.v_rows = v_rows;
  z.rows.row_stride = k_stride;
  z.v_stride = v_stride;
  z.rot = rot_table(rot);
  z.q = q;
  z.q_out = q_out;
  z.q_stride = q_stride;
  z.q_out_stride = q_out_stride;
  z.Hq = Hq;
  const cudaError_t e = hs2::launch_kv_write_rot(z, kv->d, kv->dtype, row_dtype == HS2_F32, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

hs2_status hs2_latent_write(const hs2_kv* kv, const void* c_rows, int64_t c_stride, const void* r_rows, int64_t r_stride,
                            hs2_dtype row_dtype, const int32_t* row_start, int n_rows, const hs2_rot* rot, const void* q,
                            int64_t q_stride, int64_t q_head, int Hq, void* q_out, int64_t q_out_stride,
                            int64_t q_out_head, int32_t* dev_err, void* stream) {
  if (!valid_rot(rot, hs2::kLatentRot) || rot->dim != hs2::kLatentRot) return HS2_ERR_ARG;
  if (Hq < 0) return HS2_ERR_ARG;
  bool go;
  const hs2_status st = check_latent_rows(kv, c_rows, c_stride, r_rows, r_stride, row_dtype, row_start, n_rows, &go);
  if (!go) return st;
  if ((Hq > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr)) return HS2_ERR_ARG;
  if (q) {
    // heads apart from one another, rows apart from one another
    auto apart = [&](const void* p, int64_t stride, int64_t head, hs2_dtype t) {
      return rows16(p, stride, t) && head * elem_bytes(t) % 16 == 0 && head >= hs2::kLatentRot && head <= kMaxStride &&
             stride >= (Hq - 1) * head + hs2::kLatentRot && stride <= kMaxStride;
    };
    if (Hq > 65535 || !apart(q, q_stride, q_head, row_dtype) || !apart(q_out, q_out_stride, q_out_head, kv->dtype))
      return HS2_ERR_ARG;
    if (q == q_out && (kv->dtype != row_dtype || q_stride != q_out_stride || q_head != q_out_head)) return HS2_ERR_ARG;
  }
  hs2::LatentRowsArgs z{};
  z.rot = rot_table(rot);
  z.q = q;
  z.q_out = q_out;
  z.q_stride = q_stride;
  z.q_head = q_head;
  z.q_out_stride = q_out_stride;
  z.q_out_head = q_out_head;
  z.Hq = Hq;
  return latent_rows(kv, c_rows, c_stride, r_rows, r_stride, row_dtype, row_start, n_rows, z, true, dev_err, stream);
}

hs2_status hs2_latent_read(const hs2_kv* kv, void* c_rows, int64_t c_stride, void* r_rows, int64_t r_stride,
                           hs2_dtype row_dtype, const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream) {
  bool go;
  const hs2_status st = check_latent_rows(kv, c_rows, c_stride, r_rows, r_stride, row_dtype, row_start, n_rows, &go);
  if (!go) return st;
  hs2::LatentRowsArgs z{};
  return latent_rows(kv, c_rows, c_stride, r_rows, r_stride, row_dtype, row_start, n_rows, z, false, dev_err, stream);
}

size_t hs2_latent_chunk_workspace(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t) {
  if (!valid_latent(kv) || n_rows < 0 || max_n < 0 || max_t < 0 || Hq < 1 || !heads_supported(Hq)) return 0;
  size_t need = 256;
  // narrower units are more: what a call with fewer tokens a sequence would take, too
  const long long top = (long long)std::min(max_n, n_rows) * Hq;
  const int widest = chunk_width(top);
  for (int w = 16; kv->dtype != HS2_F32 && w <= widest; w *= 2)
    if (Hq <= w) need = std::max(need, chunk_layout(n_rows, Hq, kv, w, max_t, top).total);
  return need;
}

hs2_status hs2_latent_chunk(const void* q, const int32_t* row_start, int n_rows, int max_n, int Hq, const hs2_kv* kv,
                            int max_t, float scale, void* o, hs2_dtype o_dtype, float* lse, void* workspace,
                            size_t ws_bytes, int32_t* dev_err, void* stream) {
  if (!valid_latent(kv) || !row_start || Hq < 1 || !valid_attention(n_rows, max_n, max_t, scale, o_dtype))
    return HS2_ERR_ARG;
  if (low_precision(kv) || !heads_supported(Hq)) return HS2_ERR_UNSUPPORTED;
  if ((long long)max_t > (long long)kv->max_pages * 64) return HS2_ERR_ARG;
  if (n_rows == 0 || max_n == 0) return HS2_OK;
  if (!q || !aligned16(q) || !o || !aligned16(o)) return HS2_ERR_ARG;
  const int dc = kv->d - hs2::kLatentRot;
  const long long top = (long long)std::min(max_n, n_rows) * Hq;  // rows of a sequence
  Layout L = chunk_layout(n_rows, Hq, kv, chunk_width(top), max_t, top);
  // 32-bit tile counts and pool rows
  if (kv->dtype != HS2_F32 && (L.tiles > 1LL << 30 || (long long)kv->num_pages * 64 > 0x7fffffff - 64 || kv->max_pages > (1 << 24)))
    return HS2_ERR_UNSUPPORTED;
  if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < (kv->dtype == HS2_F32 ? 256 : L.total)) return HS2_ERR_ARG;
  hs2::ChunkArgs a = chunk_args(q, row_start, n_rows, max_n, max_t, kv->batch, Hq, scale, o, o_dtype, lse, dev_err);
  a.k = kv->k;
  a.bt = kv->block_table;
  a.seq_len = kv->seq_len;
  a.num_pages = kv->num_pages;
  a.max_pages = kv->max_pages;
  a.Hkv = 1;
  a.G = Hq;
  while ((1 << a.log2G) < a.G) ++a.log2G;
  cudaStream_t s = (cudaStream_t)stream;
  if (kv->dtype == HS2_F32) {
    const cudaError_t e = hs2::launch_latent_cc(a, {}, dc, s);
    return e == cudaSuccess ? HS2_OK : cuda_fail(e);
  }
  bind(L, (char*)workspace);
  const int width = std::min(64, L.plan.tile_rows), box_heads = std::min(Hq, width);  // rows and heads of a CTA
  CUtensorMap tq, tk;
  if (!encode_3d_bf16(&tq, q, kv->d, (uint64_t)Hq, (uint64_t)n_rows, box_heads, width / box_heads) ||
      !encode_2d_bf16(&tk, kv->k, kv->d, (uint64_t)kv->num_pages * 64, 64))
    return HS2_ERR_ARG;
  cudaError_t e = L.plan.own ? cudaSuccess : hs2::launch_chunk_plan(a, &L.plan, 1, s);
  if (e == cudaSuccess) e = hs2::launch_latent_chunk(tq, tk, a, L.plan, dc, s);
  if (e == cudaSuccess && L.plan.snap) e = hs2::launch_chunk_merge(a, &L.plan, 1, dc, s);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

size_t hs2_latent_prefill_workspace(int n_rows, int Hq, int batch, int max_n, int max_t) {
  if (n_rows < 0 || Hq < 1 || batch < 1 || max_n < 0 || max_t < 0) return 0;
  return prefill_layout(n_rows, Hq, batch, max_t).total;
}

hs2_status hs2_latent_prefill(const void* q, const int32_t* row_start, int n_rows, int max_n, int Hq, int batch,
                              const hs2_latent_keys* keys, int max_t, float scale, void* o, hs2_dtype o_dtype, float* lse,
                              void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream) {
  if (!row_start || !keys || Hq < 1 || batch < 1 || !valid_attention(n_rows, max_n, max_t, scale, o_dtype) ||
      !row_type(keys->dtype) || !keys->key_start || keys->n_keys < 0)
    return HS2_ERR_ARG;
  if (n_rows == 0 || max_n == 0) return HS2_OK;
  if (!q || !aligned16(q) || !o || !aligned16(o)) return HS2_ERR_ARG;
  if (keys->n_keys > 0) {
    auto strided = [&](const void* p, int64_t token, int64_t head, int width) {
      return rows16(p, token, keys->dtype) && head * elem_bytes(keys->dtype) % 16 == 0 && head >= width &&
             head <= kMaxStride && token >= width && token <= kMaxStride;
    };
    if (!strided(keys->k, keys->k_token, keys->k_head, hs2::kLatentNope) ||
        !strided(keys->v, keys->v_token, keys->v_head, hs2::kLatentValue) ||
        !strided(keys->r, keys->r_token, hs2::kLatentRot, hs2::kLatentRot))
      return HS2_ERR_ARG;
  }
  const bool f32 = keys->dtype == HS2_F32;
  Layout L = prefill_layout(n_rows, Hq, batch, max_t);
  // grid y; 32-bit tile counts and rows
  if (Hq > 65535 || (!f32 && (L.tiles > 1LL << 30 || keys->n_keys > 0x7fffffff - 256))) return HS2_ERR_UNSUPPORTED;
  if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < (f32 ? 256 : L.total)) return HS2_ERR_ARG;
  hs2::ChunkArgs a = chunk_args(q, row_start, n_rows, max_n, max_t, batch, Hq, scale, o, o_dtype, lse, dev_err);
  a.Hkv = Hq;
  a.G = 1;
  a.k = keys->k;
  a.v = keys->v;
  a.key_start = keys->key_start;
  a.n_keys = keys->n_keys;
  const hs2::LatentKeys lk{keys->r, keys->k_token, keys->k_head, keys->v_token, keys->v_head, keys->r_token};
  cudaStream_t s = (cudaStream_t)stream;
  if (f32 || keys->n_keys == 0) {  // (no keys: nothing but what there is to flag)
    const cudaError_t e = hs2::launch_latent_cc(a, lk, 0, s);
    return e == cudaSuccess ? HS2_OK : cuda_fail(e);
  }
  bind(L, (char*)workspace);
  const uint64_t nk = keys->n_keys;
  CUtensorMap tq, tk, tr, tv;
  if (!encode_3d_bf16(&tq, q, 192, (uint64_t)Hq, (uint64_t)n_rows, 1, 128) ||
      !encode_3d_bf16(&tk, keys->k, 128, (uint64_t)Hq, nk, 1, 128, keys->k_head, keys->k_token) ||
      !encode_3d_bf16(&tr, keys->r, 64, 1, nk, 1, 128, keys->r_token, keys->r_token) ||
      !encode_3d_bf16(&tv, keys->v, 128, (uint64_t)Hq, nk, 1, 64, keys->v_head, keys->v_token))
    return HS2_ERR_ARG;
  cudaError_t e = L.plan.own ? cudaSuccess : hs2::launch_chunk_plan(a, &L.plan, 1, s);
  if (e == cudaSuccess) e = hs2::launch_latent_prefill(tq, tk, tr, tv, a, L.plan, s);
  if (e == cudaSuccess && L.plan.snap) e = hs2::launch_chunk_merge(a, &L.plan, 1, hs2::kLatentValue, s);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e);
}

}  // extern "C"
