// rot_rows.cu — rows of a ragged batch into a paged cache with K, and the queries beside them,
// rotated by their positions on the way (rot.cuh), and the rows of a latent cache.
//
// Bound by the bytes: rows in, codes and queries out; a program that rotates first writes and reads
// Q and K once more. A warp has a row (or several): it looks the row's place up once, loads the
// table's cos and sin once into registers (a lane keeps its channels from head to head), and takes
// the heads of K, V and Q, 512 channels a step.
#include "kv_rows.cuh"
#include "rot.cuh"

namespace hs2 {

namespace {

// load16 without the read-only path: q may be rotated in place
template <bool F32>
HS2_DEVI void load16_rw(const void* rows, long long at, float (&x)[16]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = p[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = p[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) x[8 * i + 2 * j] = bf16_lo(w[j]), x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// Where row r is: its position (-1: nowhere, or flagged), and the physical page.
struct RowSpot {
  int pos, phys;
};
HS2_DEVI RowSpot row_spot(const RowsArgs& a, const RotTable& rot, int r, int n_le, bool flags) {
  RowSpot s{-1, -1};
  if (r >= a.n_rows) return s;
  const RowPlace pl = row_place(a.row_start, a.seq_len, a.batch, a.max_pages, a.n_rows, r, n_le);
  if (pl.b < 0) return s;
  int bad = 0;
  if (pl.pos < 0) bad = HS2_DEV_BAD_LENGTH;
  else if (rot.table && pl.pos >= rot.n_pos) bad = HS2_DEV_BAD_INDEX;
  else {
    const int phys = a.bt[(size_t)pl.b * a.max_pages + pl.pos / kPage];
    if (phys < 0 || phys >= a.num_pages) bad = HS2_DEV_BAD_PAGE;
    else s.pos = pl.pos, s.phys = phys;
  }
  if (bad && flags) flag_error(a.dev_err, bad);
  return s;
}

// The places of TOK rows from r0 on: lane k < TOK has row r0 + k's.
template <int TOK>
HS2_DEVI RowSpot warp_spots(const RowsArgs& a, const RotTable& rot, int r0, bool flags) {
  const int lane = threadIdx.x & 31;
  int n[TOK], n_le = 0;
  warp_rows_at_most<TOK>(a.row_start, a.batch, r0, n);
#pragma unroll
  for (int k = 0; k < TOK; ++k)
    if (k == lane) n_le = n[k];
  return lane < TOK ? row_spot(a, rot, r0 + lane, n_le, flags) : RowSpot{-1, -1};
}

}  // namespace

// grid (1 + rows / (8 TOK), splits of a row's heads). Block (0, 0) checks the row starts.
template <int D, int FMT, bool ROW_F32, int TOK>
__global__ void __launch_bounds__(kRowThreads) kv_write_rot_kernel(const RotRowsArgs z) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int GPR = D / 16, HPS = 32 / GPR;  // lanes of a head; heads of a step
  const RowsArgs& a = z.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane % GPR, sub = lane / GPR;
  if (blockIdx.x == 0) {
    check_starts(a);
    return;
  }
  const int r0 = ((blockIdx.x - 1) * (kRowThreads / 32) + warp) * TOK;
  if (r0 >= a.n_rows) return;
  const RowSpot mine = warp_spots<TOK>(a, z.rot, r0, blockIdx.y == 0);
  const int kv_heads = a.v ? 2 * a.Hkv : a.Hkv, heads = kv_heads + z.Hq;
  const int steps = (heads + HPS - 1) / HPS, per = (steps + gridDim.y - 1) / gridDim.y;
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
  const bool in_rot = 16 * grp < z.rot.dim;
#pragma unroll 1
  for (int k = 0; k < TOK; ++k) {
    const int pos = __shfl_sync(0xffffffffu, mine.pos, k), phys = __shfl_sync(0xffffffffu, mine.phys, k), r = r0 + k;
    if (pos < 0) continue;
    float cs[16], sn[16];
    if (in_rot) load_angles(z.rot, pos, grp, cs, sn);
#pragma unroll 2
    for (int s = s0; s < s1; ++s) {
      const int head = s * HPS + sub, g = head < a.Hkv ? head : head - a.Hkv;
      const bool is_q = head >= kv_heads && head < heads, is_v = head >= a.Hkv && head < kv_heads;
      float x[16];
      if (head < a.Hkv) load16<ROW_F32>(a.k_rows, (long long)r * a.row_stride + g * D + 16 * grp, x);
      else if (is_v) load16<ROW_F32>(a.v_rows, (long long)r * z.v_stride + g * D + 16 * grp, x);
      else if (is_q) load16_rw<ROW_F32>(z.q, (long long)r * z.q_stride + (head - kv_heads) * D + 16 * grp, x);
      rotate16(z.rot, grp, in_rot && !is_v, cs, sn, x);  // (lanes without a head rotate what they have)
      if (is_q) {
        store16<FMT == HS2_F32>(z.q_out, (long long)r * z.q_out_stride + (head - kv_heads) * D + 16 * grp, x);
      } else if (head < kv_heads) {
        const size_t slab = (size_t)phys * a.Hkv + g;
        put16<D, FMT>(a, is_v, slab, slab * kPage + pos % kPage, grp, x);
      }
    }
  }
}

// A latent cache's row is DC channels as they are and 64 that are rotated; the queries' 64 rotated
// channels go to their place. grid as above; step 0 takes the row itself, step s > 0 queries.
template <int DC, bool CACHE_F32, bool ROW_F32, int TOK>
__global__ void __launch_bounds__(kRowThreads) latent_write_kernel(const LatentRowsArgs z) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int GPR = kLatentRot / 16, HPS = 32 / GPR;
  const RowsArgs& a = z.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane % GPR, sub = lane / GPR;
  if (blockIdx.x == 0) {
    check_starts(a);
    return;
  }
  const int r0 = ((blockIdx.x - 1) * (kRowThreads / 32) + warp) * TOK;
  if (r0 >= a.n_rows) return;
  const RowSpot mine = warp_spots<TOK>(a, z.rot, r0, blockIdx.y == 0);
  const int steps = 1 + (z.Hq + HPS - 1) / HPS, per = (steps + gridDim.y - 1) / gridDim.y;
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
#pragma unroll 1
  for (int k = 0; k < TOK; ++k) {
    const int pos = __shfl_sync(0xffffffffu, mine.pos, k), phys = __shfl_sync(0xffffffffu, mine.phys, k), r = r0 + k;
    if (pos < 0) continue;
    float cs[16], sn[16];
    load_angles(z.rot, pos, grp, cs, sn);
    const long long line = ((long long)phys * kPage + pos % kPage) * (DC + kLatentRot);
#pragma unroll 2
    for (int s = s0; s < s1; ++s) {
      float x[16];
      if (s == 0) {
        if (lane < DC / 16) {
          load16<ROW_F32>(z.c_rows, (long long)r * z.c_stride + 16 * lane, x);
          store16<CACHE_F32>(a.k, line + 16 * lane, x);
        }
        if (lane < GPR) load16<ROW_F32>(z.r_rows, (long long)r * z.r_stride + 16 * lane, x);
        rotate16(z.rot, grp, true, cs, sn, x);
        if (lane < GPR) store16<CACHE_F32>(a.k, line + DC + 16 * lane, x);
        continue;
      }
      const int head = (s - 1) * HPS + sub;
      const bool have = head < z.Hq;
      if (have) load16_rw<ROW_F32>(z.q, (long long)r * z.q_stride + head * z.q_head + 16 * grp, x);
      rotate16(z.rot, grp, true, cs, sn, x);
      if (have) store16<CACHE_F32>(z.q_out, (long long)r * z.q_out_stride + head * z.q_out_head + 16 * grp, x);
    }
  }
}

// Rows of a latent cache back to arrays: a warp has a row at a time, 16 channels a lane.
template <int DC, bool CACHE_F32, bool ROW_F32, int TOK>
__global__ void __launch_bounds__(kRowThreads) latent_read_kernel(const LatentRowsArgs z) {
  griddep_launch_dependents();
  griddep_wait();
  const RowsArgs& a = z.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    check_starts(a);
    return;
  }
  const int r0 = ((blockIdx.x - 1) * (kRowThreads / 32) + warp) * TOK;
  if (r0 >= a.n_rows) return;
  const RowSpot mine = warp_spots<TOK>(a, RotTable{}, r0, true);
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    const int pos = __shfl_sync(0xffffffffu, mine.pos, k), phys = __shfl_sync(0xffffffffu, mine.phys, k), r = r0 + k;
    if (pos < 0) continue;
    const long long line = ((long long)phys * kPage + pos % kPage) * (DC + kLatentRot);
    float x[16], y[16];
    if (lane < DC / 16) load16<CACHE_F32>(a.k, line + 16 * lane, x);
    if (lane < kLatentRot / 16) load16<CACHE_F32>(a.k, line + DC + 16 * lane, y);
    if (lane < DC / 16) store16<ROW_F32>(const_cast<void*>(z.c_rows), (long long)r * z.c_stride + 16 * lane, x);
    if (lane < kLatentRot / 16) store16<ROW_F32>(const_cast<void*>(z.r_rows), (long long)r * z.r_stride + 16 * lane, y);
  }
}

namespace {

// Rows of a warp and splits of a row's heads: few rows are spread over as many warps as there are steps.
constexpr int kManyRows = 4096;
constexpr int kRowsPerWarp = 4;

dim3 row_grid(int n_rows, int tok, int splits) {
  const int per = kRowThreads / 32 * tok;
  return dim3((n_rows + per - 1) / per + 1, splits);
}

template <int D, int FMT, bool ROW_F32>
cudaError_t launch_rot(const RotRowsArgs& z, cudaStream_t s) {
  const int hps = 512 / D, steps = ((z.rows.v ? 2 : 1) * z.rows.Hkv + z.Hq + hps - 1) / hps;
  if (z.rows.n_rows >= kManyRows)
    return launch_pdl(kv_write_rot_kernel<D, FMT, ROW_F32, kRowsPerWarp>, row_grid(z.rows.n_rows, kRowsPerWarp, 1),
                      dim3(kRowThreads), 0, s, z);
  return launch_pdl(kv_write_rot_kernel<D, FMT, ROW_F32, 1>, row_grid(z.rows.n_rows, 1, steps < 65535 ? steps : 65535),
                    dim3(kRowThreads), 0, s, z);
}

template <int D>
cudaError_t launch_rot_d(const RotRowsArgs& z, int dtype, bool row_f32, cudaStream_t s) {
  switch (dtype) {
    case HS2_F32: return row_f32 ? launch_rot<D, HS2_F32, true>(z, s) : launch_rot<D, HS2_F32, false>(z, s);
    case HS2_BF16: return row_f32 ? launch_rot<D, HS2_BF16, true>(z, s) : launch_rot<D, HS2_BF16, false>(z, s);
    case HS2_FP8_E4M3: return row_f32 ? launch_rot<D, HS2_FP8_E4M3, true>(z, s) : launch_rot<D, HS2_FP8_E4M3, false>(z, s);
    case HS2_FP4_E2M1: return row_f32 ? launch_rot<D, HS2_FP4_E2M1, true>(z, s) : launch_rot<D, HS2_FP4_E2M1, false>(z, s);
  }
  return cudaErrorInvalidValue;
}

template <int DC, bool CACHE_F32, bool ROW_F32>
cudaError_t launch_latent(const LatentRowsArgs& z, bool write, cudaStream_t s) {
  const int n = z.rows.n_rows, steps = 1 + (z.Hq + 7) / 8;
  const bool many = n >= kManyRows;
  auto kern = write ? (many ? latent_write_kernel<DC, CACHE_F32, ROW_F32, kRowsPerWarp> : latent_write_kernel<DC, CACHE_F32, ROW_F32, 1>)
                    : (many ? latent_read_kernel<DC, CACHE_F32, ROW_F32, kRowsPerWarp> : latent_read_kernel<DC, CACHE_F32, ROW_F32, 1>);
  return launch_pdl(kern, row_grid(n, many ? kRowsPerWarp : 1, many || !write ? 1 : steps), dim3(kRowThreads), 0, s, z);
}

}  // namespace

cudaError_t launch_kv_write_rot(const RotRowsArgs& z, int d, int dtype, bool row_f32, cudaStream_t s) {
  return d == 128 ? launch_rot_d<128>(z, dtype, row_f32, s) : launch_rot_d<64>(z, dtype, row_f32, s);
}

cudaError_t launch_latent_rows(const LatentRowsArgs& z, int dc, bool cache_f32, bool row_f32, bool write, cudaStream_t s) {
  if (dc == 512) {
    if (cache_f32) return row_f32 ? launch_latent<512, true, true>(z, write, s) : launch_latent<512, true, false>(z, write, s);
    return row_f32 ? launch_latent<512, false, true>(z, write, s) : launch_latent<512, false, false>(z, write, s);
  }
  if (cache_f32) return row_f32 ? launch_latent<256, true, true>(z, write, s) : launch_latent<256, true, false>(z, write, s);
  return row_f32 ? launch_latent<256, false, true>(z, write, s) : launch_latent<256, false, false>(z, write, s);
}

}  // namespace hs2
