// rot_rows.cu — rows of a ragged batch into a paged cache with K, and the queries beside them,
// rotated by their positions on the way (rot.cuh), and the rows of a latent cache.
//
// Bound by the bytes: rows in, codes and queries out; a program that rotates first writes and reads
// Q and K once more. A warp has a row (or two): it looks the row's place up once, loads the
// table's cos and sin once into registers (a lane keeps its channels from head to head), and takes
// the heads of K and V and then those of Q, 512 channels a step and of Q two steps' loads at a time.
// 32768 rows of 32 heads over 4, d = 128, bf16 to FP8 (653 MB): 120 us, 0.80 of the copy bandwidth; with K, V
// and Q in one loop 163 (16 warps an SM: the registers of the quantisation), with more warps at fewer
// registers 148 and 167. The same to FP4 123, without the queries 43. 26273 latent rows of 512 + 64 with 32
// heads (282 MB): 60 us, 0.69; HBM is 47 % busy, a third of the warps fit and wait for their loads, and at the 80
// registers that three blocks an SM leave the two-row form spills (84 bytes stored and 40 loaded a thread, other
// types up to 164 and 120); the queries are 128 bytes a head at a stride of 384 in and 1152 out. 73 us with 16 channels
// in a row per lane.
#include "kv_rows.cuh"
#include "rot.cuh"

namespace hs2 {

namespace {

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

// grid (1 + rows / (8 TOK), splits of a row's steps). Block (0, 0) checks the row starts.
template <int D, int FMT, bool ROW_F32, int TOK>
__global__ void __launch_bounds__(kRowThreads, 2) kv_write_rot_kernel(const RotRowsArgs z) {
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
  const int kv_heads = a.v ? 2 * a.Hkv : a.Hkv, kv_steps = (kv_heads + HPS - 1) / HPS;
  const int steps = kv_steps + (z.Hq + HPS - 1) / HPS, per = (steps + gridDim.y - 1) / gridDim.y;
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
  // V as it lies; an FP4 cache's groups are 16 channels in a row
  constexpr bool FP4 = FMT == HS2_FP4_E2M1;
  const LaneChannels ch = lane_channels(z.rot, D, grp), cv{FP4 ? 16 * grp : 8 * grp, FP4 ? 16 * grp + 8 : D / 2 + 8 * grp, false};
#pragma unroll 1
  for (int k = 0; k < TOK; ++k) {
    const int pos = __shfl_sync(0xffffffffu, mine.pos, k), phys = __shfl_sync(0xffffffffu, mine.phys, k), r = r0 + k;
    if (pos < 0) continue;
    float cs[8], sn[8];
    if (ch.turn) load_angles(z.rot, pos, grp, cs, sn);
    int s = s0;
#pragma unroll 1
    for (; s < min(s1, kv_steps); ++s) {  // K and V
      const int head = s * HPS + sub;
      const bool is_k = head < a.Hkv;
      const int g = is_k ? head : head - a.Hkv;
      const LaneChannels c = is_k ? ch : cv;
      float x[16];
      if (head < kv_heads) {
        const void* rows = is_k ? a.k_rows : a.v_rows;
        const long long at = r * (is_k ? a.row_stride : z.v_stride) + g * D;
        load8<ROW_F32>(rows, at + c.lo, x);
        load8<ROW_F32>(rows, at + c.hi, x + 8);
        if (c.turn) rotate16(z.rot, cs, sn, x);
      }
      if (FP4 && s * HPS < a.Hkv) {
        // K's groups of 16 channels in a row: neighbours swap, the even one takes the lower pieces' group
        const bool odd = grp & 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float got = __shfl_xor_sync(0xffffffffu, odd ? x[i] : x[8 + i], 1);
          if (is_k && odd) x[i] = got;
          if (is_k && !odd) x[8 + i] = got;
        }
      }
      if (head >= kv_heads) continue;
      const size_t slab = (size_t)phys * a.Hkv + g, line = slab * kPage + pos % kPage;
      if constexpr (FP4) {
        put16<D, FMT>(a, !is_k, slab, line, is_k ? (grp & 1 ? ch.hi - 8 : ch.lo) / 16 : grp, x);
      } else {
        void* pool = is_k ? a.k : a.v;
        if constexpr (FMT == HS2_FP8_E4M3) {
          uint32_t w[4];
          uint8_t* to = reinterpret_cast<uint8_t*>(pool) + line * D;
          if (!fp8_codes(a, (is_k ? a.k_scale : a.v_scale)[slab], x, w)) continue;
          *reinterpret_cast<uint2*>(to + c.lo) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(to + c.hi) = make_uint2(w[2], w[3]);
        } else {
          store8<FMT == HS2_F32>(pool, (long long)line * D + c.lo, x);
          store8<FMT == HS2_F32>(pool, (long long)line * D + c.hi, x + 8);
        }
      }
    }
#pragma unroll 1
    for (; s < s1; s += 2) {  // the queries, two steps' loads at a time
      float x[16], y[16];
      const int h0 = (s - kv_steps) * HPS + sub, h1 = h0 + HPS;
      const bool two = h1 < z.Hq && s + 1 < s1;
      const long long at = r * z.q_stride + h0 * D, to = r * z.q_out_stride + h0 * D;
      if (h0 < z.Hq) load8<ROW_F32>(z.q, at + ch.lo, x), load8<ROW_F32>(z.q, at + ch.hi, x + 8);
      if (two) load8<ROW_F32>(z.q, at + HPS * D + ch.lo, y), load8<ROW_F32>(z.q, at + HPS * D + ch.hi, y + 8);
      __syncwarp();  // they may be rotated in place: a head's lanes load before any stores
      if (ch.turn) rotate16(z.rot, cs, sn, x);
      if (ch.turn) rotate16(z.rot, cs, sn, y);
      if (h0 < z.Hq) store8<FMT == HS2_F32>(z.q_out, to + ch.lo, x), store8<FMT == HS2_F32>(z.q_out, to + ch.hi, x + 8);
      if (two)
        store8<FMT == HS2_F32>(z.q_out, to + HPS * D + ch.lo, y), store8<FMT == HS2_F32>(z.q_out, to + HPS * D + ch.hi, y + 8);
    }
  }
}

// A latent cache's row is DC channels as they are and 64 that are rotated; the queries' 64 rotated
// channels go to their place. grid as above; step 0 takes the row itself, step s > 0 queries.
template <int DC, bool CACHE_F32, bool ROW_F32, int TOK>
__global__ void __launch_bounds__(kRowThreads, 3) latent_write_kernel(const LatentRowsArgs z) {
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
  const LaneChannels ch = lane_channels(z.rot, kLatentRot, grp);
#pragma unroll 1
  for (int k = 0; k < TOK; ++k) {
    const int pos = __shfl_sync(0xffffffffu, mine.pos, k), phys = __shfl_sync(0xffffffffu, mine.phys, k), r = r0 + k;
    if (pos < 0) continue;
    float cs[8], sn[8];
    load_angles(z.rot, pos, grp, cs, sn);
    const long long line = ((long long)phys * kPage + pos % kPage) * (DC + kLatentRot);
    int s = s0;
    if (s == 0) {
      float x[16], y[16];
      const bool in_c = lane < DC / 16, in_r = lane < GPR;
      const long long cat = r * z.c_stride + 8 * lane, rat = r * z.r_stride;
      if (in_c) load8<ROW_F32>(z.c_rows, cat, x), load8<ROW_F32>(z.c_rows, cat + DC / 2, x + 8);
      if (in_r) load8<ROW_F32>(z.r_rows, rat + ch.lo, y), load8<ROW_F32>(z.r_rows, rat + ch.hi, y + 8);
      if (in_c) store8<CACHE_F32>(a.k, line + 8 * lane, x), store8<CACHE_F32>(a.k, line + 8 * lane + DC / 2, x + 8);
      if (in_r) {
        rotate16(z.rot, cs, sn, y);
        store8<CACHE_F32>(a.k, line + DC + ch.lo, y);
        store8<CACHE_F32>(a.k, line + DC + ch.hi, y + 8);
      }
      ++s;
    }
    auto fetch = [&](int s, float (&x)[16]) {
      const int head = (s - 1) * HPS + sub;
      if (head >= z.Hq) return;
      const long long at = r * z.q_stride + head * z.q_head;
      load8<ROW_F32>(z.q, at + ch.lo, x);
      load8<ROW_F32>(z.q, at + ch.hi, x + 8);
    };
    auto finish = [&](int s, float (&x)[16]) {
      const int head = (s - 1) * HPS + sub;
      rotate16(z.rot, cs, sn, x);
      if (head >= z.Hq) return;
      const long long at = r * z.q_out_stride + head * z.q_out_head;
      store8<CACHE_F32>(z.q_out, at + ch.lo, x);
      store8<CACHE_F32>(z.q_out, at + ch.hi, x + 8);
    };
#pragma unroll 1
    for (; s < s1; s += 2) {
      float x[16], y[16];
      fetch(s, x);
      if (s + 1 < s1) fetch(s + 1, y);
      __syncwarp();  // q may be rotated in place: a head's lanes load before any stores
      finish(s, x);
      if (s + 1 < s1) finish(s + 1, y);
    }
  }
}

// Rows of a latent cache back to arrays: a warp has a row at a time, 16 channels a lane.
template <int DC, bool CACHE_F32, bool ROW_F32, int TOK>
__global__ void __launch_bounds__(kRowThreads, 3) latent_read_kernel(const LatentRowsArgs z) {
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
    const bool in_c = lane < DC / 16, in_r = lane < kLatentRot / 16;
    void *c = const_cast<void*>(z.c_rows), *rr = const_cast<void*>(z.r_rows);
    const long long cat = r * z.c_stride + 8 * lane, rat = r * z.r_stride + 8 * lane, at = line + 8 * lane;
    if (in_c) load8<CACHE_F32>(a.k, at, x), load8<CACHE_F32>(a.k, at + DC / 2, x + 8);
    if (in_r) load8<CACHE_F32>(a.k, at + DC, y), load8<CACHE_F32>(a.k, at + DC + 32, y + 8);
    if (in_c) store8<ROW_F32>(c, cat, x), store8<ROW_F32>(c, cat + DC / 2, x + 8);
    if (in_r) store8<ROW_F32>(rr, rat, y), store8<ROW_F32>(rr, rat + 32, y + 8);
  }
}

namespace {

// Rows of a warp and splits of a row's steps: few rows are spread over a warp a step, of many a warp has
// two whole ones (32768 rows 120 us; with one 124, with eight 124). Spread and whole, by rows times steps:
//   K, V and 32 heads over 4, d = 128 (10 steps): 256 rows 4.4 and 9.0 us, 1024 9.0 and 9.9, 2048 15.6 and 10.7,
//   8192 68 and 34. Latent rows with 32 heads (5 steps): 1024 rows 4.9 and 7.4, 2048 7.0 and 8.9, 4096 12.1 and
//   10.7, 16384 55 and 44. Reading (no steps to spread) 256 rows 2.3 and 2.5, 4096 3.1 and 3.3, 8192 4.1 and 3.6.
constexpr long long kManySteps = 14000;
constexpr int kReadSteps = 2;  // what a row of the reading counts as
constexpr int kRowsPerWarp = 2;

dim3 row_grid(int n_rows, int tok, int splits) {
  const int per = kRowThreads / 32 * tok;
  return dim3((n_rows + per - 1) / per + 1, splits);
}

template <int D, int FMT, bool ROW_F32>
cudaError_t launch_rot(const RotRowsArgs& z, cudaStream_t s) {
  const int hps = 512 / D, steps = ((z.rows.v ? 2 : 1) * z.rows.Hkv + hps - 1) / hps + (z.Hq + hps - 1) / hps;
  if ((long long)z.rows.n_rows * steps >= kManySteps)
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
  const bool many = (long long)n * (write ? steps : kReadSteps) >= kManySteps;
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
