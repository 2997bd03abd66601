// latent_cc.cu — latent attention on the CUDA cores: float32 caches and float32 expanded keys.
//
// x(s) = scale (q_n . k(s) + q_r . r(s)) over the row's visible keys, o = sum softmax(x) v, one pass with
// the running maximum and sum. Absorbed form: k(s) = v(s) = the DN latent channels of the paged
// cache's row, r(s) the 64 behind them. Expanded form: k and v of the head, r shared by the heads.
// A warp takes four keys at a time, two channels a lane and step. On the CUDA cores because the tensor
// cores have no fp32 product and float32 is kept for its exactness.
#include "chunk_plan.cuh"
#include "ragged.cuh"

namespace hs2 {

namespace {

constexpr int kLcWarps = 8;
constexpr int kLcKeys = 4;  // keys per warp step: their loads and reductions overlap

HS2_DEVI float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }

}  // namespace

// grid (rows, query heads), 8 warps over the row's keys, merged through shared memory.
template <int DN, int DV, bool PAGED>
__global__ void __launch_bounds__(kLcWarps * 32) latent_cc_kernel(const ChunkArgs a, const LatentKeys lk) {
  constexpr int DQ = DN + kLatentRot, NK = DN / 64, NV = DV / 64;  // steps of 64 channels
  __shared__ float sm_m[kLcWarps], sm_l[kLcWarps], sm_o[kLcWarps][DV];
  griddep_launch_dependents();
  griddep_wait();
  const int r = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n1[1];
  warp_rows_at_most<1>(a.row_start, a.batch, r, n1);
  if (r == 0 && h == 0 && warp == 0) {
    bool bad = warp_bad_starts(a.row_start, a.batch, a.n_rows);
    if (!PAGED)
      for (int b = lane; b < a.batch; b += 32) {
        const int k0 = a.key_start[b], k1 = a.key_start[b + 1];
        bad |= k1 != k0 && (k1 < k0 || k0 < 0 || k1 > a.n_keys);
      }
    if (bad) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
  }
  const int b = n1[0] - 1;
  if (b < 0 || b >= a.batch) return;
  const int r0 = a.row_start[b], r1 = a.row_start[b + 1], n = r1 - r0;
  if (r < r0 || r >= r1) return;
  const int key0 = PAGED ? 0 : a.key_start[b], t = PAGED ? a.seq_len[b] : a.key_start[b + 1] - key0;
  if (r0 < 0 || r1 > a.n_rows || n > a.max_n || t < n || t > a.max_t || (!PAGED && (key0 < 0 || key0 > a.n_keys - t))) {
    if (threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
    return;
  }
  const int pos = t - n + (r - r0);
  const int32_t* bt = PAGED ? a.bt + (size_t)b * a.max_pages : nullptr;
  const float* qp = reinterpret_cast<const float*>(a.q) + ((size_t)r * a.Hq + h) * DQ + 2 * lane;
  float2 q[NK + 1];
#pragma unroll
  for (int i = 0; i <= NK; ++i) q[i] = load2(qp + 64 * i);
  float m = -INFINITY, l = 0.f;
  float2 o[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = make_float2(0.f, 0.f);
  for (int s0 = warp * kLcKeys; s0 <= pos; s0 += kLcWarps * kLcKeys) {
    float x[kLcKeys];
    const float* vp[kLcKeys];
#pragma unroll
    for (int j = 0; j < kLcKeys; ++j) {
      x[j] = -INFINITY;
      vp[j] = nullptr;
      const int s = s0 + j;
      if (s > pos) continue;
      const float *kp, *rp;
      if (PAGED) {
        const int phys = bt[s / kPage];
        if (phys < 0 || phys >= a.num_pages) {
          if (lane == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
          continue;
        }
        kp = reinterpret_cast<const float*>(a.k) + ((size_t)phys * kPage + s % kPage) * DQ + 2 * lane;
        rp = kp + DN;
        vp[j] = kp;
      } else {
        kp = reinterpret_cast<const float*>(a.k) + (long long)(key0 + s) * lk.k_token + h * lk.k_head + 2 * lane;
        rp = reinterpret_cast<const float*>(lk.r) + (long long)(key0 + s) * lk.r_token + 2 * lane;
        vp[j] = reinterpret_cast<const float*>(a.v) + (long long)(key0 + s) * lk.v_token + h * lk.v_head + 2 * lane;
      }
      const float2 kr = load2(rp);
      float dot = fmaf(q[NK].x, kr.x, q[NK].y * kr.y);
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const float2 k = load2(kp + 64 * i);
        dot = fmaf(q[i].x, k.x, fmaf(q[i].y, k.y, dot));
      }
      x[j] = warp_sum(dot) * a.scale_log2;
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kLcKeys; ++j) mn = fmaxf(mn, x[j]);
    const float alpha = exp2_rel(m, mn);
    l *= alpha;
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i].x *= alpha, o[i].y *= alpha;
#pragma unroll
    for (int j = 0; j < kLcKeys; ++j) {
      if (!vp[j]) continue;
      const float p = x[j] != x[j] ? x[j] : exp2_rel(x[j], mn);  // the maximum leaves NaN out
      l += p;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float2 v = load2(vp[j] + 64 * i);
        o[i].x = fmaf(p, v.x, o[i].x), o[i].y = fmaf(p, v.y, o[i].y);
      }
    }
    m = mn;
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
  for (int i = 0; i < NV; ++i) sm_o[warp][64 * i + 2 * lane] = o[i].x, sm_o[warp][64 * i + 2 * lane + 1] = o[i].y;
  __syncthreads();
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int k = 0; k < kLcWarps; ++k) M = fmaxf(M, sm_m[k]);
  float f[kLcWarps];
#pragma unroll
  for (int k = 0; k < kLcWarps; ++k) {
    f[k] = exp2_rel(sm_m[k], M);
    // (a warp that has only seen NaN: its maximum is -inf)
    L += sm_l[k] != sm_l[k] ? sm_l[k] : f[k] * sm_l[k];
  }
  const size_t at = (size_t)r * a.Hq + h;
  for (int c = threadIdx.x; c < DV; c += kLcWarps * 32) {
    float O = 0.f;
#pragma unroll
    for (int k = 0; k < kLcWarps; ++k) O = fmaf(f[k], sm_o[k][c], O);
    const float out = chunk_factor(L != L ? L : O, L);
    if (a.o_bf16) reinterpret_cast<__nv_bfloat16*>(a.o)[at * DV + c] = __float2bfloat16(out);
    else reinterpret_cast<float*>(a.o)[at * DV + c] = out;
  }
  if (a.lse && threadIdx.x == 0) a.lse[at] = chunk_lse(L, M);
}

cudaError_t launch_latent_cc(const ChunkArgs& a, const LatentKeys& lk, int dc, cudaStream_t s) {
  auto kern = !a.bt ? latent_cc_kernel<kLatentNope, kLatentValue, false>
                    : dc == 512 ? latent_cc_kernel<512, 512, true> : latent_cc_kernel<256, 256, true>;
  return launch_pdl(kern, dim3(a.n_rows, a.Hq), dim3(kLcWarps * 32), 0, s, a, lk);
}

}  // namespace hs2
