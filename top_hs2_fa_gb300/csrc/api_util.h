// api_util.h — host-side helpers of the extern "C" boundary: argument checks, error state,
// workspace arithmetic and tensor maps.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hs2.h"

namespace hs2 {
namespace api {

// The cudaError_t of the calling thread's last HS2_ERR_CUDA.
inline int& last_cuda_error() {
  static thread_local int e = 0;
  return e;
}
inline hs2_status cuda_fail(cudaError_t e) {
  last_cuda_error() = (int)e;
  (void)cudaGetLastError();  // clear the sticky-free error state of the calling thread
  return HS2_ERR_CUDA;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

inline bool valid_kv(const hs2_kv* kv, bool need_v) {
  if (!kv || !kv->k || !kv->block_table || !kv->seq_len) return false;
  if (need_v && !kv->v) return false;
  if (kv->batch < 1 || kv->num_pages < 1 || kv->max_pages < 1 || kv->Hkv < 1) return false;
  if (kv->page_size != 64) return false;
  if (kv->d != 64 && kv->d != 128) return false;
  if (kv->dtype != HS2_F32 && kv->dtype != HS2_BF16 && kv->dtype != HS2_FP8_E4M3 && kv->dtype != HS2_FP4_E2M1)
    return false;
  if ((kv->dtype == HS2_FP8_E4M3 || kv->dtype == HS2_FP4_E2M1) && (!kv->k_scale || (need_v && !kv->v_scale)))
    return false;
  if (kv->dtype == HS2_FP4_E2M1 && (!kv->k_sf || !aligned16(kv->k_sf) || (need_v && (!kv->v_sf || !aligned16(kv->v_sf)))))
    return false;
  if (!aligned16(kv->k) || (need_v && !aligned16(kv->v))) return false;
  return true;
}

// FP8 / FP4 caches (quantised codes with scales)
inline bool low_precision(const hs2_kv* kv) { return kv->dtype == HS2_FP8_E4M3 || kv->dtype == HS2_FP4_E2M1; }

inline bool pow2_le32(int g) { return g == 1 || g == 2 || g == 4 || g == 8 || g == 16 || g == 32; }

// 2-D bf16 tensor map: rows x cols (cols contiguous), box of 64 columns x box_rows rows,
// 128-byte swizzle. cuTensorMapEncodeTiled is fetched from the driver at run time so the
// library has no link-time dependency on libcuda.
// rows x cols bf16, tiles of box_rows x 64 in the 128-byte swizzle. row_step > 1: a view of
// every row_step-th row (rows / row_step view rows, row stride row_step * cols * 2 bytes).
inline bool encode_2d_bf16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows,
                    uint32_t row_step = 1) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
      (void)cudaGetLastError();
      return false;
    }
    encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
  }
  const cuuint64_t dims[2] = {cols, rows / row_step};
  const cuuint64_t strides[1] = {cols * 2 * row_step};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows x row_bytes bytes (32, 64 or 128), whole rows in tiles of box_rows, swizzled by the width.
inline bool encode_2d_bytes(CUtensorMap* map, const void* base, uint32_t row_bytes, uint64_t rows, uint32_t box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
      (void)cudaGetLastError();
      return false;
    }
    encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
  }
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {row_bytes, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                row_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                : row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                  : CU_TENSOR_MAP_SWIZZLE_32B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool encode_3d_bf16(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b1,
                    uint32_t b2) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
      (void)cudaGetLastError();
      return false;
    }
    encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
  }
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
  const cuuint32_t box[3] = {64, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace api
}  // namespace hs2
