// attn_tc_host.h -- host side of the tcgen05 attention kernel's launches: ring depths, tensor maps,
// shared-memory opt-in.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "api_common.h"
#include "attn_tc.cuh"

namespace ra {

// K ring / V ring depths: the tensor core waits on K first, so K gets the deeper ring.
template <int D>
constexpr int k_stages() { return D == 128 ? 3 : 4; }
template <int D>
constexpr int v_stages() { return D == 128 ? 2 : 4; }

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 2-D view [rows, head_dim] of a bf16 array whose rows are head_dim contiguous elements, read as
// one 64-element (128-byte, 128B-swizzled) column block of 1 row: the box a TMA gather4 takes.
inline ra_status row_gather_map(CUtensorMap* map, const void* base, int64_t rows, int32_t head_dim) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (rows <= 0 || rows > INT32_MAX) return fail(RA_ERR_UNSUPPORTED, "%lld rows exceed a TMA row coordinate", (long long)rows);
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim) * 2};
  cuuint32_t box[2] = {64, 1};
  cuuint32_t elem[2] = {1, 1};
  CUresult cr = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, elem,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled(rows) failed (%d)", static_cast<int>(cr));
  return RA_OK;
}

// Opt the kernel into its dynamic shared memory and check that it was compiled to the per-thread
// register count its setmaxnreg split is balanced against (a split above the block's launch
// allocation would leave the softmax warps waiting for registers that never come).
template <int PASS, typename Kern>
ra_status set_smem(Kern kern, int bytes, bool* configured, int device) {
  if (configured[device]) return RA_OK;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cudaFuncGetAttributes(attn_tc): %s", cudaGetErrorString(e));
  if (fa.numRegs != tc::Roles<PASS>::kLaunchRegs)
    return fail(RA_ERR_UNSUPPORTED, "attn_tc kernel compiled to %d registers per thread, its register split needs %d",
                fa.numRegs, tc::Roles<PASS>::kLaunchRegs);
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cudaFuncSetAttribute(attn_tc): %s", cudaGetErrorString(e));
  configured[device] = true;
  return RA_OK;
}

// q [total_q][Hq][D] as tiles of 128 / G tokens x the G heads of a kv head x 64 dims.
inline ra_status query_tile_map(CUtensorMap* qmap, const void* q, int64_t total_q, int32_t hq, int32_t head_dim,
                                int32_t group) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  // q viewed as [total_q][Hq][D]; one box = 128/G tokens x the G heads of a kv head x 64 dims
  const int rows_per_tile = 128 / group;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(hq),
                        static_cast<cuuint64_t>(total_q)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2,
                           static_cast<cuuint64_t>(hq) * head_dim * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(rows_per_tile)};
  cuuint32_t elem[3] = {1, 1, 1};
  CUresult cr = encode(qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, elem,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled(q) failed (%d)", static_cast<int>(cr));
  return RA_OK;
}

}  // namespace ra
