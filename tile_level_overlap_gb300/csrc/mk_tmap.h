// Host side of the TMA tensor loads: 2D bf16 tensor maps with 128-byte
// swizzle, encoded through the driver entry point (no link-time dependency on
// the driver library).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mk {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)p;
  }
  return fn;
}

// Tensor map over a row-major bf16 matrix [rows][cols] (row pitch = cols * 2
// bytes), loading boxes of 64 columns (128 B) x box_rows rows with 128-byte
// swizzle.  Requirements checked by the driver: base 16-byte aligned, pitch a
// multiple of 16 bytes, box_rows <= 256.  Out-of-range rows read as zero.
inline bool make_tmap_bf16(CUtensorMap* out, const void* base, uint64_t rows, uint64_t cols,
                           uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Tensor map over a paged cache: (element, token of the page, 64-element part of
// the head, kv head, page), boxes of 64 elements (128 B) x min(page, most) tokens
// x `parts` with 128-byte swizzle, so a box's parts lie one after another in
// shared memory.  Pages (and tokens) out of range read as zero.  Strides of
// dimensions of size one are never used and replaced by a valid one.
template <class Kv>
inline bool make_page_tmap(CUtensorMap* out, const void* base, const Kv& c, int d, int most, int parts,
                           bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[5] = {64, (cuuint64_t)c.page, (cuuint64_t)(d / 64), (cuuint64_t)c.hkv, (cuuint64_t)c.n_pages};
  cuuint64_t strides[4] = {(cuuint64_t)c.token_stride * 2, 128,
                           (cuuint64_t)(c.hkv > 1 ? c.head_stride : c.token_stride) * 2,
                           (cuuint64_t)(c.n_pages > 1 ? c.page_stride : c.token_stride) * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)(c.page < most ? c.page : most), (cuuint32_t)parts, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Tensor map over query rows [rows][heads][d] (row_stride elements from row to
// row), boxes of 64 elements x box_heads x box_rows with 128-byte swizzle.
inline bool make_rows_tmap(CUtensorMap* out, const void* base, int rows, int heads, int d,
                           int64_t row_stride, int box_heads, int box_rows, bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)row_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace mk
