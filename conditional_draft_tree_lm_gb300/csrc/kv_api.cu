// Host-side helpers of the key/value cache entry points.
#include <cuda.h>

#include "kv.cuh"

namespace dt {

dt_status kv_check_cache(const char* who, const dt_kv_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null cache or a null pointer in it", who);
  if (c->n_pages < 1 || c->n_kv < 1) return kv_fail(DT_ERR_INVALID_ARG, "%s: need n_pages and n_kv >= 1", who);
  if (!kv_page_ok(c->page)) return kv_fail(DT_ERR_SHAPE, "%s: page %d is not 16, 32, 64 or 128", who, c->page);
  if (c->head_dim != 64 && c->head_dim != 128)
    return kv_fail(DT_ERR_SHAPE, "%s: head_dim %d is not 64 or 128", who, c->head_dim);
  if (((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) != 0)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: the cache is not 16-byte aligned", who);
  return DT_OK;
}

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeFn>(f) : nullptr;
  }();
  return fn;
}

}  // namespace

bool kv_tmap_heads(CUtensorMap* tm, const void* base, int head_dim, int heads, int64_t rows, int64_t head_stride,
                   int64_t row_stride, int box_heads, int box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  // (the stride of a dimension of one entry is never used; zero is not encodable)
  if (heads == 1 && head_stride == 0) head_stride = head_dim;
  if (rows == 1 && row_stride == 0) row_stride = head_dim;
  if (head_stride <= 0 || row_stride <= 0) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool kv_tmap_rows(CUtensorMap* tm, const void* base, int row_bytes, int64_t rows, int box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(row_bytes), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1u, 1u};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dt
