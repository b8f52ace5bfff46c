// Host-side helpers of the key/value cache entry points.
#include <mutex>

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

cudaError_t kv_num_sms(int* n) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    e = cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
  }
  *n = known[dev];
  return cudaSuccess;
}

}  // namespace dt
