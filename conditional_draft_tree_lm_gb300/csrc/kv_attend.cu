// dt_cache_attention and dt_prompt_attention, the plain form: one warp per row
// and head, one key at a time with a running maximum and sum.
#include "kv.cuh"
#include "kv_decode.cuh"

namespace dt {
namespace {

template <int HD>
struct Row {
  static constexpr int N = HD / 32;
  float q[N], o[N], m, l;
  DT_DEVINL void start(const __nv_bfloat16* p, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __bfloat162float(p[lane * N + i]), o[i] = 0.0f;
    m = -INFINITY;
    l = 0.0f;
  }
  DT_DEVINL void step(const float (&k)[N], const float (&v)[N], float scale) {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) z += q[i] * k[i];
    z = warp_sum(z) * scale;
    const float m2 = fmaxf(m, z), base = m2 == -INFINITY ? 0.0f : m2;
    const float a = expf(m - base), e = expf(z - base);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * a + e * v[i];
    m = m2;
  }
  DT_DEVINL void end(__nv_bfloat16* p, float* lse, int lane) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < N; ++i) p[lane * N + i] = __float2bfloat16(o[i] * inv);
    if (lse && lane == 0) *lse = l == 0.0f ? -INFINITY : m + logf(l);
  }
};

template <int HD>
__global__ void k_plain_cache(const dt_kv_cache c, const dt_cache_attention_args a) {
  constexpr int N = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.n_req) * a.slots * a.n_q) return;
  const int h = static_cast<int>(w % a.n_q), kvh = h / (a.n_q / c.n_kv);
  const int64_t row = w / a.n_q;
  const int slot = static_cast<int>(row % a.slots), req = static_cast<int>(row / a.slots);
  Row<HD> r;
  r.start(static_cast<const __nv_bfloat16*>(a.q) + row * a.q_row_stride + h * a.q_head_stride, lane);
  int len = a.length[req];
  len = min(max(len, 0), a.max_blocks * c.page);
  for (int t = 0; t < len; ++t) {
    const int page = a.block_table[static_cast<size_t>(req) * a.max_blocks + t / c.page];
    if (page < 0 || page >= c.n_pages) {
      if (a.status && lane == 0) atomicOr(a.status, DT_KV_BAD_INDEX);
      continue;
    }
    const size_t tile = static_cast<size_t>(page) * c.n_kv + kvh;
    const size_t at = (tile * c.page + t % c.page) * HD + lane * N;
    float k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(c.k)[at + i]) * c.k_scale[tile];
      v[i] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(c.v)[at + i]) * c.v_scale[tile];
    }
    r.step(k, v, a.scale);
  }
  if (a.k_new) {
    for (int b = 0; b < a.slots; ++b) {
      const bool see = a.mask ? a.mask[row * a.slots + b] != 0 : b <= slot;
      if (!see) continue;
      const int64_t s = static_cast<int64_t>(req) * a.slots + b;
      float k[N], v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        k[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.k_new)[s * a.k_row_stride + kvh * a.k_head_stride + lane * N + i]);
        v[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.v_new)[s * a.v_row_stride + kvh * a.v_head_stride + lane * N + i]);
      }
      r.step(k, v, a.scale);
    }
  }
  r.end(static_cast<__nv_bfloat16*>(a.out) + row * a.out_row_stride + h * a.out_head_stride, a.lse ? a.lse + w : nullptr, lane);
}

}  // namespace
}  // namespace dt

extern "C" size_t dt_cache_attention_workspace(int n_req, int slots, int n_q, int n_kv, int head_dim) {
  if (n_req < 1 || slots < 1 || n_kv < 1 || n_q < n_kv || n_q % n_kv != 0 || (head_dim != 64 && head_dim != 128)) return 0;
  const int rows = slots * (n_q / n_kv);
  if (rows <= dt::kDecodeMaxRows) return dt::decode_workspace(rows, head_dim);
  return 256;
}

extern "C" dt_status dt_cache_attention(const dt_kv_cache* cache, const dt_cache_attention_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_cache_attention";
  if (dt_status s = kv_check_cache(who, cache)) return s;
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  const dt_cache_attention_args& a = *args;
  if (a.n_req < 1 || a.slots < 1 || a.n_q < 1 || a.max_blocks < 1)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: need n_req, slots, n_q, max_blocks >= 1", who);
  if (a.n_q % cache->n_kv != 0 || a.n_q / cache->n_kv > 128)
    return kv_fail(DT_ERR_SHAPE, "%s: %d query heads over %d key/value heads: need a multiple, at most 128 a head", who,
                   a.n_q, cache->n_kv);
  if (static_cast<int64_t>(a.n_req) * a.slots > 0x7FFFFFFF || static_cast<int64_t>(a.max_blocks) * cache->page > 0x7FFFFFFF)
    return kv_fail(DT_ERR_SHAPE, "%s: more than 2^31-1 rows or tokens", who);
  if (!(a.scale - a.scale == 0.0f)) return kv_fail(DT_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (!a.block_table || !a.length || !kv_rows_ok(a.q, a.q_row_stride, a.q_head_stride) ||
      !kv_rows_ok(a.out, a.out_row_stride, a.out_head_stride))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null or misaligned q, out, block_table or length", who);
  if ((a.k_new != nullptr) != (a.v_new != nullptr) ||
      (a.k_new && (!kv_rows_ok(a.k_new, a.k_row_stride, a.k_head_stride) || !kv_rows_ok(a.v_new, a.v_row_stride, a.v_head_stride))))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: k_new and v_new: one is null or misaligned", who);
  if (a.mask && !a.k_new) return kv_fail(DT_ERR_INVALID_ARG, "%s: a mask without new keys", who);
  const size_t need = dt_cache_attention_workspace(a.n_req, a.slots, a.n_q, cache->n_kv, cache->head_dim);
  if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u) != 0 || a.workspace_bytes < need)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: the workspace is null, misaligned or below %zu bytes", who, need);
  if (static_cast<int64_t>(a.n_req) * cache->n_kv > kMaxJoins)
    return kv_fail(DT_ERR_SHAPE, "%s: n_req * n_kv above %d", who, kMaxJoins);
  if ((static_cast<int64_t>(a.max_blocks) * cache->page / kDecodeTile + 1) * a.n_req * cache->n_kv > (1 << 30))
    return kv_fail(DT_ERR_SHAPE, "%s: more than 2^37 cached tokens over all requests and heads", who);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int group = a.n_q / cache->n_kv;
  if (a.slots * group <= kDecodeMaxRows) {
    DecodeParams p = {};
    p.c = *cache;
    p.a = a;
    p.group = group;
    p.rows = a.slots * group;
    p.shift = 4;
    while ((1 << p.shift) < cache->page) ++p.shift;
    p.done = static_cast<unsigned*>(a.workspace);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kCounterBytes);
    const int grid = decode_grid(a.n_req, cache->n_kv, static_cast<long long>(a.max_blocks) * cache->page);
    cudaError_t e;
    if (cache->head_dim == 64) e = p.rows <= 8 ? launch_decode<64, 1>(p, grid, st) : launch_decode<64, 2>(p, grid, st);
    else e = p.rows <= 8 ? launch_decode<128, 1>(p, grid, st) : launch_decode<128, 2>(p, grid, st);
    return kv_launched(who, e);
  }
  const int64_t warps = static_cast<int64_t>(a.n_req) * a.slots * a.n_q;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  if (cache->head_dim == 64) k_plain_cache<64><<<grid, 128, 0, st>>>(*cache, a);
  else k_plain_cache<128><<<grid, 128, 0, st>>>(*cache, a);
  return kv_launched(who, cudaGetLastError());
}
