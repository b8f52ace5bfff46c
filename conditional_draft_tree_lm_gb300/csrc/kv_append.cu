// dt_kv_append: bf16 keys and values of new tokens into the 8-bit cache.
//
// Per page touched, head and tensor ("run": the new tokens that go to one page):
//   need  = smallest power of two with 448 need >= max |x| over the run's finite x
//   scale' = need at a page's start, else max(scale, need)
//   earlier codes of the page -> RNE(code * scale / scale') where scale' > scale
//   new codes = RNE(x / scale')
// Powers of two make x / scale' exact, so that each value is rounded once, and
// move earlier codes without rounding until they become subnormal.
//
// What bounds it: bytes (4 read and 2 written per channel pair), or latency for
// a few tokens.  A run's part of one head and tensor is held in registers by a CTA
// (16-byte loads), so that it is read once: amax first, codes from the same
// registers.  Runs are found from the slot map itself: a row leads a run unless
// its slot is the previous row's plus one inside the same page, so no list of
// pages is needed and no CTA waits for another.  With enough runs a CTA takes
// several heads and tensors of its run, the next one's loads in flight while one
// is reduced and written; with few, one each, for latency.
#include "kv.cuh"

namespace dt {
namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
  const __nv_bfloat16* x[2];
  int64_t row_stride[2], head_stride[2];
  uint8_t* codes[2];
  float* scale[2];
  const int64_t* slot_map;
  const int32_t* src_rows;
  int* status;
  int64_t n_rows, n_src, n_slots;
  int n_kv, shift, window, items;  // items: (head, tensor) pairs of a CTA
};

// Two bf16 in a word, as fp32.
DT_DEVINL float2 bf16x2_f32(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
DT_DEVINL float finite_or(float x, float other) { return fabsf(x) <= 3.402823466e38f ? x : other; }

// NV: 16-byte vectors per thread of a full page (page * HD / 8 / threads, at least 1).
template <int HD, int NV>
__global__ void __launch_bounds__(kAppendThreads, NV >= 8 ? 2 : 4) k_kv_append(const AppendParams p) {
  constexpr int kVecs = HD / 8;  // vectors per row
  constexpr int kWarps = kAppendThreads / 32;
  __shared__ float warp_max_s[2][kWarps];
  __shared__ int run_len_s;
  const int tid = threadIdx.x;
  const int page = 1 << p.shift;
  const int item0 = blockIdx.y * p.items, item1 = min(item0 + p.items, 2 * p.n_kv);  // item: 2 * head + tensor
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.window;
  const int64_t t1 = t0 + p.window < p.n_rows ? t0 + p.window : p.n_rows;

  for (int64_t t = t0; t < t1;) {
    const int64_t slot = p.slot_map[t];
    const int64_t before = t > 0 ? p.slot_map[t - 1] : -1;
    const int off = static_cast<int>(slot & (page - 1));
    if (slot < 0 || slot >= p.n_slots) {
      if (slot >= 0 && p.status && tid == 0) atomicOr(p.status, DT_KV_BAD_INDEX);
      ++t;
      continue;
    }
    if (before >= 0 && before + 1 == slot && off != 0) {  // inside a run that starts before this row
      ++t;
      continue;
    }
    // the run: rows whose slots count up inside the page
    __syncthreads();
    if (tid == 0) run_len_s = page - off;
    __syncthreads();
    if (tid < page - off && (t + tid >= p.n_rows || p.slot_map[t + tid] != slot + tid)) atomicMin(&run_len_s, tid);
    __syncthreads();
    const int len = run_len_s;

    // this thread's vectors: rows of the source, the same for every head and tensor
    int64_t src[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = (tid + i * kAppendThreads) / kVecs;
      src[i] = -1;
      if (r < len) {
        src[i] = p.src_rows ? p.src_rows[t + r] : t + r;
        if (src[i] < 0 || src[i] >= p.n_src) {
          if (p.status) atomicOr(p.status, DT_KV_BAD_INDEX);
          src[i] = -1;
        }
      }
    }
    const int c = (tid % kVecs) * 8;  // (threads are a multiple of a row's vectors)
    auto load = [&](uint4 (&v)[NV], int item) {
      const int which = item & 1;
      const __nv_bfloat16* x = p.x[which] + (item >> 1) * p.head_stride[which] + c;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        v[i] = src[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(x + src[i] * p.row_stride[which])) : make_uint4(0, 0, 0, 0);
    };
    auto use = [&](const uint4 (&v)[NV], int item) {
      const int which = item & 1, head = item >> 1;
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = bf16x2_f32(w[k]);
          amax = fmaxf(amax, fmaxf(fabsf(finite_or(f.x, 0.0f)), fabsf(finite_or(f.y, 0.0f))));
        }
      }
      const int64_t tile = (slot >> p.shift) * p.n_kv + head;  // the page's part of this head
      float* scale_at = p.scale[which] + tile;
      const float old = off > 0 ? *scale_at : 0.0f;  // (read by all before thread 0 may write it)
      float* warp_max_at = warp_max_s[item & 1];     // (the next item's write is behind this one's barrier)
      amax = warp_max(amax);
      if ((tid & 31) == 0) warp_max_at[tid >> 5] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, warp_max_at[w]);

      uint8_t* codes = p.codes[which] + tile * page * HD;
      const float need = kv_pow2_scale(amax);
      const float now = off > 0 && old > need ? old : need;
      if (off > 0 && now > old) {
        const float ratio = old / now;
        for (int i = tid; i < off * kVecs; i += kAppendThreads) {
          uint2* at = reinterpret_cast<uint2*>(codes + static_cast<size_t>(i) * 8);
          const uint2 w = *at;
          uint32_t r[2];
          const uint32_t in[2] = {w.x, w.y};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(in[k], lo, hi);
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            r[k] = __nv_cvt_float2_to_fp8x2(make_float2(a.x * ratio, a.y * ratio), __NV_SATFINITE, __NV_E4M3) |
                   static_cast<uint32_t>(
                       __nv_cvt_float2_to_fp8x2(make_float2(b.x * ratio, b.y * ratio), __NV_SATFINITE, __NV_E4M3))
                       << 16;
          }
          *at = make_uint2(r[0], r[1]);
        }
      }
      // (1 / now is exact for a power of two; a scale that a caller set otherwise is divided by)
      const float nan = __uint_as_float(0x7FC00000u);
      const bool pow2 = (__float_as_uint(now) & 0x7FFFFFu) == 0;
      const float inv = 1.0f / now;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = (tid + i * kAppendThreads) / kVecs;
        if (r >= len) continue;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 f = bf16x2_f32(w[k]);
          f.x = finite_or(f.x, nan);
          f.y = finite_or(f.y, nan);
          f = pow2 ? make_float2(f.x * inv, f.y * inv) : make_float2(f.x / now, f.y / now);
          o[k >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << ((k & 1) * 16);
        }
        *reinterpret_cast<uint2*>(codes + static_cast<size_t>(off + r) * HD + c) = make_uint2(o[0], o[1]);
      }
      if (tid == 0 && now != old) *scale_at = now;
    };
    uint4 v[2][NV];
    load(v[0], item0);
    for (int item = item0; item < item1; item += 2) {
      if (item + 1 < item1) load(v[1], item + 1);
      use(v[0], item);
      if (item + 1 >= item1) break;
      if (item + 2 < item1) load(v[0], item + 2);
      use(v[1], item + 1);
    }
    t += len;
  }
}

template <int HD>
cudaError_t launch(const AppendParams& p, dim3 grid, cudaStream_t st) {
  switch ((1 << p.shift) * HD / 8 / kAppendThreads) {
    case 0:
    case 1: k_kv_append<HD, 1><<<grid, kAppendThreads, 0, st>>>(p); break;
    case 2: k_kv_append<HD, 2><<<grid, kAppendThreads, 0, st>>>(p); break;
    case 4: k_kv_append<HD, 4><<<grid, kAppendThreads, 0, st>>>(p); break;
    default: k_kv_append<HD, 8><<<grid, kAppendThreads, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace dt

extern "C" dt_status dt_kv_append(const dt_kv_cache* cache, const dt_kv_append_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_kv_append";
  if (dt_status s = kv_check_cache(who, cache)) return s;
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  const dt_kv_append_args& a = *args;
  if (a.n_rows < 0 || a.n_src < 0) return kv_fail(DT_ERR_INVALID_ARG, "%s: a negative row count", who);
  if (a.n_rows > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: n_rows above 2^31-1", who);
  if (cache->n_kv > 32767) return kv_fail(DT_ERR_SHAPE, "%s: n_kv above 32767", who);
  if (a.n_rows == 0) return DT_OK;
  if (!a.slot_map || !kv_rows_ok(a.k, a.k_row_stride, a.k_head_stride) || !kv_rows_ok(a.v, a.v_row_stride, a.v_head_stride))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null or misaligned k, v or slot_map", who);
  AppendParams p = {};
  p.x[0] = static_cast<const __nv_bfloat16*>(a.k);
  p.x[1] = static_cast<const __nv_bfloat16*>(a.v);
  p.row_stride[0] = a.k_row_stride;
  p.row_stride[1] = a.v_row_stride;
  p.head_stride[0] = a.k_head_stride;
  p.head_stride[1] = a.v_head_stride;
  p.codes[0] = static_cast<uint8_t*>(cache->k);
  p.codes[1] = static_cast<uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.slot_map = a.slot_map;
  p.src_rows = a.src_rows;
  p.status = a.status;
  p.n_rows = a.n_rows;
  p.n_src = a.n_src;
  p.n_kv = cache->n_kv;
  while ((16 << p.shift) < cache->page) ++p.shift;
  p.shift += 4;
  p.n_slots = static_cast<int64_t>(cache->n_pages) << p.shift;
  // Rows a CTA looks for runs in: one while the CTAs still fit the GPU a few times over
  // (each row may be a run of its own, a token per request), up to a page for long prompts.
  p.window = 1;
  while (p.window < cache->page && (a.n_rows / p.window) * cache->n_kv * 2 > 16384) p.window *= 2;
  const int64_t windows = (a.n_rows + p.window - 1) / p.window;
  // (head, tensor) pairs a CTA takes one after the other: one until there are 16 CTAs for each SM (40960 rows of
  // prompts: 81 us, 86 with 8 or 4, 96 with 32; 512 padded rows of accepted paths: 10.2, 13.0, 20.8 and 9.0 us)
  p.items = 1;
  while (p.items < 2 * cache->n_kv && windows * 2 * cache->n_kv / p.items > kSms * 16) p.items *= 2;
  const dim3 grid(static_cast<unsigned>(windows), static_cast<unsigned>((2 * cache->n_kv + p.items - 1) / p.items));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_launched(who, cache->head_dim == 64 ? launch<64>(p, grid, st) : launch<128>(p, grid, st));
}
