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
// pages is needed and no CTA waits for another.  A CTA looks at a window of rows, a
// warp at a row at a time: a run of up to eight rows (tokens, accepted paths) is the
// warp's own, longer ones (prompts) are taken by the whole CTA afterwards, several
// heads and tensors one after the other, the next one's loads in flight while one is
// reduced and written.
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

// One vector of 8 channels: its largest finite magnitude, and its codes.
DT_DEVINL float largest_finite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = bf16x2_f32(w[k]);
    amax = fmaxf(amax, fmaxf(fabsf(finite_or(f.x, 0.0f)), fabsf(finite_or(f.y, 0.0f))));
  }
  return amax;
}
// Of a thread's vectors the largest finite magnitude, two channels at a time; odd: an infinity is among them.
// (The maximum passes over NaNs, whose codes come out right by themselves.  Channel by channel, and with codes
// that look for infinities, prompts took 77 us instead of 58: half the issue slots were in use.)
template <int N>
DT_DEVINL float largest(const uint4 (&v)[N], bool& odd) {
  __nv_bfloat162 m = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = w[k] & 0x7FFF7FFFu;
      m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&a));
    }
  }
  float amax = fmaxf(__low2float(m), __high2float(m));
  odd = !(amax <= 3.402823466e38f);
  if (odd) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, largest_finite(v[i]));
  }
  return amax;
}
// Codes of values among which there is no infinity, inv: 1 / scale, a power of two.
DT_DEVINL uint2 encode_plain(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = bf16x2_f32(w[k]);
    o[k >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * inv, f.y * inv), __NV_SATFINITE, __NV_E4M3)) << ((k & 1) * 16);
  }
  return make_uint2(o[0], o[1]);
}
DT_DEVINL bool is_pow2(float x) { return (__float_as_uint(x) & 0x7FFFFFu) == 0; }
// (1 / now is exact for a power of two; a scale that a caller set otherwise is divided by)
DT_DEVINL uint2 encode(const uint4& v, float now) {
  const float nan = __uint_as_float(0x7FC00000u);
  const bool pow2 = is_pow2(now);
  const float inv = 1.0f / now;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 f = bf16x2_f32(w[k]);
    f.x = finite_or(f.x, nan);
    f.y = finite_or(f.y, nan);
    f = pow2 ? make_float2(f.x * inv, f.y * inv) : make_float2(f.x / now, f.y / now);
    o[k >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << ((k & 1) * 16);
  }
  return make_uint2(o[0], o[1]);
}
// 8 earlier codes, moved to a scale that is 1 / ratio times as large.
DT_DEVINL void move_codes(uint8_t* codes, float ratio) {
  uint2* at = reinterpret_cast<uint2*>(codes);
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
           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(b.x * ratio, b.y * ratio), __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  *at = make_uint2(r[0], r[1]);
}

// A run of up to kShort rows, of one head and tensor, by a warp.
constexpr int kShort = 8;
template <int HD>
DT_DEVINL void append_short(const AppendParams& p, int64_t t, int64_t slot, int len, int item) {
  constexpr int kVecs = HD / 8, kRowsAtOnce = 32 / kVecs, kHeld = kShort / kRowsAtOnce;
  const int lane = threadIdx.x & 31, head = item >> 1, which = item & 1;
  const int page = 1 << p.shift, off = static_cast<int>(slot & (page - 1));
  const int c = (lane % kVecs) * 8, r0 = lane / kVecs;
  uint4 v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < len) {
      const int64_t src = p.src_rows ? p.src_rows[t + r] : t + r;
      if (src >= 0 && src < p.n_src)
        v[i] = __ldg(reinterpret_cast<const uint4*>(p.x[which] + src * p.row_stride[which] + head * p.head_stride[which] + c));
      else if (p.status)
        atomicOr(p.status, DT_KV_BAD_INDEX);
    }
  }
  const int64_t tile = (slot >> p.shift) * p.n_kv + head;  // the page's part of this head
  float* scale_at = p.scale[which] + tile;
  const float old = off > 0 ? *scale_at : 0.0f;
  bool odd;
  const float need = kv_pow2_scale(warp_max(largest(v, odd)));
  const float now = off > 0 && old > need ? old : need;
  const bool plain = !odd && is_pow2(now);
  const float inv = 1.0f / now;
  uint8_t* codes = p.codes[which] + tile * page * HD;
  if (off > 0 && now > old) {
    const float ratio = old / now;
    for (int i = lane; i < off * kVecs; i += 32) move_codes(codes + static_cast<size_t>(i) * 8, ratio);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    if (r < len) *reinterpret_cast<uint2*>(codes + static_cast<size_t>(off + r) * HD + c) = plain ? encode_plain(v[i], inv) : encode(v[i], now);
  }
  __syncwarp();  // (every lane has read the old scale)
  if (lane == 0 && now != old) *scale_at = now;
}

// NV: 16-byte vectors per thread of a full page (page * HD / 8 / threads, at least 1).
template <int HD, int NV>
__global__ void __launch_bounds__(kAppendThreads, NV >= 8 ? 2 : 4) k_kv_append(const AppendParams p) {
  constexpr int kVecs = HD / 8;  // vectors per row
  constexpr int kWarps = kAppendThreads / 32;
  __shared__ float warp_max_s[2][kWarps];
  __shared__ int n_long, long_at[128 / kShort + 1], long_len[128 / kShort + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int page = 1 << p.shift;
  const int item0 = blockIdx.y * p.items, item1 = min(item0 + p.items, 2 * p.n_kv);  // item: 2 * head + tensor
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.window;
  if (tid == 0) n_long = 0;
  __syncthreads();

  for (int i = warp; i < p.window && t0 + i < p.n_rows; i += kWarps) {
    const int64_t t = t0 + i, slot = p.slot_map[t], before = t > 0 ? p.slot_map[t - 1] : -1;
    const int off = static_cast<int>(slot & (page - 1));
    if (slot < 0) continue;
    if (slot >= p.n_slots) {
      if (p.status && lane == 0) atomicOr(p.status, DT_KV_BAD_INDEX);
      continue;
    }
    if (before >= 0 && before + 1 == slot && off != 0) continue;  // inside a run that starts before this row
    // the run: rows whose slots count up inside the page
    int len = 1;
    for (int x = 1; x < page - off; x += 32) {
      const int r = x + lane;
      const bool same = r < page - off && t + r < p.n_rows && p.slot_map[t + r] == slot + r;
      const uint32_t more = __ballot_sync(0xFFFFFFFFu, same);
      len += more == 0xFFFFFFFFu ? 32 : __ffs(~more) - 1;
      if (more != 0xFFFFFFFFu) break;
    }
    if (len <= kShort) {
      for (int item = item0; item < item1; ++item) append_short<HD>(p, t, slot, len, item);
    } else if (lane == 0) {
      const int at = atomicAdd(&n_long, 1);
      long_at[at] = i;
      long_len[at] = len;
    }
  }
  __syncthreads();

  for (int run = 0; run < n_long; ++run) {
    const int64_t t = t0 + long_at[run], slot = p.slot_map[t];
    const int off = static_cast<int>(slot & (page - 1)), len = long_len[run];

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
      bool odd;
      float amax = largest(v, odd);
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
      const float now = off > 0 && old > need ? old : need, inv = 1.0f / now;
      const bool plain = !odd && is_pow2(now);
      if (off > 0 && now > old) {
        const float ratio = old / now;
        for (int i = tid; i < off * kVecs; i += kAppendThreads) move_codes(codes + static_cast<size_t>(i) * 8, ratio);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = (tid + i * kAppendThreads) / kVecs;
        if (r < len) *reinterpret_cast<uint2*>(codes + static_cast<size_t>(off + r) * HD + c) = plain ? encode_plain(v[i], inv) : encode(v[i], now);
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
    __syncthreads();  // (the next run's maxima take the same places)
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
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Rows of a window: eight, a row a warp, up to a page with many rows, so that the CTAs stay some waves.
  p.window = 8;
  while (p.window < cache->page && (a.n_rows / p.window) * cache->n_kv * 2 > kSms * 32) p.window *= 2;
  const int64_t windows = (a.n_rows + p.window - 1) / p.window;
  // (head, tensor) pairs a CTA takes one after the other: one until there are 16 CTAs for each SM.  (40960 rows of
  // prompts, 8 heads of 128: 58 us, 4.3 TB/s; the accepted paths of 32 trees 4.5 us, 32 tokens 2.8 us.  One CTA for
  // each run, head and tensor took 165, 10.2 and 4.2 us, with channels taken one by one.)
  p.items = 1;
  while (p.items < 2 * cache->n_kv && windows * 2 * cache->n_kv / p.items > kSms * 16) p.items *= 2;
  const dim3 grid(static_cast<unsigned>(windows), static_cast<unsigned>((2 * cache->n_kv + p.items - 1) / p.items));
  return kv_launched(who, cache->head_dim == 64 ? launch<64>(p, grid, st) : launch<128>(p, grid, st));
}
