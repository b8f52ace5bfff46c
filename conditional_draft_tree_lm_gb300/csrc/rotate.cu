// dt_qk_norm_rope: norms of queries and keys for each head and their rotation by position, in one pass.
//
// A head is held by G lanes (a power of two), 16 channels a lane, as the two pieces of 8 whose channels turn together:
// pieces i and i + rot / 2 (halves) or 16 neighbouring channels.  So a lane reads and writes 16 bytes at a time, the sum
// of squares takes log2 G shuffles, and the rotation none.  A lane's 8 angles are the same for every head of a row: a
// warp takes several heads of one row, and has cosines and sines once.
//
// Angles: a position times turns[i], in 64-bit integers, wraps by whole turns; the upper 32 bits are what is left of a
// turn, and exact for any position (fp32 has lost a radian at position 2^24).
//
// Bound by memory where there are many rows, by the latency of one pass where there are few.
#include "kv.cuh"

namespace dt {
namespace {

constexpr int kRotateThreads = 256;

struct RotateParams {
  dt_qk_norm_rope_args a;
  int64_t rows;
  int lanes;      // of a head that hold channels
  int pairs;      // of those, lanes whose channels turn
  int per_warp;   // heads of a warp
  int row_warps;  // warps of a row
};

DT_DEVINL void unpack8(const uint4& r, float* v) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
DT_DEVINL uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int G, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotateThreads) k_rotate(const RotateParams p) {
  const dt_qk_norm_rope_args& a = p.a;
  const int lane = threadIdx.x & 31, part = lane % G;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kRotateThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = warp / p.row_warps;
  if (row >= p.rows) return;
  const int first = static_cast<int>(warp - row * p.row_warps) * p.per_warp, heads = a.n_q + a.n_kv;
  const int last = min(heads, first + p.per_warp);
  const bool holds = part < p.lanes, turns = part < p.pairs;
  const int at0 = !INTERLEAVED && turns ? 8 * part : 16 * part, at1 = !INTERLEAVED && turns ? a.rot / 2 + 8 * part : 16 * part + 8;

  const int off = a.positions ? a.positions[row] : 0;
  if (off < 0) return;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
  if (turns) {
    const int64_t req = row / a.slots;
    const int64_t pos = (a.base ? static_cast<int64_t>(a.base[req]) : 0) + (a.positions ? off : row - req * a.slots);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int left = static_cast<int>((a.turns[8 * part + i] * static_cast<uint64_t>(pos)) >> 32);
      sincospif(static_cast<float>(left) * 0x1p-31f, &sn[i], &cs[i]);
      cs[i] *= a.amplitude;
      sn[i] *= a.amplitude;
    }
  }
  for (int h0 = first; h0 < last; h0 += 32 / G) {
    const int h = h0 + lane / G;
    const bool here = holds && h < last, key = h >= a.n_q;
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(key ? a.k : a.q) +
                                (key ? row * a.k_row_stride + (h - a.n_q) * a.k_head_stride : row * a.q_row_stride + h * a.q_head_stride);
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(key ? a.k_out : a.q_out) +
                        (key ? row * a.k_out_row_stride + (h - a.n_q) * a.k_out_head_stride : row * a.q_out_row_stride + h * a.q_out_head_stride);
    const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(key ? a.k_weight : a.q_weight);
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (here) {
      unpack8(*reinterpret_cast<const uint4*>(from + at0), v);
      unpack8(*reinterpret_cast<const uint4*>(from + at1), v + 8);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (!here) continue;
    if (weight) {
      const float r = rsqrtf(sum / static_cast<float>(a.head_dim) + a.eps);
      float w[16];
      unpack8(*reinterpret_cast<const uint4*>(weight + at0), w);
      unpack8(*reinterpret_cast<const uint4*>(weight + at1), w + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] * r * w[i];
    }
    if (turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& x = INTERLEAVED ? v[2 * i] : v[i];
        float& y = INTERLEAVED ? v[2 * i + 1] : v[8 + i];
        const float u = x * cs[i] - y * sn[i];
        y = y * cs[i] + x * sn[i];
        x = u;
      }
    }
    *reinterpret_cast<uint4*>(to + at0) = pack8(v);
    *reinterpret_cast<uint4*>(to + at1) = pack8(v + 8);
  }
}

template <int G>
cudaError_t launch(const RotateParams& p, int64_t blocks, cudaStream_t st) {
  if (p.a.interleaved) k_rotate<G, true><<<static_cast<unsigned>(blocks), kRotateThreads, 0, st>>>(p);
  else k_rotate<G, false><<<static_cast<unsigned>(blocks), kRotateThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dt

extern "C" dt_status dt_qk_norm_rope(const dt_qk_norm_rope_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_qk_norm_rope";
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  dt_qk_norm_rope_args a = *args;
  if (!a.k) a.n_kv = 0;
  if (a.n_req < 0 || a.slots < 0 || a.n_q < 1 || a.n_kv < (a.k ? 1 : 0))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: need n_req, slots >= 0 and n_q, n_kv >= 1", who);
  if (a.n_q > 4096 || a.n_kv > 4096) return kv_fail(DT_ERR_SHAPE, "%s: more than 4096 heads", who);
  const int64_t rows = static_cast<int64_t>(a.n_req) * a.slots;
  if (rows > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: more than 2^31-1 rows", who);
  if (a.head_dim < 32 || a.head_dim > 256 || a.head_dim % 16 != 0)
    return kv_fail(DT_ERR_SHAPE, "%s: head_dim %d is not a multiple of 16 in 32..256", who, a.head_dim);
  if (a.rot < 0 || a.rot > a.head_dim || a.rot % 16 != 0 || (a.turns != nullptr) != (a.rot > 0))
    return kv_fail(DT_ERR_SHAPE, "%s: rot %d: a multiple of 16 up to head_dim, with turns, or 0 without", who, a.rot);
  if (!(a.eps >= 0.0f) || a.eps - a.eps != 0.0f || a.amplitude - a.amplitude != 0.0f)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: eps or amplitude is not finite, or eps below 0", who);
  if (!a.turns && !a.q_weight && !a.k_weight) return kv_fail(DT_ERR_INVALID_ARG, "%s: neither weights nor turns", who);
  if (rows == 0) return DT_OK;
  if (!kv_rows_ok(a.q, a.q_row_stride, a.q_head_stride) || !kv_rows_ok(a.q_out, a.q_out_row_stride, a.q_out_head_stride) ||
      (a.k && (!kv_rows_ok(a.k, a.k_row_stride, a.k_head_stride) || !kv_rows_ok(a.k_out, a.k_out_row_stride, a.k_out_head_stride))))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null or misaligned q, k, q_out or k_out", who);
  if (((reinterpret_cast<uintptr_t>(a.q_weight) | reinterpret_cast<uintptr_t>(a.k_weight)) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(a.turns) & 7u) != 0)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: misaligned weights or turns", who);
  if (!kv_rows_apart(rows, a.n_q, a.head_dim, a.q_out_row_stride, a.q_out_head_stride) ||
      (a.k && !kv_rows_apart(rows, a.n_kv, a.head_dim, a.k_out_row_stride, a.k_out_head_stride)))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: rows of q_out or k_out overlap", who);
  RotateParams p = {};
  p.a = a;
  p.rows = rows;
  p.lanes = a.head_dim / 16;
  p.pairs = a.rot / 16;
  int g = 2;
  while (g < p.lanes) g *= 2;
  // A warp takes as many heads of a row as leave 16 warps an SM (its cosines are had once), at least one of each lane group.
  const int heads = a.n_q + a.n_kv, step = 32 / g, most = (heads + step - 1) / step;
  const int64_t wanted = (16 * kSms + rows - 1) / rows;
  p.row_warps = static_cast<int>(wanted < most ? wanted : most);
  p.per_warp = (most + p.row_warps - 1) / p.row_warps * step;
  p.row_warps = (heads + p.per_warp - 1) / p.per_warp;
  const int64_t blocks = (rows * p.row_warps + kRotateThreads / 32 - 1) / (kRotateThreads / 32);
  if (blocks > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: too many rows and heads for one launch", who);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_launched(who, g == 2 ? launch<2>(p, blocks, st) : g == 4 ? launch<4>(p, blocks, st) : g == 8 ? launch<8>(p, blocks, st) : launch<16>(p, blocks, st));
}
