// dt_qk_norm_rope: norms of queries and keys for each head and their rotation by position, in one pass.
//
// A head is held by G lanes (a power of two), 16 channels a lane, as the two pieces of 8 whose channels turn together:
// pieces i and i + rot / 2 (halves) or 16 neighbouring channels.  So a lane reads and writes 16 bytes at a time, the sum
// of squares takes log2 G shuffles, and the rotation none.  A CTA takes all heads of a row (of several rows beside each
// other where heads are few), so that its cosines are had once, by its threads together, into shared memory, and where rows
// are many two such rows one after the other, whose channels are all on their way before the cosines are computed: a
// thread keeps its place in the heads, so that its addresses and weights serve two rows.
//
// Angles: a position times turns[i], in 64-bit integers, wraps by whole turns; the upper 32 bits are what is left of a
// turn, and exact for any position (fp32 has lost a radian at position 2^24).
//
// Squares are summed in fp32; a head for which they leave it (channels of 2^63 and more, or of 2^-45 and less where eps is as small)
// is taken once more by a power of two, so that any finite head has its norm.  The check costs 3 % (32k rows 124.3 us without).
//
// Bound by instructions and memory alike where there are many rows: 32k rows of 32 + 8 heads of 128 127 us, 5.3 TB/s (before that check one
// row a CTA 159 us, with 326 instructions a warp in 67 % of the issue slots; four rows 127 us; persistent CTAs with the next row ahead
// 149 us); without norms 116 us; by the latency of one pass where there are few: 32 rows 2.3 us.
#include "kv_flash.cuh"

namespace dt {
namespace {

constexpr int kRotateThreads = 512;  // of a CTA at most
constexpr int kMaxAngles = 1024;     // of the rows that a CTA takes at once

struct RotateParams {
  dt_qk_norm_rope_args a;
  int64_t rows;
  int lanes;   // of a head that hold channels
  int pairs;   // of those, lanes whose channels turn
  int heads;   // of a CTA (blockIdx.y counts those)
  int at_once; // rows of a CTA
  float one_over;  // 1 / head_dim
};

// 8 bf16 as pairs of fp32, and back.
DT_DEVINL void unpack8(const uint4& r, uint64_t* v) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
DT_DEVINL uint4 pack8(const uint64_t* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f32x2_parts(v[i], lo, hi);
    w[i] = pack_p(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Of a head's channels, in all of its lanes.
template <int G>
DT_DEVINL float sum_squares(const uint64_t (&v)[8], int tid) {
  uint64_t sum2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum2 = fma2(v[i], v[i], sum2);
  float sum, other;
  f32x2_parts(sum2, sum, other);
  sum += other;
  const uint32_t lanes = ((1u << G) - 1u) << (tid & 31 & ~(G - 1));
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
  return sum;
}

template <int G, bool INTERLEAVED, int ROWS>
__global__ void __launch_bounds__(kRotateThreads, ROWS == 1 ? 3 : 2) k_rotate(const RotateParams p) {
  __shared__ __align__(16) float s_cos[kMaxAngles], s_sin[kMaxAngles];
  const dt_qk_norm_rope_args& a = p.a;
  const int tid = threadIdx.x, part = tid % G, unit = tid / G;
  const int nth = p.at_once == 1 ? 0 : unit / p.heads, h = blockIdx.y * p.heads + unit - nth * p.heads;  // row beside the others, head
  const bool key = h >= a.n_q, turns = part < p.pairs;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (ROWS * p.at_once), row0 = first + nth;
  // (units behind the CTA's own, with which its last warp is filled, have nothing: their heads are the next CTA's)
  const bool holds = part < p.lanes && unit < p.heads * p.at_once && h < a.n_q + a.n_kv;
  const int left_rows = holds ? static_cast<int>(min(static_cast<int64_t>(ROWS * p.at_once), p.rows - row0)) : 0;  // row r is there where r at_once < left_rows
  const int at0 = !INTERLEAVED && turns ? 8 * part : 16 * part, apart = !INTERLEAVED && turns ? a.rot / 2 : 8;
  const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(key ? a.k_weight : a.q_weight);
  const int head = key ? h - a.n_q : h;
  const int64_t from_row = key ? a.k_row_stride : a.q_row_stride;
  const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(key ? a.k : a.q) + row0 * from_row + head * (key ? a.k_head_stride : a.q_head_stride) + at0;
  dt_grid_wait();
  uint4 x[ROWS][2];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (r * p.at_once < left_rows) {
      const __nv_bfloat16* at = from + r * p.at_once * from_row;
      x[r][0] = *reinterpret_cast<const uint4*>(at);
      x[r][1] = *reinterpret_cast<const uint4*>(at + apart);
    } else {
      x[r][0] = x[r][1] = make_uint4(0, 0, 0, 0);
    }
  uint4 w0 = {}, w1 = {};
  if (holds && weight) {
    w0 = *reinterpret_cast<const uint4*>(weight + at0);
    w1 = *reinterpret_cast<const uint4*>(weight + at0 + apart);
  }
  // (the channels are asked for whether a row is written or not: else they would wait for its position)
  int off[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) off[r] = a.positions && r * p.at_once < left_rows ? a.positions[row0 + r * p.at_once] : 0;
  const int angles = a.rot / 2, rows = static_cast<int>(min(static_cast<int64_t>(ROWS * p.at_once), p.rows - first));
  for (int e = tid; e < rows * angles; e += blockDim.x) {
    const int r = e / angles, i = e - r * angles;
    const uint32_t row = static_cast<uint32_t>(first + r), req = a.base || !a.positions ? row / static_cast<uint32_t>(a.slots) : 0;
    const int64_t pos = (a.base ? static_cast<int64_t>(a.base[req]) : 0) + (a.positions ? a.positions[row] : static_cast<int>(row - req * a.slots));
    const int left = static_cast<int>((a.turns[i] * static_cast<uint64_t>(pos)) >> 32);
    float c, s;
    sincospif(static_cast<float>(left) * 0x1p-31f, &s, &c);
    s_cos[e] = c * a.amplitude;
    s_sin[e] = s * a.amplitude;
  }
  __syncthreads();
  uint64_t w[8];
  unpack8(w0, w);
  unpack8(w1, w + 4);
  const int64_t to_row = key ? a.k_out_row_stride : a.q_out_row_stride;
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(key ? a.k_out : a.q_out) + row0 * to_row + head * (key ? a.k_out_head_stride : a.q_out_head_stride) + at0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    uint64_t v[8];
    unpack8(x[r][0], v);
    unpack8(x[r][1], v + 4);
    if (weight) {  // (the same for all lanes of a head)
      float mean = fmaf(sum_squares<G>(v, tid), p.one_over, a.eps);
      // Squares that leave fp32 (a mean below 2^-90, infinite or NaN): the head by a power of two larger or smaller.
      constexpr uint32_t kLeast = (127 - 90) << 23, kInfinite = 255u << 23;
      if (__float_as_uint(mean) - kLeast >= kInfinite - kLeast) {
        const float unit = mean > 1.0f ? 0x1p-70f : 0x1p75f;
        const uint64_t unit2 = f32x2(unit, unit);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], unit2);
        mean = fmaf(sum_squares<G>(v, tid), p.one_over, a.eps * unit * unit);
      }
      const float scale = rsqrtf(mean);
      const uint64_t scale2 = f32x2(scale, scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mul2(mul2(v[i], scale2), w[i]);
    }
    if (r * p.at_once >= left_rows || off[r] < 0) continue;
    if (turns) {
      const int at = (r * p.at_once + nth) * angles + 8 * part;
      const float4* cs = reinterpret_cast<const float4*>(&s_cos[at]);
      const float4* sn = reinterpret_cast<const float4*>(&s_sin[at]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 c = cs[j], s = sn[j];
        if (INTERLEAVED) {  // (a, b) (c, c) + (b, a) (-s, s)
          const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y, z;
            f32x2_parts(v[4 * j + i], y, z);
            v[4 * j + i] = fma2(f32x2(z, y), f32x2(-s4[i], s4[i]), mul2(v[4 * j + i], f32x2(c4[i], c4[i])));
          }
        } else {
          const uint64_t c2[2] = {f32x2(c.x, c.y), f32x2(c.z, c.w)}, s2[2] = {f32x2(s.x, s.y), f32x2(s.z, s.w)};
          const uint64_t minus[2] = {f32x2(-s.x, -s.y), f32x2(-s.z, -s.w)};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t y = v[2 * j + i], z = v[4 + 2 * j + i];
            v[2 * j + i] = fma2(z, minus[i], mul2(y, c2[i]));
            v[4 + 2 * j + i] = fma2(y, s2[i], mul2(z, c2[i]));
          }
        }
      }
    }
    __nv_bfloat16* at = to + r * p.at_once * to_row;
    *reinterpret_cast<uint4*>(at) = pack8(v);
    *reinterpret_cast<uint4*>(at + apart) = pack8(v + 4);
  }
}

template <int G, bool INTERLEAVED>
cudaError_t launch(const RotateParams& p, int sequence, dim3 grid, int threads, cudaStream_t st) {
  return launch_behind(sequence == 2 ? k_rotate<G, INTERLEAVED, 2> : k_rotate<G, INTERLEAVED, 1>, grid, threads, 0, st, 1, p);
}
template <int G>
cudaError_t launch(const RotateParams& p, int sequence, dim3 grid, int threads, cudaStream_t st) {
  return p.a.interleaved ? launch<G, true>(p, sequence, grid, threads, st) : launch<G, false>(p, sequence, grid, threads, st);
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
  if (!kv_aligned(16, a.q_weight, a.k_weight) || !kv_aligned(8, a.turns) || !kv_aligned(4, a.positions, a.base))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: misaligned weights, turns, positions or base", who);
  if (!kv_rows_apart(rows, a.n_q, a.head_dim, a.q_out_row_stride, a.q_out_head_stride) ||
      (a.k && !kv_rows_apart(rows, a.n_kv, a.head_dim, a.k_out_row_stride, a.k_out_head_stride)))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: rows of q_out or k_out overlap", who);
  struct Heads {
    const void* at;
    int heads;
    int64_t row_stride, head_stride;
  };
  // (the larger stride's as rows, whatever order they stand in)
  auto in_memory = [&](const Heads& h) {
    const bool head_rows = h.heads > 1 && (rows == 1 || h.head_stride > h.row_stride);
    const int64_t in = head_rows ? (rows - 1) * h.row_stride : (h.heads - 1) * h.head_stride;
    return MemoryRows{reinterpret_cast<uintptr_t>(h.at), head_rows ? h.heads : rows, 2 * (head_rows ? h.head_stride : h.row_stride), 2 * (in + a.head_dim)};
  };
  auto meet = [&](const Heads& x, const Heads& y) { return rows_meet(in_memory(x), in_memory(y)); };
  auto same = [&](const Heads& x, const Heads& y) {
    return x.at == y.at && (rows == 1 || x.row_stride == y.row_stride) && (x.heads == 1 || x.head_stride == y.head_stride);
  };
  const Heads q = {a.q, a.n_q, a.q_row_stride, a.q_head_stride}, q_out = {a.q_out, a.n_q, a.q_out_row_stride, a.q_out_head_stride};
  const Heads k = {a.k, a.n_kv, a.k_row_stride, a.k_head_stride}, k_out = {a.k_out, a.n_kv, a.k_out_row_stride, a.k_out_head_stride};
  auto over = [&](const void* d, int64_t bytes) {  // whether what is written lies over d
    const MemoryRows r = {reinterpret_cast<uintptr_t>(d), 1, 0, bytes};
    return d && (rows_meet(in_memory(q_out), r) || (a.k && rows_meet(in_memory(k_out), r)));
  };
  if ((!same(q, q_out) && meet(q, q_out)) || (a.k && ((!same(k, k_out) && meet(k, k_out)) || meet(q, k_out) || meet(k, q_out) || meet(q_out, k_out))) ||
      over(a.q_weight, 2 * a.head_dim) || over(a.k_weight, 2 * a.head_dim) || over(a.turns, 4 * a.rot) || over(a.positions, 4 * rows) || over(a.base, 4 * static_cast<int64_t>(a.n_req)))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: q_out or k_out overlaps another tensor and is not q or k itself", who);
  RotateParams p = {};
  p.a = a;
  p.rows = rows;
  p.lanes = a.head_dim / 16;
  p.pairs = a.rot / 16;
  p.one_over = 1.0f / static_cast<float>(a.head_dim);
  int g = 2;
  while (g < p.lanes) g *= 2;
  // All heads of a row to a CTA where they fit, as many rows beside each other as make 256 threads, and two of those one
  // after the other, while two CTAs an SM are left.
  const int heads = a.n_q + a.n_kv, most = kRotateThreads / g, parts = (heads + most - 1) / most;
  p.heads = (heads + parts - 1) / parts;
  auto enough = [&](int n) { return n * (a.rot / 2) <= kMaxAngles && rows >= 2 * kSms * static_cast<int64_t>(n); };
  p.at_once = 256 / (p.heads * g) > 1 ? 256 / (p.heads * g) : 1;
  while (p.at_once > 1 && !enough(p.at_once)) --p.at_once;
  const int sequence = enough(2 * p.at_once) ? 2 : 1;
  const int threads = (p.at_once * p.heads * g + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>((rows + p.at_once * sequence - 1) / (p.at_once * sequence)), static_cast<unsigned>(parts));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_launched(who, g == 2 ? launch<2>(p, sequence, grid, threads, st) : g == 4 ? launch<4>(p, sequence, grid, threads, st) : g == 8 ? launch<8>(p, sequence, grid, threads, st) : launch<16>(p, sequence, grid, threads, st));
}
