// dt_linear for one or two tokens: weights straight from memory to registers, fp32 products on the ordinary cores.
//
// Every lane has 8 pieces of 16 bytes of the weights on their way before it uses one, and takes the tokens' pieces, which
// all warps read, from L1.  Where there are enough rows of weight to keep 16 warps an SM busy, a warp has two of them (with
// a gate one, and the gate's); else the four warps of a CTA share the inner dimension of four rows, so that few rows
// keep as many bytes in flight as many do.  Products are added in pairs of channels (fma.rn.f32x2), then over lanes
// and warps.  us by a warp alone, by four and by the
// tensor-core kernels for few tokens, one token: 2560 to 6144 7.2, 8.0, 9.6; 4096 to 2560 7.9, 5.6, 8.1; 10240 to 2560 16.7, 10.6, 12.9;
// 2560 to 2 x 10240 18.6, 19.2, 20.7; two tokens: 8.0, 9.5, 9.5; 8.5, 5.9, 8.1; 17.6, 10.8, 13.0; 20.7, 22.5, 21.0; with three, products and
// the tokens' reads take over: 2560 to 6144 11.4, 10.4, 9.2.
// Bound by the latency of that stream: a warp asks for its next pieces when it has used the ones before, three times one after the other
// for 2560 channels, so that one token streams 4.3 TB/s to 6144 outputs and 5.6 to 2 x 10240; no tensor memory, barrier or cluster stands
// before the first byte.
#include "linear.cuh"
#include "kv_flash.cuh"

namespace dt {
namespace {

constexpr int kTokenThreads = 128, kTokenWarps = kTokenThreads / 32;

DT_DEVINL uint64_t pair_of(uint32_t w) { return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

// 16 bytes that are read once.  (volatile: no load may be moved before dt_grid_wait)
DT_DEVINL uint4 stream16(const uint4* at) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at) : "memory");
  return v;
}

struct TokenOperands {
  const uint16_t* x;
  const uint16_t* w;
  const uint16_t* g;
  int64_t x_stride, w_stride, g_stride;
  int inner;
};

// SHARE: warps that share a row's inner dimension, 1 or all four.
template <int SIDES, int T, int SHARE>
__global__ void __launch_bounds__(kTokenThreads) k_token(const TokenOperands o, const LinearParams p) {
  // rows of weight and gate of a warp (of the CTA), outputs of those, pieces of each on their way
  constexpr int kStreams = SHARE == 1 ? 2 : 4, ROWS = kStreams / SIDES, AHEAD = 8 / kStreams, STEP = 32 * SHARE;
  __shared__ float sums[SHARE][kStreams * T];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = SHARE == 1 ? lane : static_cast<int>(threadIdx.x);
  const int n0 = (SHARE == 1 ? static_cast<int>(blockIdx.x) * kTokenWarps + warp : static_cast<int>(blockIdx.x)) * ROWS;
  if (SHARE == 1 && n0 >= p.outer) return;
  const uint4* row[kStreams];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t n = min(n0 + r, p.outer - 1);  // (rows behind the last are the last once more, and not written)
    row[r] = reinterpret_cast<const uint4*>(o.w + n * o.w_stride);
    if (SIDES == 2) row[ROWS + r] = reinterpret_cast<const uint4*>(o.g + n * o.g_stride);
  }
  uint64_t acc[kStreams][T];
#pragma unroll
  for (int r = 0; r < kStreams; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = 0;
  const int pieces = o.inner / 8;
  dt_grid_wait();
  for (int k = tid; k < pieces; k += STEP * AHEAD) {
    uint4 w[AHEAD][kStreams];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int r = 0; r < kStreams; ++r)
        if (k + STEP * u < pieces) w[u][r] = stream16(row[r] + k + STEP * u);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (k + STEP * u >= pieces) break;
      uint4 x[T];
#pragma unroll
      for (int t = 0; t < T; ++t) x[t] = reinterpret_cast<const uint4*>(o.x + t * o.x_stride)[k + STEP * u];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t x2[T];
#pragma unroll
        for (int t = 0; t < T; ++t) x2[t] = pair_of(i == 0 ? x[t].x : i == 1 ? x[t].y : i == 2 ? x[t].z : x[t].w);
#pragma unroll
        for (int r = 0; r < kStreams; ++r) {
          const uint64_t w2 = pair_of(i == 0 ? w[u][r].x : i == 1 ? w[u][r].y : i == 2 ? w[u][r].z : w[u][r].w);
#pragma unroll
          for (int t = 0; t < T; ++t) acc[r][t] = fma2(w2, x2[t], acc[r][t]);
        }
      }
    }
  }
  float mine = 0.0f;  // of stream r and token t, with thread r T + t
#pragma unroll
  for (int r = 0; r < kStreams; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float lo, hi;
      f32x2_parts(acc[r][t], lo, hi);
      const float a = warp_sum(lo + hi);
      if (lane == r * T + t) mine = a;
    }
  if (SHARE > 1) {
    if (lane < kStreams * T) sums[warp][lane] = mine;
    __syncthreads();
    if (tid < kStreams * T) mine = (sums[0][tid] + sums[SHARE / 4][tid]) + (sums[SHARE / 2][tid] + sums[SHARE - 1][tid]);
    if (warp > 0) return;
  }
  static_assert(SHARE == 1 || SHARE == 4, "");
  const float gate = SIDES == 2 ? __shfl_down_sync(0xFFFFFFFFu, mine, ROWS * T) : 0.0f;
  const int r = lane / T, t = lane - r * T, n = n0 + r;
  if (r >= ROWS || n >= p.outer) return;
  finish<SIDES>(p, t, n, mine, gate);
}

template <int SIDES, int T>
cudaError_t launch(const TokenOperands& o, const LinearParams& p, cudaStream_t st) {
  if (static_cast<int64_t>(p.outer) * SIDES / 2 >= 16 * kSms) {
    const int rows = kTokenWarps * 2 / SIDES;
    return launch_behind(k_token<SIDES, T, 1>, static_cast<unsigned>((p.outer + rows - 1) / rows), kTokenThreads, 0, st, 1, o, p);
  } else {
    const int rows = 4 / SIDES;
    return launch_behind(k_token<SIDES, T, 4>, static_cast<unsigned>((p.outer + rows - 1) / rows), kTokenThreads, 0, st, 1, o, p);
  }
}

}  // namespace

cudaError_t launch_linear_token(const dt_linear_args& a, const LinearParams& p, cudaStream_t st) {
  const TokenOperands o = {static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.weight), static_cast<const uint16_t*>(a.gate),
                           a.x_row_stride, a.weight_row_stride, a.gate_row_stride, a.inner};
  if (p.rows == 1) return a.gate ? launch<2, 1>(o, p, st) : launch<1, 1>(o, p, st);
  return a.gate ? launch<2, 2>(o, p, st) : launch<1, 2>(o, p, st);
}

}  // namespace dt
