// What the kernels of dt_linear share: arguments on the device, activations, the last step of an output.
#pragma once

#include "kv.cuh"

namespace dt {

struct LinearParams {
  const uint16_t* bias;
  const uint16_t* gate_bias;
  const uint16_t* residual;
  void* out;
  int64_t residual_stride, out_stride;
  int rows, outer, inner, k_blocks;  // k_blocks: of 64
  int per, k_steps;           // blocks of a step, steps
  int segment_steps;          // steps that one accumulator adds
  int sum_tokens;             // tokens whose sums stand in shared memory
  int activation, out_fp32;
  int bn, stages, tmem_cols;        // bn: few rows: tokens of a tile; many: its columns (with a gate, two for an output)
  int split;                  // CTAs of a cluster
  uint32_t stage_bytes;
  int m_tiles, n_tiles, tile_outs;  // tiles of tokens, of outputs, and outputs of a tile
  int wide;  // outputs (and residuals) are written and read 4 at a time, or 16 bytes where rows are many
  int32_t* status;
};

template <int ACT>
DT_DEVINL float activate(float z) {
  if (ACT == DT_ACT_RELU) return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
  if (ACT == DT_ACT_SILU) return z / (1.0f + expf(-z));
  if (ACT == DT_ACT_GELU) return 0.5f * z * erfcf(-0.707106781186547524f * z);
  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
  if (ACT == DT_ACT_GELU_TANH) return z / (1.0f + expf(-1.59576912160573071f * fmaf(0.044715f * z * z, z, z)));
  return z;
}
template <int ACT, int N>
DT_DEVINL void activate_all(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = activate<ACT>(v[i]);
}
template <int N>
DT_DEVINL void activate(float (&v)[N], int act) {
  switch (act) {
    case DT_ACT_RELU: activate_all<DT_ACT_RELU>(v); break;
    case DT_ACT_SILU: activate_all<DT_ACT_SILU>(v); break;
    case DT_ACT_GELU: activate_all<DT_ACT_GELU>(v); break;
    case DT_ACT_GELU_TANH: activate_all<DT_ACT_GELU_TANH>(v); break;
    default: break;
  }
}

// One output, column n of row t: the sums of the product (and of the gate's) in, bias, activation and residual, one
// rounding, out.
template <int SIDES>
DT_DEVINL void finish(const LinearParams& p, int64_t t, int n, float product, float gate) {
  float y[1] = {product}, z[1] = {gate};
  if (p.bias) y[0] += bf16_to_f32(p.bias[n]);
  if (SIDES == 2) {
    if (p.gate_bias) z[0] += bf16_to_f32(p.gate_bias[n]);
    activate(z, p.activation);
    y[0] *= z[0];
  } else {
    activate(y, p.activation);
  }
  if (p.residual) y[0] += bf16_to_f32(p.residual[t * p.residual_stride + n]);
  if (p.out_fp32) static_cast<float*>(p.out)[t * p.out_stride + n] = y[0];
  else static_cast<__nv_bfloat16*>(p.out)[t * p.out_stride + n] = __float2bfloat16_rn(y[0]);
}

// Four neighbouring outputs from column n on (those behind the last column are left out) of rows t, t + step, .. (`count` of N): the
// product's sums y and the gate's z.  All rows step by step together: a warp's own chain of instructions is what an epilogue of few
// warps takes its time for.
template <int SIDES, int N>
DT_DEVINL void finish_rows(const LinearParams& p, int64_t t, int step, int count, int n, float (&y)[4 * N], float (&z)[4 * N]) {
  if (n >= p.outer) return;
  if (!p.wide || n + 4 > p.outer) {
#pragma unroll
    for (int i = 0; i < 4 * N; ++i)
      if (i / 4 < count && n + i % 4 < p.outer) finish<SIDES>(p, t + i / 4 * step, n + i % 4, y[i], z[i]);
    return;
  }
  uint2 r[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    r[i] = p.residual && i < count ? *reinterpret_cast<const uint2*>(p.residual + (t + i * step) * p.residual_stride + n) : make_uint2(0, 0);
  if (p.bias) {
    float b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = bf16_to_f32(p.bias[n + j]);
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) y[i] += b[i % 4];
  }
  if (SIDES == 2) {
    if (p.gate_bias) {
      float b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = bf16_to_f32(p.gate_bias[n + j]);
#pragma unroll
      for (int i = 0; i < 4 * N; ++i) z[i] += b[i % 4];
    }
    activate(z, p.activation);
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) y[i] *= z[i];
  } else {
    activate(y, p.activation);
  }
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      y[4 * i] += __uint_as_float(r[i].x << 16);
      y[4 * i + 1] += __uint_as_float(r[i].x & 0xFFFF0000u);
      y[4 * i + 2] += __uint_as_float(r[i].y << 16);
      y[4 * i + 3] += __uint_as_float(r[i].y & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i >= count) break;
    const int64_t at = (t + i * step) * p.out_stride + n;
    if (p.out_fp32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(y[4 * i], y[4 * i + 1]), b = __floats2bfloat162_rn(y[4 * i + 2], y[4 * i + 3]);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
}

// Rows of bf16 (stride in elements) as a 3D map, swizzled by 128 bytes: boxes of 64 channels x box_rows rows x per blocks of
// 64 channels, which have to be whole where per > 1 (per 1: the first coordinate is the channel, the third 0).
bool linear_map(CUtensorMap* m, const void* base, int inner, int64_t rows, int64_t stride, int box_rows, int per);

constexpr int kSegmentBlocks = 8;          // blocks of 64 channels that an accumulator adds, for outputs in 32 bits
// Shared memory of launch_linear_wide: the places through which its 8 epilogue warps write 32 x 32 outputs, and its stages.
constexpr uint32_t wide_staging(bool fp32) { return fp32 ? 4096 : 2048; }
constexpr uint32_t wide_ring(bool fp32) { return 224 * 1024 - 8 * wide_staging(fp32); }
constexpr int kTokensMost = 2;  // of launch_linear_token
cudaError_t launch_linear_token(const dt_linear_args& a, const LinearParams& p, cudaStream_t st);
cudaError_t launch_linear_wide(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, bool gate,
                               cudaStream_t st);

}  // namespace dt
