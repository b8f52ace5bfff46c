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

// Four neighbouring outputs from column n on (those behind the last column are left out).
template <int SIDES>
DT_DEVINL void finish4(const LinearParams& p, int64_t t, int n, const float4& y4, const float4& z4) {
  float y[4] = {y4.x, y4.y, y4.z, y4.w}, z[4] = {z4.x, z4.y, z4.z, z4.w};
  if (!p.wide || n + 4 > p.outer) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.outer) finish<SIDES>(p, t, n + i, y[i], z[i]);
    return;
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += bf16_to_f32(p.bias[n + i]);
  }
  if (SIDES == 2) {
    if (p.gate_bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] += bf16_to_f32(p.gate_bias[n + i]);
    }
    activate(z, p.activation);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= z[i];
  } else {
    activate(y, p.activation);
  }
  if (p.residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(p.residual + t * p.residual_stride + n);
    y[0] += __uint_as_float(r.x << 16);
    y[1] += __uint_as_float(r.x & 0xFFFF0000u);
    y[2] += __uint_as_float(r.y << 16);
    y[3] += __uint_as_float(r.y & 0xFFFF0000u);
  }
  const int64_t at = t * p.out_stride + n;
  if (p.out_fp32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
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
