// dt_linear: matrix product with bias, activation or gate, and residual, on tcgen05.
//
// k_few: 128 rows of weight are the product's rows (its A operand) and up to 256 tokens its columns, so that few tokens
// still fill the tensor core's 128 lanes, and the kernel streams the weights once; with a gate, 128 rows of each of the
// two matrices, whose sums meet in one epilogue.  Where the tiles are fewer than the SMs, a cluster shares one: every CTA
// takes a part of the inner dimension, and the partial sums, fp32 in shared memory, are added over distributed shared
// memory in the order of ranks, each CTA finishing a part of the tile.  Tensor memory is given back before the cluster's
// barrier: a CTA that holds some waits for no other, so that kernels side by side on an SM cannot wait in a circle.
#include "linear.cuh"
#include "cluster.cuh"
#include "kv_flash.cuh"

namespace dt {
namespace {

constexpr int kFewThreads = 256;
constexpr uint32_t kTileBytes = 128 * 128;  // 128 rows of 64 bf16

// Shared memory from the 1024-aligned base: the ring of stages (and behind the products the partial sums, in its place),
// then the barriers.
DT_HOST_DEVICE_INLINE uint32_t few_bars(const LinearParams& p, int sides) {
  const uint32_t ring = p.stages * p.stage_bytes, sums = p.bn * sides * 512u;
  return ring > sums ? ring : sums;
}

template <int SIDES>
__global__ void __launch_bounds__(kFewThreads)
    k_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_g,
          const __grid_constant__ CUtensorMap tm_x, const LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + few_bars(p, SIDES));
  uint64_t* empty = full + p.stages;
  uint64_t* done = empty + p.stages;
  uint64_t* drained = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.split, tile = static_cast<int>(blockIdx.x) / p.split;
  const int n0 = tile * 128, t0 = static_cast<int>(blockIdx.y) * p.bn;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / p.split);
  const uint64_t stream = l2_policy_evict_first(), keep = l2_policy_evict_last();
  auto load = [&](int kb, uint32_t stage) {
    uint8_t* at = smem + stage * p.stage_bytes;
    mbar_arrive_expect_tx(&full[stage], p.stage_bytes);
    if (SIDES == 2) tma_load_2d(at, &tm_g, &full[stage], kb * 64, n0, stream);
    tma_load_2d(at + (SIDES - 1) * kTileBytes, &tm_w, &full[stage], kb * 64, n0, stream);
    tma_load_2d(at + SIDES * kTileBytes, &tm_x, &full[stage], kb * 64, t0, keep);
  };
  // the first loads are under way before tensor memory is asked for
  const int ahead = min(p.stages, kb1 - kb0);
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      mbar_init(done, 1);
      mbar_init(drained, 1);
      fence_mbar_init();
      for (int s = 0; s < ahead; ++s) load(kb0 + s, s);
    }
    __syncwarp();
  }
  if (warp == 1) tmem_alloc(tmem_slot, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    for (int kb = kb0 + ahead; kb < kb1; ++kb) {
      ok = warp_wait(&empty[stage], phase);
      if (!ok) break;
      if (elect_one()) load(kb, stage);
      __syncwarp();
      if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(128, p.bn);
    uint32_t stage = 0, phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = warp_wait(&full[stage], phase);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem + stage * p.stage_bytes);
      const uint64_t a = sdesc_k_sw128(at), b = sdesc_k_sw128(at + SIDES * kTileBytes);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int s = 0; s < SIDES; ++s)
            tc_mma_bf16(tmem + s * p.bn, a + ((s * kTileBytes + k * 32) >> 4), b + (k * 32 >> 4), idesc, kb != kb0 || k != 0);
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
    }
    if (elect_one()) tc_commit(ok ? done : drained);
    __syncwarp();
    // (where a wait gave up: no product may outlive its operands and tensor memory)
    if (!ok) mbar_wait(drained, 0, nullptr);
  }

  // the sums into shared memory, [token][side][row], where the stages were (all of them have been used)
  float* sums = reinterpret_cast<float*>(smem);
  const int tokens = min(p.bn, p.rows - t0);
  ok = ok && warp_wait(done, 0);
  tc_fence_after();
  if (ok) {
    const int quarter = warp & 3;
    for (int x = warp >> 2; x < SIDES * p.bn / 16; x += 2) {
      const int side = x / (p.bn / 16), c0 = (x - side * (p.bn / 16)) * 16;
      uint32_t v[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + side * p.bn + c0, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) sums[((c0 + j) * SIDES + side) * 128 + quarter * 32 + lane] = __uint_as_float(v[j]);
    }
  } else if (p.status && lane == 0) {
    atomicOr(p.status, DT_KV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  __syncwarp();
  if (p.split > 1) cluster_barrier();
  // four neighbouring rows of weight for a token at a time, an equal share of them for each rank
  const int units = tokens * 32;
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (rank + 1) / p.split);
  for (int u = static_cast<int>(static_cast<int64_t>(units) * rank / p.split) + tid; u < u1; u += kFewThreads) {
    const int t = u >> 5, f = (u & 31) * 4;
    if (n0 + f >= p.outer) continue;
    float4 acc[SIDES];
#pragma unroll
    for (int s = 0; s < SIDES; ++s) {
      const float* at = sums + (t * SIDES + s) * 128 + f;
      acc[s] = p.split > 1 ? peer_ld4(peer_addr(at, 0)) : *reinterpret_cast<const float4*>(at);
      for (int r = 1; r < p.split; ++r) {
        const float4 v = peer_ld4(peer_addr(at, r));
        acc[s].x += v.x, acc[s].y += v.y, acc[s].z += v.z, acc[s].w += v.w;
      }
    }
    finish4<SIDES>(p, t0 + t, n0 + f, acc[SIDES - 1], acc[0]);
  }
  if (p.split > 1) cluster_barrier();  // (no CTA leaves while its sums are read)
}

template <int SIDES>
cudaError_t launch_few(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, cudaStream_t st) {
  const uint32_t smem = 1024 + few_bars(p, SIDES) + (2 * p.stages + 2) * 8 + 16;
  cudaError_t e = cudaFuncSetAttribute(k_few<SIDES>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.outer + 127) / 128 * p.split), static_cast<unsigned>((p.rows + p.bn - 1) / p.bn));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_few<SIDES>, w, g, x, p);
}

// Few tokens: one tile of them, padded to 16, two CTAs an SM where their sums leave room for it, and clusters of as many
// CTAs as leave all of them beside each other (clusters do not fill every SM), with four blocks of 64 or more each.
void plan_few(LinearParams& p, int sides) {
  const int most = 256 / sides, token_tiles = (p.rows + most - 1) / most;
  p.bn = ((p.rows + token_tiles - 1) / token_tiles + 15) & ~15;
  p.tmem_cols = 32;
  while (p.tmem_cols < sides * p.bn) p.tmem_cols *= 2;
  p.stage_bytes = sides * kTileBytes + p.bn * 128;
  const bool two = sides * p.bn <= 128;
  p.stages = static_cast<int>((two ? 110u * 1024 : 220u * 1024) / p.stage_bytes);
  if (p.stages > 8) p.stages = 8;
  const int64_t tiles = static_cast<int64_t>((p.outer + 127) / 128) * token_tiles;
  p.split = 1;
  while (p.split < 8 && tiles * (p.split + 1) <= (two ? 2 * kSms : kSms) * 7 / 8 && p.k_blocks >= 4 * (p.split + 1)) ++p.split;
}

// Many tokens: the tile's columns so that the pairs' rounds of tiles cost least, a tile as much as its columns and 32 more.
void plan_many(LinearParams& p, int sides) {
  p.m_tiles = (p.rows + 255) / 256;
  int64_t least = INT64_MAX;
  for (int bn = 256; bn >= 64; bn -= 32 * sides) {
    const int outs = bn / sides;
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * ((p.outer + outs - 1) / outs);
    const int64_t cost = (tiles + kSms / 2 - 1) / (kSms / 2) * (bn + 32);
    if (cost < least) {
      least = cost;
      p.bn = bn;
      p.tile_outs = outs;
      p.n_tiles = (p.outer + outs - 1) / outs;
    }
  }
}

}  // namespace

bool make_tmap_bf16_2d(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t rows, uint64_t row_stride_bytes, uint32_t box_rows);

}  // namespace dt

extern "C" dt_status dt_linear(const dt_linear_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_linear";
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  const dt_linear_args& a = *args;
  if (a.rows < 0 || a.rows > 0x7FFFFFFF - 256) return kv_fail(DT_ERR_SHAPE, "%s: rows outside 0..2^31-257", who);
  if (a.outer < 1 || a.outer > 0x7FFFFFFF - 256) return kv_fail(DT_ERR_SHAPE, "%s: outer outside 1..2^31-257", who);
  if (a.inner < 8 || a.inner % 8 != 0) return kv_fail(DT_ERR_SHAPE, "%s: inner %d is not a multiple of 8", who, a.inner);
  if (a.activation < DT_ACT_NONE || a.activation > DT_ACT_GELU_TANH)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: unknown activation %d", who, a.activation);
  if (a.gate_bias && !a.gate) return kv_fail(DT_ERR_INVALID_ARG, "%s: a gate_bias without a gate", who);
  if (a.rows == 0) return DT_OK;
  auto operand = [&](const void* d, int64_t stride, int64_t rows) {
    return d && (reinterpret_cast<uintptr_t>(d) & 15u) == 0 && (rows == 1 || (stride >= a.inner && stride % 8 == 0));
  };
  if (!operand(a.x, a.x_row_stride, a.rows) || !operand(a.weight, a.weight_row_stride, a.outer) || (a.gate && !operand(a.gate, a.gate_row_stride, a.outer)))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: x, weight or gate is null or misaligned, or its rows overlap or are not multiples of 8 apart", who);
  const uintptr_t out = reinterpret_cast<uintptr_t>(a.out), bytes = a.out_fp32 ? 4 : 2;
  if (!a.out || out % bytes != 0 || (a.rows > 1 && a.out_row_stride < a.outer))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: out is null or misaligned, or its rows overlap", who);
  if (((reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.bias) | reinterpret_cast<uintptr_t>(a.gate_bias)) & 1u) != 0)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: misaligned residual or bias", who);
  LinearParams p = {};
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.gate_bias = static_cast<const uint16_t*>(a.gate_bias);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.residual_stride = a.residual_row_stride;
  p.out = a.out;
  p.out_stride = a.out_row_stride;
  p.rows = static_cast<int>(a.rows);
  p.outer = a.outer;
  p.k_blocks = (a.inner + 63) / 64;
  p.activation = a.activation;
  p.out_fp32 = a.out_fp32 != 0;
  p.status = a.status;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.rows <= kTokensMost) return kv_launched(who, launch_linear_token(a, p, st));
  const int sides = a.gate ? 2 : 1;
  const bool many = p.rows > 256;
  const uintptr_t res = reinterpret_cast<uintptr_t>(a.residual);
  const int64_t at_once = many ? 16 / static_cast<int64_t>(bytes) : 4;  // outputs written together
  p.wide = out % (at_once * bytes) == 0 && (a.rows == 1 || a.out_row_stride % at_once == 0) &&
           (!res || (many ? res % 16 == 0 && a.residual_row_stride % 8 == 0 : res % 8 == 0 && (a.rows == 1 || a.residual_row_stride % 4 == 0)));
  if (many) {
    plan_many(p, sides);
    if (static_cast<int64_t>(p.m_tiles) * p.n_tiles > (1 << 30)) return kv_fail(DT_ERR_SHAPE, "%s: more than 2^30 tiles", who);
  } else {
    plan_few(p, sides);
    if (static_cast<int64_t>((a.outer + 127) / 128) * p.split > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: too many tiles", who);
  }
  auto stride = [&](int64_t s, int64_t rows) { return static_cast<uint64_t>(rows == 1 ? (a.inner + 7) / 8 * 8 : s) * 2; };
  CUtensorMap w, g, x;
  if (!make_tmap_bf16_2d(&w, a.weight, a.inner, a.outer, stride(a.weight_row_stride, a.outer), many ? p.bn / 2 : 128) ||
      !make_tmap_bf16_2d(&g, a.gate ? a.gate : a.weight, a.inner, a.outer, stride(a.gate ? a.gate_row_stride : a.weight_row_stride, a.outer), many ? p.bn / 2 : 128) ||
      !make_tmap_bf16_2d(&x, a.x, a.inner, a.rows, stride(a.x_row_stride, a.rows), many ? 128 : p.bn))
    return kv_fail(DT_ERR_SHAPE, "%s: strides that a tensor map does not take (2^40 bytes and more)", who);
  if (many) return kv_launched(who, launch_linear_wide(w, g, x, p, sides == 2, st));
  return kv_launched(who, sides == 2 ? launch_few<2>(w, g, x, p, st) : launch_few<1>(w, g, x, p, st));
}
