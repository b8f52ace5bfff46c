// dt_prompt_attention: causal attention over packed prompts, on the tensor cores.
//
// Rows of a tile.  128 rows = (128 / group) positions x the group's query heads of
// one key/value head, so that all of a group's heads use each key tile once and
// short prompts fill tiles `group` times better than one head at a time would.  A
// CTA takes two such tiles (neighbouring positions) and walks the key tiles up to
// its last position; causality costs the part of one or two diagonal tiles.
//
// What bounds it: 4 * head_dim flops for every visible (row, key) on the tensor
// cores, and about as many cycles of exponentials and their surroundings on the
// ordinary cores; the two overlap (kv_flash.cuh).  One warp feeds K and V by TMA
// into a ring of five stages, one thread issues the products, two warpgroups do
// the softmax of a tile each.  CTAs are started heaviest first.
//
// P is rounded to bf16 (operands of one product have one type, and V is bf16):
// 2^-8 relative a weight at most, as the rounding of the output itself.
//
// Tiles that hold keys which some row must not see are cleaned before their
// product (0 * NaN would reach that row): values behind the sequence become
// zeros, and a key whose value is not finite becomes zeros and is noted, which
// makes the rows that do see it NaN.
#include <cuda.h>

#include "kv_flash.cuh"

namespace dt {
namespace {

constexpr int kStages = 5;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp = 10, kCleanWarps = 1;
constexpr int kPromptThreads = 32 * (kCleanWarp + kCleanWarps);
// Tiles of which some row does not see all: keys behind the first of a CTA's (at most 256) positions
// lie in three at most, so each has a barrier and a word of its own.
constexpr int kMaskedTiles = 3;

struct PromptParams {
  __nv_bfloat16* out;
  float* lse;
  const int32_t* row_start;
  int64_t n_rows, out_row_stride, out_head_stride;
  int n_seq, n_q, n_kv, group, positions;  // positions: of a tile (128 / group)
  int slots;                               // CTAs per key/value head
  float c;                                 // scale * log2(e)
};

template <int HD>
struct PromptSmem {
  static constexpr uint32_t kOperand = kOperandBytes<HD>;
  static constexpr uint32_t kQ = 0, kRing = 2 * kOperand, kBars = kRing + kStages * kOperand;
  static constexpr uint32_t kBytes = kBars + 512 + 1024;  // + alignment
};

DT_DEVINL void tma_load_3d(uint32_t dst, const void* tmap, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

template <int HD>
__global__ void __launch_bounds__(kPromptThreads, 1)
    k_prompt(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const PromptParams p) {
  using Smem = PromptSmem<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem::kBars);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;
  uint64_t* s_full = q_full + 1;  // [2]
  uint64_t* p_full = s_full + 2;  // [2]
  uint64_t* o_full = p_full + 2;  // [2]
  uint64_t* clean = o_full + 2;   // [kMaskedTiles] a masked tile's values are clean
  uint64_t* dirty = clean + kMaskedTiles;  // [kMaskedTiles] its values are there to be cleaned
  uint32_t* bad_key = reinterpret_cast<uint32_t*>(dirty + kMaskedTiles);  // [kMaskedTiles][4] keys of the masked tiles whose values are not finite
  __shared__ uint32_t tmem_slot;
  __shared__ int s_seq[3];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.x % p.n_kv, slot = p.slots - 1 - static_cast<int>(blockIdx.x / p.n_kv);
  const int span = 2 * p.positions;  // positions of a CTA

  // Sequence i's CTAs stand from start_i / span + i on: at least as many places as it needs, found without a sum.
  if (tid == 0) s_seq[2] = 0;
  if (warp == kMmaWarp) tmem_alloc(&tmem_slot, 512);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < kMaskedTiles; ++i) {
      mbar_init(&clean[i], kCleanWarps);
      mbar_init(&dirty[i], 1);
    }
    for (int i = 0; i < 4 * kMaskedTiles; ++i) bad_key[i] = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  {
    const int first = p.row_start[0];
    for (int i = tid; i < p.n_seq; i += kPromptThreads) {
      const int64_t a = p.row_start[i], b = p.row_start[i + 1];
      const int64_t at = (a - first) / span + i;
      if (slot >= at && slot < (b - first) / span + i + 1 && a >= 0 && b <= p.n_rows && (slot - at) * span < b - a) {
        s_seq[0] = static_cast<int>(a);
        s_seq[1] = static_cast<int>(b - a);
        s_seq[2] = static_cast<int>(slot - at) + 1;
      }
    }
  }
  __syncthreads();
  const uint32_t tmem = tmem_slot;
  const int row0 = s_seq[0], len = s_seq[1], block = s_seq[2] - 1;
  if (block >= 0) {
    const int pos0 = block * span;
    // key tiles that each row tile walks, and the first one of which some row does not see all
    int n_tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int a = pos0 + t * p.positions;
      n_tiles[t] = a < len ? (min(len, a + p.positions) + kKeyTile - 1) / kKeyTile : 0;
    }
    const int n = max(n_tiles[0], n_tiles[1]);
    const int masked0 = (pos0 + 1) / kKeyTile;  // tiles from here on hold a key behind pos0
    const uint32_t q_s = smem_u32(smem + Smem::kQ), ring = smem_u32(smem + Smem::kRing);

    if (warp == kLoadWarp) {
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, 2u * (HD / 64) * 128u * p.group * p.positions);
        for (int t = 0; t < 2; ++t)
          for (int h = 0; h < HD / 64; ++h)
            tma_load_3d(q_s + t * Smem::kOperand + h * kHalfBytes, &tm_q, q_full, h * 64, kvh * p.group,
                        row0 + pos0 + t * p.positions);
        // K(0), V(0), K(1), V(1), ...
        uint32_t stage = 0, phase = 0;
        for (int i = 0; i < 2 * n; ++i) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, nullptr)) break;
          mbar_arrive_expect_tx(&full[stage], Smem::kOperand);
          for (int h = 0; h < HD / 64; ++h)
            tma_load_3d(ring + stage * Smem::kOperand + h * kHalfBytes, (i & 1) ? &tm_v : &tm_k, &full[stage], h * 64, kvh,
                        row0 + (i >> 1) * kKeyTile);
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
      }
    } else if (warp == kMmaWarp) {
      if (lane == 0) {
        auto full_wait = [&](int i) { return mbar_wait(&full[i % kStages], (i / kStages) & 1, nullptr); };
        auto at = [&](int i) { return ring + (i % kStages) * Smem::kOperand; };
        bool ok = mbar_wait(q_full, 0, nullptr) && full_wait(0);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (n_tiles[t] > 0) {
              issue_qk<HD, true>(tmem + t * 128, q_s + t * Smem::kOperand, at(0));
              tc_commit(&s_full[t]);
            }
          tc_commit(&empty[0]);
        }
        for (int j = 0; j < n && ok; ++j) {
          const int vi = 2 * j + 1, ki = 2 * j + 2;
          // (the cleaning warp cannot wait on the ring itself: it would meet its stage in some earlier turn)
          ok = full_wait(vi);
          if (ok && j >= masked0) mbar_arrive(&dirty[j - masked0]);
          ok = ok && (j + 1 >= n || full_wait(ki));
          if (ok && j >= masked0) ok = mbar_wait(&clean[j - masked0], 0, nullptr);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || j >= n_tiles[t]) continue;
            if (!mbar_wait(&p_full[t], j & 1, nullptr)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            issue_pv<HD, true>(tmem + 256 + t * 128, tmem + t * 128, at(vi), j == 0);
            if (j + 1 < n_tiles[t]) {
              issue_qk<HD, true>(tmem + t * 128, q_s + t * Smem::kOperand, at(ki));
              tc_commit(&s_full[t]);
            } else {
              tc_commit(&o_full[t]);
            }
          }
          if (ok) {
            tc_commit(&empty[vi % kStages]);
            if (j + 1 < n) tc_commit(&empty[ki % kStages]);
          }
        }
      }
    } else if (warp >= kCleanWarp) {
      // values of the masked tiles, 16 bytes of each half at a time
      const int ct = tid - kCleanWarp * 32;
      for (int j = masked0; j < n; ++j) {
        const int i = 2 * j + 1;
        if (!mbar_wait(&dirty[j - masked0], 0, nullptr)) break;
        uint8_t* v = smem + Smem::kRing + (i % kStages) * Smem::kOperand;
        uint32_t* bad = bad_key + (j - masked0) * 4;
        const int valid = len - j * kKeyTile;
        for (int x = ct; x < kKeyTile * 8; x += 32 * kCleanWarps) {
          const int key = x >> 3;
          uint4* at[HD / 64];
          bool nan = false;
#pragma unroll
          for (int h = 0; h < HD / 64; ++h) {
            at[h] = reinterpret_cast<uint4*>(v + h * kHalfBytes + x * 16);  // (the swizzle stays within a key's row)
            const uint4 w = *at[h];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              nan |= (ws[k] & 0x7F80u) == 0x7F80u || (ws[k] & 0x7F800000u) == 0x7F800000u;
          }
          if (key >= valid || nan) {
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) *at[h] = make_uint4(0, 0, 0, 0);
            if (key < valid) atomicOr(&bad[key >> 5], 1u << (key & 31));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&clean[j - masked0]);
      }
    } else {
      // softmax: warpgroup t, a row a thread
      const int t = warp >> 2, r = tid & 127;
      const int pos = pos0 + t * p.positions + r / p.group, head = kvh * p.group + r % p.group;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + 256 + t * 128 + lanes;
      const float c = p.c;
      float m = -INFINITY, l = 0.0f;  // m: the maximum in use, in powers of two
      bool ok = true;
      for (int j = 0; j < n_tiles[t]; ++j) {
        if (!mbar_wait(&s_full[t], j & 1, nullptr)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int w = 0; w < 4; ++w) tmem_ld32(s_at + 32 * w, s + 32 * w);
        tmem_wait_ld();
        const bool masked = (j + 1) * kKeyTile > pos0 + t * p.positions + 1;  // (for the tile's first row)
        const int seen = pos + 1 - j * kKeyTile;                              // of this tile's keys, by this row
        if (masked) {
          const float out = c >= 0.0f ? -INFINITY : INFINITY;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= seen) s[i] = __float_as_uint(out);
        }
        float top;
        if (c >= 0.0f) {
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i & 3] = fmaxf(x[i & 3], __uint_as_float(s[i]));
          top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        } else {
          float x[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i & 3] = fminf(x[i & 3], __uint_as_float(s[i]));
          top = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
        }
        top = c == 0.0f ? 0.0f : top * c;
        // (an infinite logit would make exp2(inf - inf): NaN, as the formula has it)
        const bool grow = top > m + 8.0f;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float m2 = fmaxf(m, top), f = m2 == -INFINITY ? 1.0f : ex2(m - m2);
          if (j > 0) rescale_o<HD>(o_at, f);
          l *= f;
          m = m2;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0 = ex2(fmaf(__uint_as_float(s[32 * w + 2 * i]), c, -base));
            float e1 = ex2(fmaf(__uint_as_float(s[32 * w + 2 * i + 1]), c, -base));
            if (masked) {
              if (32 * w + 2 * i >= seen) e0 = 0.0f;
              if (32 * w + 2 * i + 1 >= seen) e1 = 0.0f;
            }
            sum[(2 * i) & 3] += e0;
            sum[(2 * i + 1) & 3] += e1;
            pk[i] = pack_p<true>(e0, e1);
          }
          tmem_st16(s_at + 16 * w, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (n_tiles[t] > 0 && ok && mbar_wait(&o_full[t], 0, nullptr)) {
        tc_fence_after();
        // rows that see a key whose value is not finite (all cleaned tiles lie behind every o_full)
        for (int j = masked0; j < n_tiles[t]; ++j)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (bad_key[(j - masked0) * 4 + w] & first_bits(pos + 1 - j * kKeyTile, w)) l = NAN;
        const bool live = r < p.group * p.positions && pos < len;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        __nv_bfloat16* out = p.out + static_cast<int64_t>(row0 + pos) * p.out_row_stride + head * p.out_head_stride;
#pragma unroll
        for (int x = 0; x < HD; x += 32) {
          uint32_t v[32];
          tmem_ld32(o_at + x, v);
          tmem_wait_ld();
          if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 w;
              w.x = pack_p<true>(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv);
              w.y = pack_p<true>(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
              w.z = pack_p<true>(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv);
              w.w = pack_p<true>(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv);
              *reinterpret_cast<uint4*>(out + x + i) = w;
            }
          }
        }
        if (live && p.lse)
          p.lse[static_cast<int64_t>(row0 + pos) * p.n_q + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PromptParams& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_prompt<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptSmem<HD>::kBytes);
  if (e != cudaSuccess) return e;
  k_prompt<HD><<<static_cast<unsigned>(p.slots) * p.n_kv, kPromptThreads, PromptSmem<HD>::kBytes, st>>>(q, k, v, p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dt

extern "C" dt_status dt_prompt_attention(const dt_prompt_attention_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_prompt_attention";
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  const dt_prompt_attention_args& a = *args;
  if (a.n_seq < 1 || a.n_rows < 1 || a.n_kv < 1 || a.n_q < 1)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: need n_seq, n_rows, n_q, n_kv >= 1", who);
  if (a.head_dim != 64 && a.head_dim != 128)
    return kv_fail(DT_ERR_SHAPE, "%s: head_dim %d is not 64 or 128", who, a.head_dim);
  if (a.n_q % a.n_kv != 0 || a.n_q / a.n_kv > 128)
    return kv_fail(DT_ERR_SHAPE, "%s: %d query heads over %d key/value heads: need a multiple, at most 128 a head", who,
                   a.n_q, a.n_kv);
  if (a.n_rows > 0x7FFFFFFF - 256) return kv_fail(DT_ERR_SHAPE, "%s: n_rows above 2^31-257", who);
  if (!(a.scale - a.scale == 0.0f)) return kv_fail(DT_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (!a.row_start || !kv_rows_ok(a.q, a.q_row_stride, a.q_head_stride) || !kv_rows_ok(a.k, a.k_row_stride, a.k_head_stride) ||
      !kv_rows_ok(a.v, a.v_row_stride, a.v_head_stride) || !kv_rows_ok(a.out, a.out_row_stride, a.out_head_stride))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null or misaligned q, k, v, out or row_start", who);
  PromptParams p = {};
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.row_start = a.row_start;
  p.n_rows = a.n_rows;
  p.out_row_stride = a.out_row_stride;
  p.out_head_stride = a.out_head_stride;
  p.n_seq = a.n_seq;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.group = a.n_q / a.n_kv;
  p.positions = 128 / p.group;
  const int64_t slots = a.n_rows / (2 * p.positions) + a.n_seq;
  if (slots * a.n_kv > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: too many rows and heads for one launch", who);
  p.slots = static_cast<int>(slots);
  p.c = a.scale * kLog2e;
  CUtensorMap q, k, v;
  if (!make_tmap_bf16_heads(&q, a.q, a.head_dim, a.n_q, a.n_rows, a.q_head_stride, a.q_row_stride, p.group, p.positions) ||
      !make_tmap_bf16_heads(&k, a.k, a.head_dim, a.n_kv, a.n_rows, a.k_head_stride, a.k_row_stride, 1, kKeyTile) ||
      !make_tmap_bf16_heads(&v, a.v, a.head_dim, a.n_kv, a.n_rows, a.v_head_stride, a.v_row_stride, 1, kKeyTile))
    return kv_fail(DT_ERR_SHAPE, "%s: strides that a tensor map does not take (zero, or 2^40 bytes and more)", who);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_launched(who, a.head_dim == 64 ? launch<64>(q, k, v, p, st) : launch<128>(q, k, v, p, st));
}
