// dt_linear for many tokens: 256 tokens x up to 256 columns a tile, by pairs of CTAs.
//
// The two CTAs of a cluster run one product of 256 rows (tcgen05.mma.cta_group::2): each holds 128 tokens (operand A) and
// half of the tile's rows of weight (operand B), so that an SM stages 32 KB for 128 x 256 x 64 products where it would
// stage 48 KB alone.  With a gate the first CTA's half are rows of the gate and the second's the same rows of the
// weight: a token's two sums stand in one lane of tensor memory, 128 columns apart.
// Persistent: a pair takes every pairs-th tile, and its accumulators are two of 256 columns, so that the epilogue of a
// tile runs under the next one's products.  Warp 0 issues the copies (each CTA its own, counted on the first CTA's
// barrier), warp 1 of the first CTA the products, warps 4 to 11 the epilogue, a quarter of the lanes and every second
// group of 32 columns each.
// Outputs in 32 bits: an accumulator takes 512 channels (linear.cu says why), and the epilogue's warps hold a tile's sums, 128 a
// thread, in registers that the other warps give up.  Every change of accumulator costs about 500 clocks: 4096 tokens, 2560 to
// 10240 152 us, in bf16 119 us (by single CTAs, which stage twice as much, 220 us).
// Bound by the tensor cores where tiles are whole: 8192 tokens gated, 2560 to 2 x 10240 432 us in a burst at the full clock (2070 MHz; 1.99
// PFLOP/s, a library's product of the same operands 2.10), 507 us call after call, where the power limit lowers the clock; 4096 to 4096 141 us.
// Else by operands, of which a narrower tile brings as many for fewer products, and by whole tiles: 2080 tokens, 4096 to 2560 34 us, 1.3
// PFLOP/s, 144 tiles of 256 x 160 over 76 pairs, two a pair but for eight, so that an SM takes 113 GB/s (copies alone reach
// 137; tokens and weights by a warp each the same times), and the last 32 tokens cost as much as 256.
// Both CTAs hold all of their SM's tensor memory while they wait for one another: with 220 KB of shared memory no CTA
// that holds any can stand beside them, so that nobody waits in a circle.
#include "cluster.cuh"
#include "kv_flash.cuh"
#include "linear.cuh"

namespace dt {
namespace {

constexpr int kWideThreads = 384, kEpilogueWarps = 8;
constexpr int kOtherRegs = 72, kSumRegs = 216;  // of the warps that issue and of the epilogue's, outputs in 32 bits
constexpr uint32_t kHalf = 128 * 128;  // 128 rows of 64 bf16
constexpr uint32_t kWideSmem = 1024 + 224 * 1024 + 512;
static_assert(kWideSmem <= kSmemBytes, "");

DT_DEVINL void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
DT_DEVINL void tmem_dealloc_pair(uint32_t at, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
DT_DEVINL void tc_mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` in both CTAs once the products issued so far are complete.
DT_DEVINL void tc_commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}
// A step's rows into this CTA's shared memory, counted on a barrier of either CTA (a cluster address).
template <int PER>
DT_DEVINL void tma_load_pair(void* dst, const void* tmap, uint32_t bar, int step, int row, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(PER == 1 ? step * 64 : 0), "r"(row), "r"(PER == 1 ? 0 : step * PER), "l"(policy)
      : "memory");
}
DT_DEVINL void peer_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory"); }
// Bounded wait of a warp for arrivals from the whole cluster.
DT_DEVINL bool pair_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok = 0, n = 0;
  uint64_t t0 = 0;
  for (;;) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) break;
    if (t0 == 0) t0 = dt_globaltimer();
    if ((++n & 63u) == 0 && dt_globaltimer() - t0 > DT_WAIT_LIMIT_NS) break;
  }
  return __all_sync(0xFFFFFFFFu, ok != 0);
}

// Tiles in groups of 8 rows of tiles, whose tokens stay in L2 while the weights pass.
struct Place {
  int m0, n0;
};
DT_DEVINL Place place(const LinearParams& p, int tile) {
  const int group = tile / (8 * p.n_tiles), left = tile - group * 8 * p.n_tiles;
  const int rows = min(8, p.m_tiles - group * 8);
  const int n = left / rows;
  return {(group * 8 + left - n * rows) * 256, n * p.tile_outs};
}

// The 32 rows x 32 columns of a warp between memory and a row a lane, through the warp's own shared memory: several
// lanes read or write a row together.  E: bytes of an element.  Pieces of 16 bytes, swizzled.
template <int E>
DT_DEVINL uint32_t piece_at(int row, int k) {
  return E == 2 ? row * 64 + ((k ^ (row >> 1 & 3)) << 4) : row * 128 + ((k ^ (row & 7)) << 4);
}

// A warp's chunk of an output tile: rows t0 .. of 32, columns n .. of 32, of which `rows` and `cols` are there.
struct Chunk {
  int t0, n, rows, cols, lane;
  bool whole;  // 16 bytes at a time
  uint8_t* mine;
};
// The residual's, lanes 4 i .. 4 i + 3 a row.
DT_DEVINL void ask_residual(const LinearParams& p, const Chunk& at, uint4 (&res)[4]) {
  if (!p.residual || !at.whole) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (at.lane >> 2);
    res[i] = r < at.rows ? *reinterpret_cast<const uint4*>(p.residual + (at.t0 + r) * p.residual_stride + at.n + 8 * (at.lane & 3)) : make_uint4(0, 0, 0, 0);
  }
}
// y (and the gate's z): the sums of the product, a row a lane; bias, activation and residual, and out.
template <int SIDES, bool FULL>
DT_DEVINL void finish_chunk(const LinearParams& p, const Chunk& at, float (&y)[32], float (&z)[32], const uint4 (&res)[4]) {
  const int lane = at.lane, rows = at.rows, cols = at.cols, n = at.n, t0 = at.t0;
  uint8_t* mine = at.mine;
  if (p.bias) {
    const float b = lane < cols ? bf16_to_f32(p.bias[n + lane]) : 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) y[j] += __shfl_sync(0xFFFFFFFFu, b, j);
  }
  if (SIDES == 2) {
    if (p.gate_bias) {
      const float b = lane < cols ? bf16_to_f32(p.gate_bias[n + lane]) : 0.0f;
#pragma unroll
      for (int j = 0; j < 32; ++j) z[j] += __shfl_sync(0xFFFFFFFFu, b, j);
    }
    activate(z, p.activation);
#pragma unroll
    for (int j = 0; j < 32; ++j) y[j] *= z[j];
  } else {
    activate(y, p.activation);
  }
  if (p.residual) {
    __syncwarp();  // (what stood there has been read)
    if (at.whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(mine + piece_at<2>(i * 8 + (lane >> 2), lane & 3)) = res[i];
    } else if (lane < cols) {
      for (int r = 0; r < rows; ++r)
        *reinterpret_cast<uint16_t*>(mine + piece_at<2>(r, lane >> 3) + 2 * (lane & 7)) = p.residual[(t0 + r) * p.residual_stride + n + lane];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 w = *reinterpret_cast<const uint4*>(mine + piece_at<2>(lane, k));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 8 * k + 2 * i;
        y[j] += __uint_as_float(u[i] << 16);
        y[j + 1] += __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
  }
  __syncwarp();
  if (FULL) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float4*>(mine + piece_at<4>(lane, k)) = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    __syncwarp();
    float* out = static_cast<float*>(p.out) + t0 * p.out_stride + n;
    if (at.whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (r < rows) *reinterpret_cast<uint4*>(out + r * p.out_stride + 4 * (lane & 7)) = *reinterpret_cast<const uint4*>(mine + piece_at<4>(r, lane & 7));
      }
    } else if (lane < cols) {
      for (int r = 0; r < rows; ++r) out[r * p.out_stride + lane] = *reinterpret_cast<const float*>(mine + piece_at<4>(r, lane >> 2) + 4 * (lane & 3));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_p(y[8 * k + 2 * i], y[8 * k + 2 * i + 1]);
      *reinterpret_cast<uint4*>(mine + piece_at<2>(lane, k)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    uint16_t* out = static_cast<uint16_t*>(p.out) + t0 * p.out_stride + n;
    if (at.whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        if (r < rows) *reinterpret_cast<uint4*>(out + r * p.out_stride + 8 * (lane & 3)) = *reinterpret_cast<const uint4*>(mine + piece_at<2>(r, lane & 3));
      }
    } else if (lane < cols) {
      for (int r = 0; r < rows; ++r) out[r * p.out_stride + lane] = *reinterpret_cast<const uint16_t*>(mine + piece_at<2>(r, lane >> 3) + 2 * (lane & 7));
    }
  }
  __syncwarp();  // (the staging place has been read)
}

// FULL: outputs in 32 bits.
template <int SIDES, int PER, bool FULL>
__global__ void __launch_bounds__(kWideThreads, 1)
    k_wide(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_g,
           const __grid_constant__ CUtensorMap tm_x, const LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = smem + wide_ring(FULL);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpilogueWarps * wide_staging(FULL));
  uint64_t* empty = full + p.stages;
  uint64_t* tfull = empty + p.stages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drained = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cta_rank());
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1, tiles = p.m_tiles * p.n_tiles;
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpilogueWarps);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  dt_grid_wait();
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_barrier();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int segment = FULL ? kSegmentBlocks / PER : p.k_steps;  // steps that an accumulator adds
  bool ok = true;

  // (the epilogue's sums: 72 + 2 x 216 = 3 x 168, what the block was launched with)
  static_assert(kOtherRegs + 2 * kSumRegs <= 3 * 168, "");
  if (FULL && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 0) {
    const uint64_t keep = l2_policy_evict_last();
    uint32_t stage = 0, phase = 0;
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      const Place at = place(p, tile);
      const int t0 = at.m0 + rank * 128, n0 = SIDES == 2 ? at.n0 : at.n0 + rank * (p.bn / 2);
      const void* tm_b = SIDES == 2 && rank == 0 ? static_cast<const void*>(&tm_g) : static_cast<const void*>(&tm_w);
      for (int ks = 0; ks < p.k_steps; ++ks) {
        ok = pair_wait(&empty[stage], phase ^ 1u);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* to = smem + stage * p.stage_bytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * p.stage_bytes);  // (both CTAs')
          const uint32_t bar = peer_addr(&full[stage], 0);
          tma_load_pair<PER>(to, &tm_x, bar, ks, t0, keep);
          tma_load_pair<PER>(to + PER * kHalf, tm_b, bar, ks, n0, keep);
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
      }
    }
    // no copy may outlive the CTA, whichever wait gave up (the first CTA's barriers count both CTAs' copies)
    for (uint32_t s = 0; rank == 0 && s < static_cast<uint32_t>(p.stages); ++s) mbar_wait(&full[s], s < stage ? phase : phase ^ 1u, nullptr);
  } else if (warp == 1 && rank == 0) {
    const uint32_t idesc = idesc_bf16_f32(256, p.bn);
    uint32_t stage = 0, phase = 0;
    int local = 0;  // accumulators filled
    bool there = false;
    for (int tile = pair; tile < tiles && ok; tile += pairs)
      for (int ks0 = 0; ks0 < p.k_steps && ok; ks0 += segment, ++local) {
        const int acc = local & 1, ks1 = FULL ? min(p.k_steps, ks0 + segment) : p.k_steps;
        ok = pair_wait(&tempty[acc], (local >> 1 & 1) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * 256;
        for (int ks = ks0; ks < ks1; ++ks) {
          ok = there || pair_wait(&full[stage], phase);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = smem_u32(smem + stage * p.stage_bytes);
          const uint64_t a = sdesc_k_sw128(at), b = sdesc_k_sw128(at + PER * kHalf);
          uint64_t* used = &empty[stage];
          if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
          const bool next = mbar_test(&full[stage], phase);  // (asked before the products that stand in its way)
          if (elect_one()) {
            // (straight on: a loop of a length that is known late cost 5 % of large products, an eighth of ordinary ones)
#pragma unroll
            for (int k = 0; k < 4; ++k) tc_mma_pair(d, a + (k * 32 >> 4), b + (k * 32 >> 4), idesc, ks != ks0 || k != 0);
            if (PER == 2) {
              const uint64_t b1 = b + (p.bn * 64 >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k) tc_mma_pair(d, a + ((kHalf + k * 32) >> 4), b1 + (k * 32 >> 4), idesc, 1u);
            }
            tc_commit_pair(used);
            if (ks + 1 == ks1) tc_commit_pair(&tfull[acc]);
          }
          there = __all_sync(0xFFFFFFFFu, next);
        }
      }
    if (!ok) {  // (no product may outlive its operands and tensor memory)
      if (elect_one()) tc_commit_pair(drained);
      __syncwarp();
      pair_wait(drained, 0);
    }
  } else if (warp >= 4) {
    if (FULL) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int quarter = warp & 3, group = (warp - 4) >> 2;
    uint8_t* mine = staging + (warp - 4) * wide_staging(FULL);
    auto give_back = [&](int acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) peer_arrive(peer_addr(&tempty[acc], 0));
    };
    int local = 0;
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      const Place at = place(p, tile);
      const int t0 = at.m0 + rank * 128 + quarter * 32, rows = min(32, p.rows - t0);
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      auto chunk_at = [&](int c) {
        const int n = at.n0 + c, cols = min(32, p.outer - n);
        return Chunk{t0, n, rows, cols, lane, p.wide && cols == 32, mine};
      };
      uint4 res[4];
      if (FULL) {
        // sums of up to 4 / SIDES chunks of 32 columns, [chunk][side], over the accumulators of the tile
        float sum[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
        for (int ks0 = 0; ks0 < p.k_steps && ok; ks0 += segment, ++local) {
          const int acc = local & 1;
          ok = pair_wait(&tfull[acc], local >> 1 & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = group * 32 + 64 * (i / SIDES);
            if (c >= p.tile_outs) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t v[16];
              tmem_ld16(lanes + acc * 256 + (i % SIDES) * p.tile_outs + c + 16 * q, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[i][16 * q + j] += __uint_as_float(v[j]);
            }
          }
          give_back(acc);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; i += SIDES) {
          const int c = group * 32 + 64 * (i / SIDES);
          const Chunk chunk = chunk_at(c);
          if (c >= p.tile_outs || chunk.cols <= 0 || rows <= 0) break;
          ask_residual(p, chunk, res);
          finish_chunk<SIDES, FULL>(p, chunk, sum[i + SIDES - 1], sum[i], res);
        }
      } else {
        const int acc = local & 1;
        ok = pair_wait(&tfull[acc], local >> 1 & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = lanes + acc * 256;
        for (int c = group * 32; c < p.tile_outs; c += 64) {
          const Chunk chunk = chunk_at(c);
          if (chunk.cols <= 0 || rows <= 0) break;
          ask_residual(p, chunk, res);
          uint32_t raw[32 * SIDES];
          tmem_ld32(from + c, raw);
          if (SIDES == 2) tmem_ld32(from + p.tile_outs + c, raw + 32);
          tmem_wait_ld();
          tmem_landed32(raw);
          if (SIDES == 2) tmem_landed32(raw + 32);
          float y[32], z[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            y[j] = __uint_as_float(raw[32 * (SIDES - 1) + j]);
            z[j] = __uint_as_float(raw[j]);
          }
          finish_chunk<SIDES, FULL>(p, chunk, y, z, res);
        }
        give_back(acc);
        ++local;
      }
    }
  }
  if (!ok && p.status && lane == 0) atomicOr(p.status, DT_KV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // (no CTA leaves while the other may signal it, read its operands or write its tensor memory)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int SIDES, int PER, bool FULL>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_a_device(done, [] { return cudaFuncSetAttribute(k_wide<SIDES, PER, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem); });
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  return launch_behind(k_wide<SIDES, PER, FULL>, 2 * static_cast<unsigned>(tiles < kSms / 2 ? tiles : kSms / 2), kWideThreads, kWideSmem, st, 2, w, g, x, p);
}

template <int SIDES, int PER>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, cudaStream_t st) {
  return p.out_fp32 ? launch<SIDES, PER, true>(w, g, x, p, st) : launch<SIDES, PER, false>(w, g, x, p, st);
}

}  // namespace

cudaError_t launch_linear_wide(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, bool gate, cudaStream_t st) {
  if (p.per == 2) return gate ? launch<2, 2>(w, g, x, p, st) : launch<1, 2>(w, g, x, p, st);
  return gate ? launch<2, 1>(w, g, x, p, st) : launch<1, 1>(w, g, x, p, st);
}

}  // namespace dt
