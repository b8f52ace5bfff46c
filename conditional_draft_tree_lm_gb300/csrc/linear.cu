// dt_linear: matrix product with bias, activation or gate, and residual, on tcgen05.
//
// Few tokens.  Rows of weight are the product's rows (its A operand, up to 128 of them) and up to 256 tokens its columns,
// so that few tokens still fill the tensor core's lanes, and the kernels stream the weights once; with a gate, as many
// rows of each of the two matrices, whose sums meet in one epilogue.
//
// k_stream, where there are tiles for half of the SMs or more: persistent, one CTA an SM with all its shared memory for the
// stream, which runs on from tile to tile; two sets of accumulators, so that the epilogue of a tile stands beside the next
// one's products.
//
// k_few, where there are fewer: a cluster shares a tile.  Every CTA takes a part of the inner dimension, and the partial
// sums, fp32 in shared memory, are added over distributed shared memory in the order of ranks, each CTA finishing a
// part of the tile.  Tensor memory is given back before the cluster's barrier: a CTA that holds some waits for no other, so
// that kernels side by side on an SM cannot wait in a circle.
//
// Outputs in 32 bits: the tensor core cuts what it adds to an accumulator, and hundreds of additions of 16 channels lean to
// one side (2560 channels: 3e-6 of the result, six times what sums in fp32 are off by).  So an accumulator takes 512
// channels, and these parts are added in fp32, rounded: in shared memory by k_stream's epilogue, from accumulators
// beside each other by k_few.  Outputs in bf16 (half a step is 4e-3) have one accumulator over all channels.
//
// Bound by streaming the weights where they are many: 65 tokens' logits (2560 to 151936, fp32) 129 us, 6.2 TB/s; gated 32 tokens
// (2560 to 2 x 10240) 21 us, 5.1 TB/s, a quarter of it before the first products and behind the last.  By that latency where
// they are few: 65 tokens, 4096 to 2560 9.8 us, of which the copies take 2.  Tokens by the hundred: by the operands that every SM
// brings and by the sums of a split, which come over distributed shared memory at 18 bytes a clock (bulk copies are no faster): 200
// tokens, 2560 to 6144 14.6 us, 256, 4096 to 4096 16.3.
#include "linear.cuh"
#include "cluster.cuh"
#include "kv_flash.cuh"

namespace dt {
namespace {

constexpr int kFewThreads = 256, kMostSplit = 8;
constexpr int kFewSmem = 222 * 1024;  // of k_few at most
constexpr uint32_t kTileBytes = 128 * 128;  // 128 rows of 64 bf16

// A step of a stage: PER blocks of 64 of the inner dimension (one copy: the map has them as a third dimension, where they
// are whole), rows from `row` on, block after block.
template <int PER>
DT_DEVINL void load_step(void* to, const CUtensorMap& map, uint64_t* bar, int step, int row, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(
          smem_u32(to)),
      "l"(reinterpret_cast<uint64_t>(&map)), "r"(smem_u32(bar)), "r"(PER == 1 ? step * 64 : 0), "r"(row), "r"(PER == 1 ? 0 : step * PER), "l"(policy)
      : "memory");
}
// Its products (one block or two, straight on); tile: bytes of a block of one side's rows.
template <int SIDES, int PER>
DT_DEVINL void step_products(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, const LinearParams& p, uint32_t tile, bool more) {
  const uint64_t side = PER * tile >> 4;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int s = 0; s < SIDES; ++s) tc_mma_bf16(d + s * p.bn, a + s * side + (k * 32 >> 4), b + (k * 32 >> 4), idesc, more || k != 0);
  if (PER == 2) {
    const uint64_t a1 = a + (tile >> 4), b1 = b + (p.bn * 128 >> 4);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int s = 0; s < SIDES; ++s) tc_mma_bf16(d + s * p.bn, a1 + s * side + (k * 32 >> 4), b1 + (k * 32 >> 4), idesc, 1u);
  }
}

// Shared memory from the 1024-aligned base: the ring of stages (and behind the products the partial sums, in its place),
// then the barriers.
DT_HOST_DEVICE_INLINE uint32_t few_bars(const LinearParams& p, int sides) {
  const uint32_t ring = p.stages * p.stage_bytes, sums = p.bn * sides * 512u;
  return ring > sums ? ring : sums;
}

// A CTA's share of a tile: four neighbouring rows of weight for a token at a time, their sums over the cluster's CTAs.  A thread's
// units are 8 tokens apart, of the same rows; the reads of several are on their way together.  RANKS: the cluster's CTAs at most.
// gave_up: a wait of one of them gave up, so that sums are missing and nothing of the tile is written (looked at once the sums are here,
// since both come from the peers' memory).
template <int SIDES, int RANKS>
DT_DEVINL void finish_share(const LinearParams& p, const float* sums, const uint32_t* gave_up, int rank, int tokens, int t0, int n0) {
  constexpr int kFit = 16 / (RANKS * SIDES), kUnits = kFit > 4 ? 4 : kFit < 1 ? 1 : kFit, kStep = kFewThreads / 32;
  // (whole tokens)
  const int first = tokens * rank / p.split, end = tokens * (rank + 1) / p.split, f = (threadIdx.x & 31) * 4;
  const uint32_t lost = gave_up_beside(gave_up, RANKS == 1 ? 1 : p.split);
  for (int t = first + static_cast<int>(threadIdx.x >> 5); t < end; t += kUnits * kStep) {
    float4 v[kUnits][SIDES][RANKS];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int s = 0; s < SIDES; ++s) {
        const float* at = sums + (min(t + i * kStep, end - 1) * SIDES + s) * 128 + f;
        if (RANKS == 1) {
          v[i][s][0] = *reinterpret_cast<const float4*>(at);
          continue;
        }
#pragma unroll
        for (int r = 0; r < RANKS; ++r)
          if (r < p.split) v[i][s][r] = peer_ld4(peer_addr(at, r));
      }
    if (__any_sync(0xFFFFFFFFu, lost != 0)) return;
    float y[4 * kUnits], z[4 * kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int s = 0; s < SIDES; ++s) {
        float4& acc = v[i][s][0];
#pragma unroll
        for (int r = 1; r < RANKS; ++r)
          if (r < p.split) acc.x += v[i][s][r].x, acc.y += v[i][s][r].y, acc.z += v[i][s][r].z, acc.w += v[i][s][r].w;
        float* to = s == SIDES - 1 ? y : z;
        to[4 * i] = acc.x, to[4 * i + 1] = acc.y, to[4 * i + 2] = acc.z, to[4 * i + 3] = acc.w;
      }
    finish_rows<SIDES, kUnits>(p, t0 + t, kStep, (end - t + kStep - 1) / kStep, n0 + f, y, z);
  }
}

template <int SIDES, int PER>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_g,
          const __grid_constant__ CUtensorMap tm_x, const LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + few_bars(p, SIDES));
  uint64_t* empty = full + p.stages;
  uint64_t* done = empty + p.stages;
  uint64_t* drained = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  uint32_t* gave_up = tmem_slot + 1;  // (a wait of a warp)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.split, tile = static_cast<int>(blockIdx.x) / p.split;
  const int n0 = tile * 128, t0 = static_cast<int>(blockIdx.y) * p.bn;
  const int ks0 = static_cast<int>(static_cast<int64_t>(p.k_steps) * rank / p.split);
  const int ks1 = static_cast<int>(static_cast<int64_t>(p.k_steps) * (rank + 1) / p.split);
  const uint64_t stream = l2_policy_evict_first(), keep = l2_policy_evict_last();
  const uint32_t side_bytes = PER * kTileBytes;
  auto load = [&](int ks, uint32_t stage) {
    uint8_t* at = smem + stage * p.stage_bytes;
    mbar_arrive_expect_tx(&full[stage], p.stage_bytes);
    if (SIDES == 2) load_step<PER>(at, tm_g, &full[stage], ks, n0, stream);
    load_step<PER>(at + (SIDES - 1) * side_bytes, tm_w, &full[stage], ks, n0, stream);
    load_step<PER>(at + SIDES * side_bytes, tm_x, &full[stage], ks, t0, keep);
  };
  // the first loads are under way before tensor memory is asked for
  const int ahead = min(p.stages, ks1 - ks0);
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      mbar_init(done, 1);
      mbar_init(drained, 1);
      *gave_up = 0;
      fence_mbar_init();
      dt_grid_wait();
      for (int s = 0; s < ahead; ++s) load(ks0 + s, s);
    }
    __syncwarp();
  }
  dt_grid_wait();
  if (warp == 1) tmem_alloc(tmem_slot, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    for (int ks = ks0 + ahead; ks < ks1; ++ks) {
      ok = warp_wait(&empty[stage], phase);
      if (!ok) break;
      if (elect_one()) load(ks, stage);
      __syncwarp();
      if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
    }
    // no copy may outlive the CTA, whichever wait gave up
    for (uint32_t s = 0; s < static_cast<uint32_t>(ahead); ++s) mbar_wait(&full[s], s < stage ? phase ^ 1u : phase, nullptr);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(128, p.bn);
    uint32_t stage = 0, phase = 0;
    int segment = 0, in_segment = 0;
    bool there = false;
    for (int ks = ks0; ks < ks1; ++ks) {
      ok = there || warp_wait(&full[stage], phase);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem + stage * p.stage_bytes);
      const uint64_t a = sdesc_k_sw128(at), b = sdesc_k_sw128(at + SIDES * side_bytes);
      uint64_t* used = &empty[stage];
      if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
      const bool next = mbar_test(&full[stage], phase);  // (asked before the products that stand in its way)
      if (elect_one()) {
        step_products<SIDES, PER>(tmem + segment * (SIDES * p.bn), a, b, idesc, p, kTileBytes, in_segment != 0);
        tc_commit(used);
      }
      if (++in_segment == p.segment_steps) in_segment = 0, ++segment;
      there = __all_sync(0xFFFFFFFFu, next);
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
    // (32 columns of the sides' accumulators, which lie one behind the other, at a time; 16 behind the last are nobody's)
    const int quarter = warp & 3, columns = SIDES * p.bn;
    for (int c = (warp >> 2) * 32; c < columns; c += kFewThreads / 4) {
      const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c;
      uint32_t v[32];
      tmem_ld32(from, v);
      tmem_wait_ld();
      tmem_landed32(v);
      for (int i = p.segment_steps; i < ks1 - ks0; i += p.segment_steps) {
        uint32_t w[32];
        tmem_ld32(from + i / p.segment_steps * columns, w);
        tmem_wait_ld();
        tmem_landed32(w);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c16 = c + 16 * h, side = SIDES == 2 && c16 >= p.bn ? 1 : 0;
        float* to = sums + ((c16 - side * p.bn) * SIDES + side) * 128 + quarter * 32 + lane;
        if (c16 < columns)
#pragma unroll
          for (int j = 0; j < 16; ++j) to[j * SIDES * 128] = __uint_as_float(v[16 * h + j]);
      }
    }
  } else if (lane == 0) {
    *gave_up = 1;
    if (p.status) atomicOr(p.status, DT_KV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  __syncwarp();
  if (p.split > 1) cluster_barrier();
  if (p.split == 1) finish_share<SIDES, 1>(p, sums, gave_up, rank, tokens, t0, n0);
  else if (p.split == 2) finish_share<SIDES, 2>(p, sums, gave_up, rank, tokens, t0, n0);
  else if (p.split <= 4) finish_share<SIDES, 4>(p, sums, gave_up, rank, tokens, t0, n0);
  else finish_share<SIDES, kMostSplit>(p, sums, gave_up, rank, tokens, t0, n0);
  if (p.split > 1) cluster_barrier();  // (no CTA leaves while its sums are read)
}

constexpr int kStreamThreads = 384, kStreamWarps = 8;  // (epilogue warps)

// Shared memory: the ring of stages, the sums of sum_tokens tokens, the barriers.
DT_HOST_DEVICE_INLINE uint32_t stream_sums(const LinearParams& p) { return p.stages * p.stage_bytes; }
DT_HOST_DEVICE_INLINE uint32_t stream_bars(const LinearParams& p, int sides) { return stream_sums(p) + p.sum_tokens * sides * 512u; }

template <int SIDES, int PER>
__global__ void __launch_bounds__(kStreamThreads, 1)
    k_stream(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_g,
             const __grid_constant__ CUtensorMap tm_x, const LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* sums = reinterpret_cast<float*>(smem + stream_sums(p));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + stream_bars(p, SIDES));
  uint64_t* empty = full + p.stages;
  uint64_t* tfull = empty + p.stages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drained = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = p.n_tiles * p.m_tiles;  // (m_tiles: of tokens)
  const uint32_t tile_bytes = p.tile_outs * 128u, side_bytes = PER * tile_bytes, acc_cols = SIDES * p.bn;
  const uint64_t keep = l2_policy_evict_last(), stream = p.m_tiles == 1 ? l2_policy_evict_first() : keep;
  auto load = [&](int tile, int ks, uint32_t stage) {
    const int n0 = tile / p.m_tiles * p.tile_outs, t0 = tile % p.m_tiles * p.bn;
    uint8_t* at = smem + stage * p.stage_bytes;
    mbar_arrive_expect_tx(&full[stage], p.stage_bytes);
    if (SIDES == 2) load_step<PER>(at, tm_g, &full[stage], ks, n0, stream);
    load_step<PER>(at + (SIDES - 1) * side_bytes, tm_w, &full[stage], ks, n0, stream);
    load_step<PER>(at + SIDES * side_bytes, tm_x, &full[stage], ks, t0, keep);
  };
  // the first loads are under way before tensor memory is asked for
  const int ahead = min(p.stages, p.k_steps);
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(&tfull[a], 1);
        mbar_init(&tempty[a], kStreamWarps);
      }
      mbar_init(drained, 1);
      fence_mbar_init();
      dt_grid_wait();
      for (int s = 0; s < ahead; ++s) load(blockIdx.x, s, s);
    }
    __syncwarp();
  }
  dt_grid_wait();
  if (warp == 1) tmem_alloc(tmem_slot, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 0) {
    uint32_t stage = ahead == p.stages ? 0 : ahead, phase = ahead == p.stages;
    int begun = ahead;  // steps of the first tile
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, begun = 0)
      for (int ks = begun; ks < p.k_steps; ++ks) {
        ok = warp_wait(&empty[stage], phase ^ 1u);
        if (!ok) break;
        if (elect_one()) load(tile, ks, stage);
        __syncwarp();
        if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
      }
    // no copy may outlive the CTA, whichever wait gave up
    for (uint32_t s = 0; s < static_cast<uint32_t>(p.stages); ++s) mbar_wait(&full[s], s < stage ? phase : phase ^ 1u, nullptr);
  } else if (warp == 1) {
    // (rows of the product behind the tile's rows of weight come from whatever follows them, and go nowhere)
    const uint32_t idesc = idesc_bf16_f32(128, p.bn);
    uint32_t stage = 0, phase = 0;
    int local = 0;  // segments so far
    bool there = false;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x)
      for (int ks0 = 0; ks0 < p.k_steps && ok; ks0 += p.segment_steps, ++local) {
        const int acc = local & 1, ks1 = min(p.k_steps, ks0 + p.segment_steps);
        ok = warp_wait(&tempty[acc], (local >> 1 & 1) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * acc_cols;
        for (int ks = ks0; ks < ks1; ++ks) {
          ok = there || warp_wait(&full[stage], phase);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = smem_u32(smem + stage * p.stage_bytes);
          const uint64_t a = sdesc_k_sw128(at), b = sdesc_k_sw128(at + SIDES * side_bytes);
          uint64_t* used = &empty[stage];
          if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
          const bool next = mbar_test(&full[stage], phase);  // (asked before the products that stand in its way)
          if (elect_one()) {
            step_products<SIDES, PER>(d, a, b, idesc, p, tile_bytes, ks != ks0);
            tc_commit(used);
            if (ks + 1 == ks1) tc_commit(&tfull[acc]);
          }
          there = __all_sync(0xFFFFFFFFu, next);
        }
      }
    if (!ok) {  // (no product may outlive its operands and tensor memory)
      if (elect_one()) tc_commit(drained);
      __syncwarp();
      mbar_wait(drained, 0, nullptr);
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3, half = (warp - 4) >> 2, et = tid - 128;
    auto together = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    // the warps' common verdict: what a wait of one of them has missed is in the outputs of all
    auto all_together = [](bool mine) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"(static_cast<uint32_t>(mine))
          : "memory");
      return r != 0;
    };
    static_assert(kStreamWarps * 32 == 256, "");
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    // 16 tokens from column c of an accumulator on, to or onto the sums from token `at` on
    auto take = [&](uint32_t acc, int c, int at, bool onto) {
#pragma unroll
      for (int s = 0; s < SIDES; ++s) {
        uint32_t v[16];
        tmem_ld16(tmem + lanes + acc * acc_cols + s * p.bn + c, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float& sum = sums[((at + j) * SIDES + s) * 128 + quarter * 32 + lane];
          sum = onto ? sum + __uint_as_float(v[j]) : __uint_as_float(v[j]);
        }
      }
    };
    auto give_back = [&](uint32_t acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    };
    int local = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int n0 = tile / p.m_tiles * p.tile_outs, t0 = tile % p.m_tiles * p.bn, tokens = min(p.bn, p.rows - t0);
      auto write = [&](int c0, int count) {  // tokens c0 .. of the tile, whose sums are complete; a thread's are 8 apart
        const int f = (et & 31) * 4;
        if (f >= p.tile_outs || !ok) return;
        for (int t = et >> 5; t < count; t += 32) {
          float y[16], z[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4* at = reinterpret_cast<const float4*>(sums + min(t + 8 * i, count - 1) * SIDES * 128 + f);
            const float4 a = at[(SIDES - 1) * 32], b = at[0];
            y[4 * i] = a.x, y[4 * i + 1] = a.y, y[4 * i + 2] = a.z, y[4 * i + 3] = a.w;
            z[4 * i] = b.x, z[4 * i + 1] = b.y, z[4 * i + 2] = b.z, z[4 * i + 3] = b.w;
          }
          finish_rows<SIDES, 4>(p, t0 + c0 + t, 8, (count - t + 7) / 8, n0 + f, y, z);
        }
      };
      // (a wait that gave up in one warp: the others would wait for it at the barrier, so it goes on, and none of them writes)
      if (p.segment_steps < p.k_steps) {  // all tokens' sums, part by part
        for (int ks = 0; ks < p.k_steps; ks += p.segment_steps, ++local) {
          ok = ok && warp_wait(&tfull[local & 1], local >> 1 & 1);
          tc_fence_after();
          for (int c = 16 * half; c < p.bn && ok; c += 32) take(local & 1, c, c, ks > 0);
          give_back(local & 1);
        }
        ok = all_together(ok);
        write(0, tokens);
        together();
      } else {  // 32 tokens after 32
        const int acc = local & 1;
        ok = ok && warp_wait(&tfull[acc], local >> 1 & 1);
        tc_fence_after();
        for (int c0 = 0; c0 < tokens; c0 += 32) {
          if (c0 + 16 * half < p.bn && ok) take(acc, c0 + 16 * half, 16 * half, false);
          if (c0 + 32 >= tokens) give_back(acc);
          ok = all_together(ok);
          write(c0, min(32, tokens - c0));
          together();
        }
        ++local;
      }
    }
  }
  if (!ok && p.status && lane == 0) atomicOr(p.status, DT_KV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

template <int SIDES, int PER>
cudaError_t launch_stream(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_a_device(done, [] { return cudaFuncSetAttribute(k_stream<SIDES, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024); });
  if (e != cudaSuccess) return e;
  const uint32_t smem = 1024 + stream_bars(p, SIDES) + (2 * p.stages + 5) * 8 + 16;
  return launch_behind(k_stream<SIDES, PER>, min(p.n_tiles * p.m_tiles, kSms), kStreamThreads, smem, st, 1, w, g, x, p);
}
cudaError_t launch_stream(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, bool gate, cudaStream_t st) {
  if (p.per == 2) return gate ? launch_stream<2, 2>(w, g, x, p, st) : launch_stream<1, 2>(w, g, x, p, st);
  return gate ? launch_stream<2, 1>(w, g, x, p, st) : launch_stream<1, 1>(w, g, x, p, st);
}

template <int SIDES, int PER>
cudaError_t launch_few(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, cudaStream_t st) {
  const uint32_t smem = 1024 + few_bars(p, SIDES) + (2 * p.stages + 2) * 8 + 16;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_a_device(done, [] { return cudaFuncSetAttribute(k_few<SIDES, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024); });
  if (e != cudaSuccess) return e;
  return launch_behind(k_few<SIDES, PER>, dim3(static_cast<unsigned>(p.n_tiles * p.split), static_cast<unsigned>(p.m_tiles)), kFewThreads, smem, st, p.split,
                       w, g, x, p);
}
cudaError_t launch_few(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x, const LinearParams& p, bool gate, cudaStream_t st) {
  if (p.per == 2) return gate ? launch_few<2, 2>(w, g, x, p, st) : launch_few<1, 2>(w, g, x, p, st);
  return gate ? launch_few<2, 1>(w, g, x, p, st) : launch_few<1, 1>(w, g, x, p, st);
}

// Tokens in tiles, padded to 16: of 256 at most, 128 where their sums stay in shared memory.
void plan_tokens(LinearParams& p, int sides) {
  const int most = (p.out_fp32 ? 128 : 256) / sides;
  p.m_tiles = (p.rows + most - 1) / most;
  p.bn = ((p.rows + p.m_tiles - 1) / p.m_tiles + 15) & ~15;
  p.m_tiles = (p.rows + p.bn - 1) / p.bn;
}
// Steps of the inner dimension and their stages in `room` bytes: two blocks of 64 a step where blocks are whole and three
// such stages fit, since a step's copies, waits and products each have costs of their own.
void steps_of(LinearParams& p, int sides, uint32_t room) {
  const uint32_t block = (sides * p.tile_outs + p.bn) * 128u;
  p.per = p.inner % 128 == 0 && room / (2 * block) >= 3 ? 2 : 1;
  p.k_steps = (p.k_blocks + p.per - 1) / p.per;
  p.stage_bytes = p.per * block;
  p.stages = static_cast<int>(room / p.stage_bytes);
  if (p.stages > 12) p.stages = 12;
  p.segment_steps = p.out_fp32 ? kSegmentBlocks / p.per : p.k_steps;
}
int tmem_columns(int n) {
  int cols = 32;
  while (cols < n) cols *= 2;
  return cols;
}

// Persistent CTAs: rows of weight for tiles that divide evenly over them.
void plan_stream(LinearParams& p, int sides, int64_t tiles) {
  const int64_t rounds = (tiles + kSms - 1) / kSms;
  const int64_t per = (static_cast<int64_t>(p.outer) * p.m_tiles + rounds * kSms - 1) / (rounds * kSms);
  p.tile_outs = static_cast<int>((per + 7) / 8 * 8);
  if (p.tile_outs > 128) p.tile_outs = 128;
  auto n_tiles = [&] { return (p.outer + p.tile_outs - 1) / p.tile_outs; };
  while (p.tile_outs < 128 && static_cast<int64_t>(n_tiles()) * p.m_tiles > rounds * kSms) p.tile_outs += 8;
  p.n_tiles = n_tiles();
  p.tmem_cols = tmem_columns(2 * sides * p.bn);
  p.sum_tokens = p.out_fp32 ? (p.bn + 31) & ~31 : 32;
  steps_of(p, sides, 224u * 1024 - 1024 - p.sum_tokens * sides * 512);
}

// How many clusters of k_few stand beside each other, a CTA an SM: a property of the device (GPCs differ in their SMs), asked for
// once.  (Here 76 of 2, 46, 36, 28, 23, 15, 15 of 8.)
int clusters_beside(int size) {
  static std::atomic<int> known[64][kMostSplit + 1];  // 0: not asked for yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int>* at = dev < 64 ? &known[dev][size] : nullptr;
  int n = at ? at->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kFewSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(k_few<1, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k_few<1, 1>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (at) at->store(n, std::memory_order_relaxed);
  return n;
}

// Clusters of as many CTAs as leave all of them beside each other, with four blocks of 64 or more each.  A CTA has an SM with all its
// shared memory: two an SM, in clusters twice as large, were ahead up to 4 tokens only (2560 to 6144 9.2 us, one 9.5; 16 tokens the same;
// 65 tokens, 4096 to 2560 13.0, one 9.8).
// False where there are too few accumulators for outputs in 32 bits.
bool plan_few(LinearParams& p, int sides, int64_t tiles) {
  p.tile_outs = 128;
  p.n_tiles = (p.outer + 127) / 128;
  steps_of(p, sides, kFewSmem - 2048);
  p.split = 1;
  for (int n = 2; n <= kMostSplit && p.k_steps * p.per >= 4 * n; ++n)
    if (tiles <= clusters_beside(n)) p.split = n;
  const int steps = (p.k_steps + p.split - 1) / p.split, segments = (steps + p.segment_steps - 1) / p.segment_steps;
  const int columns = (segments - 1) * sides * p.bn + (sides * p.bn + 31) / 32 * 32;  // (they are read by 32)
  p.tmem_cols = tmem_columns(columns);
  return columns <= 512;
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
  // A CTA's part of a step: 128 tokens and half of the columns.  Two blocks of 64 channels a step while four such stages fit (up to 160
  // columns, for outputs in 32 bits 128): copies of 32 KB come in faster than of 16 (512 tokens, 4096 to 2560, 96 columns 17.1 us, by one block
  // 18.3; in 32 bits 19.6 and 21.8; 2080 tokens, 160 columns 32.4 and 33.1), three stages are too few (in 32 bits 43.8 us, by one block 41.3).
  const uint32_t block = 16384 + p.bn * 64;
  p.per = p.inner % 128 == 0 && wide_ring(p.out_fp32) / (2 * block) >= 4 ? 2 : 1;
  p.k_steps = (p.k_blocks + p.per - 1) / p.per;
  p.stage_bytes = p.per * block;
  p.stages = static_cast<int>(wide_ring(p.out_fp32) / p.stage_bytes);
}

}  // namespace

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
  if (!kv_aligned(2, a.residual, a.bias, a.gate_bias) || !kv_aligned(4, a.status))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: misaligned residual, bias or status", who);
  const MemoryRows to = {out, a.rows, a.out_row_stride * static_cast<int64_t>(bytes), a.outer * static_cast<int64_t>(bytes)};
  auto meets = [&](const void* d, int64_t rows, int64_t stride, int64_t width) {
    return d && rows_meet(to, {reinterpret_cast<uintptr_t>(d), rows, stride * 2, width * 2});
  };
  const bool in_place = a.residual == a.out && !a.out_fp32 && (a.rows == 1 || a.residual_row_stride == a.out_row_stride);
  if (meets(a.x, a.rows, a.x_row_stride, a.inner) || meets(a.weight, a.outer, a.weight_row_stride, a.inner) ||
      meets(a.gate, a.outer, a.gate_row_stride, a.inner) || (!in_place && meets(a.residual, a.rows, a.residual_row_stride, a.outer)) ||
      meets(a.bias, 1, 0, a.outer) || meets(a.gate_bias, 1, 0, a.outer) || meets(a.status, 1, 0, 2))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: out overlaps an input and is not the residual itself", who);
  LinearParams p = {};
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.gate_bias = static_cast<const uint16_t*>(a.gate_bias);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.residual_stride = a.residual_row_stride;
  p.out = a.out;
  p.out_stride = a.out_row_stride;
  p.rows = static_cast<int>(a.rows);
  p.outer = a.outer;
  p.inner = a.inner;
  p.k_blocks = (a.inner + 63) / 64;
  p.activation = a.activation;
  p.out_fp32 = a.out_fp32 != 0;
  p.status = a.status;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.rows <= kTokensMost) return kv_launched(who, launch_linear_token(a, p, st));
  const int sides = a.gate ? 2 : 1;
  // From here on pairs of CTAs, which split nothing.  us by clusters or persistent CTAs and by pairs: 4096 to 2560 13.8 and 14.4 at 224 tokens,
  // 15.3 and 14.5 at 256, 14.1 and 16.6 at 272, 18.0 and 16.9 at 512; 2560 to 6144 15.0 and 13.6, 16.3 and 13.8, 16.1 and 15.8, 22.8 and 16.4; to
  // 10240 20.0 and 17.2, 21.0 and 17.4, 26.5 and 23.8, 33.5 and 25.0; but 10240 to 2560 19.7 and 28.6, 21.9 and 28.7, 22.8 and 33.9, 30.0 and 34.4:
  // the sides meet below 160 tokens where rows of weight are many (160 gated to 2 x 10240 34.8 and 31.9) and above 512 where channels are.
  const bool many = p.rows > 256;
  const uintptr_t res = reinterpret_cast<uintptr_t>(a.residual);
  const int64_t at_once = many ? 16 / static_cast<int64_t>(bytes) : 4;  // outputs written together
  p.wide = out % (at_once * bytes) == 0 && (a.rows == 1 || a.out_row_stride % at_once == 0) &&
           (!res || (many ? res % 16 == 0 && a.residual_row_stride % 8 == 0 : res % 8 == 0 && (a.rows == 1 || a.residual_row_stride % 4 == 0)));
  bool stream_tiles = false;
  if (many) {
    plan_many(p, sides);
    if (static_cast<int64_t>(p.m_tiles) * p.n_tiles > (1 << 30)) return kv_fail(DT_ERR_SHAPE, "%s: more than 2^30 tiles", who);
  } else {
    plan_tokens(p, sides);
    const int64_t tiles = static_cast<int64_t>((a.outer + 127) / 128) * p.m_tiles;
    if (tiles > (1 << 29)) return kv_fail(DT_ERR_SHAPE, "%s: more than 2^29 tiles", who);
    // Clusters where tiles leave half of the SMs without one.  us by clusters and by persistent CTAs: 65 tokens, 2560 to 6144 10.8 and 12.1,
    // to 8192 12.1 and 12.6, to 9728 13.4 and 13.4; 200 tokens 14.6 and 17.7, 15.7 and 18.3, 18.0 and 18.9.
    stream_tiles = tiles >= kSms / 2 || !plan_few(p, sides, tiles);
    if (stream_tiles) plan_stream(p, sides, tiles);
  }
  const int w_rows = many ? p.bn / 2 : p.tile_outs;
  auto map = [&](CUtensorMap* m, const void* d, int64_t stride, int64_t rows, int box) {
    return linear_map(m, d, a.inner, rows, rows == 1 ? a.inner : stride, box, p.per);
  };
  CUtensorMap w, g, x;
  if (!map(&w, a.weight, a.weight_row_stride, a.outer, w_rows) ||
      !map(&g, a.gate ? a.gate : a.weight, a.gate ? a.gate_row_stride : a.weight_row_stride, a.outer, w_rows) ||
      !map(&x, a.x, a.x_row_stride, a.rows, many ? 128 : p.bn))
    return kv_fail(DT_ERR_SHAPE, "%s: strides that a tensor map does not take (2^40 bytes and more)", who);
  if (many) return kv_launched(who, launch_linear_wide(w, g, x, p, sides == 2, st));
  return kv_launched(who, stream_tiles ? launch_stream(w, g, x, p, sides == 2, st) : launch_few(w, g, x, p, sides == 2, st));
}
