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
// into a ring of four stages, one thread issues the products, two warpgroups do
// the softmax of a tile each.  The grid has a CTA for every item, but a running CTA
// takes over items whose CTA has not started (cluster launch control), so that one
// item's loads and first products run under the last one's softmax and output, and
// SMs end together: items differ by their position in the prompt (with a fixed list
// of items for each SM, the SMs of 48 ragged prompts ended 30 % apart).
//
// P is rounded to bf16 (operands of one product have one type, and V is bf16):
// 2^-8 relative a weight at most, as the rounding of the output itself.
//
// Tiles that hold keys which some row must not see are cleaned before their
// product (0 * NaN would reach that row): values behind the sequence become
// zeros, and a key whose value is not finite becomes zeros and is noted, which
// makes the output of the rows that do see it NaN (their lse has no values in it).
//
// Measured, 32 heads of 128 over 8: one prompt of 16k tokens 1335 us, 1.64 PFLOP/s, 87 %
// of the measured bf16 rate (the exponentials and the maximum are what the products
// wait for); 48 ragged prompts of up to 1k tokens 267 us, a third of the tensor
// cores' time and 38 % of the measured bandwidth: an item has four key tiles on
// average, so that its start (the first product) and its end (the last one, the output) weigh as much as
// they; one of 300 tokens 11.1 us, one item's chain (40 items, one a CTA).
#include <cuda.h>

#include <type_traits>

#include "kv_flash.cuh"

namespace dt {
namespace {

constexpr int kStages = 4;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp = 10, kCleanWarps = 2;
constexpr int kPromptThreads = 384;
// Registers: 384 threads start with 168; the softmax's 256 go to 208 and the others' 128 to 80 (63488 of 64512).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
// Tiles of which some row does not see all: keys behind the first of an item's (at most 256) positions
// lie in three at most, so each has barriers and a word of its own.
constexpr int kMaskedTiles = 3;

struct PromptParams {
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
  const int32_t* row_start;
  int64_t n_rows, out_row_stride, out_head_stride;
  int n_seq, n_q, n_kv, group, positions;  // positions: of a tile (128 / group)
  int slots;                               // items per key/value head
  uint32_t inverse;                        // group_inverse(group)
  float c;                                 // scale * log2(e)
};

DT_DEVINL void tma_load_3d(uint32_t dst, const void* tmap, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Two row tiles of a sequence, as every role sees them.
struct PromptItem {
  int kvh, row0, len, pos0;  // row0: the sequence's first row
  int n_tiles[2], n;         // key tiles of each row tile
  int masked0;               // the first key tile that holds a key behind pos0
};

constexpr int kItemSlots = 4;
struct __align__(16) PromptPlace {  // what a slot of the schedule holds
  int kvh, row0, len, pos0;  // len 0: nothing to do, < 0: no more items
};

// full, empty; q_full, q_free, s_full, o_full, told of two each, p_full of four; clean, dirty; item_full, item_free; answered and
// what brings the places to 16 bytes
constexpr int kPromptBarriers = 2 * kStages + 5 * 2 + 4 + 2 * kMaskedTiles + 2 * kItemSlots + 2;
template <int HD>
struct PromptSmem {
  static constexpr uint32_t kOperand = kOperandBytes<HD>;
  static constexpr uint32_t kQ = 0, kRing = 2 * kOperand, kOut = kRing + kStages * kOperand, kBars = kOut + 8 * 4096;
  static constexpr uint32_t kPlaces = kBars + kPromptBarriers * 8, kBytes = kPlaces + kItemSlots * sizeof(PromptPlace) + 16 + kMaskedTiles * 16 + 1024;  // + alignment
  static_assert(kPlaces % 16 == 0 && kBytes + kStaticBytes <= kSmemBytes, "");
};

// The place of item `at`, by a whole warp: sequence q's places stand from
// start_q / span + q on, at least as many as it needs, found without a sum.
DT_DEVINL PromptPlace prompt_place(const PromptParams& p, int at) {
  const int lane = threadIdx.x & 31;
  PromptPlace x = {at % p.n_kv, 0, 0, 0};
  // heaviest first: late positions
  const int slot = p.slots - 1 - at / p.n_kv, span = 2 * p.positions;
  const int first = __ldg(p.row_start);
  int lo = 0, n = p.n_seq;  // the last sequence whose first place is not behind `slot` is one of lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, q = lo + lane * step;
    const bool before = lane * step < n && (__ldg(p.row_start + q) - first) / span + q <= slot;
    const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, before) | 1u);
    n = min(step, n - k * step);
    lo += k * step;
  }
  const int a = __ldg(p.row_start + lo), b = __ldg(p.row_start + lo + 1);
  const int block = slot - ((a - first) / span + lo);
  if (a < 0 || b < a || b > p.n_rows || block < 0 || block > (b - a) / span || block * span >= b - a) return x;
  x.row0 = a;
  x.len = b - a;
  x.pos0 = block * span;
  return x;
}

DT_DEVINL void prompt_item(const PromptParams& p, const PromptPlace& x, PromptItem& it) {
  it.kvh = x.kvh;
  it.row0 = x.row0;
  it.len = x.len;
  it.pos0 = x.pos0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int from = x.pos0 + t * p.positions;
    it.n_tiles[t] = from < x.len ? (min(x.len, from + p.positions) + kKeyTile - 1) / kKeyTile : 0;
  }
  it.n = max(it.n_tiles[0], it.n_tiles[1]);
  it.masked0 = (x.pos0 + 1) / kKeyTile;
}

template <int HD, bool NEGATIVE>  // NEGATIVE: the softmax's scale is
__global__ void __launch_bounds__(kPromptThreads, 1)
    k_prompt(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const PromptParams p) {
  using Smem = PromptSmem<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem::kBars);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;      // [2]
  uint64_t* q_free = q_full + 2;           // [2] the item's products with this Q are done
  uint64_t* s_full = q_free + 2;           // [2]
  uint64_t* p_full = s_full + 2;           // [2][2] halves of P
  uint64_t* o_full = p_full + 4;           // [2]
  uint64_t* clean = o_full + 2;            // [kMaskedTiles] a masked tile's values are clean
  uint64_t* dirty = clean + kMaskedTiles;  // [kMaskedTiles] its values are there to be cleaned
  uint64_t* told = dirty + kMaskedTiles;   // [2] row tile t's softmax has read bad_key
  uint64_t* item_full = told + 2;                // [kItemSlots] the schedule
  uint64_t* item_free = item_full + kItemSlots;  // [kItemSlots]
  uint64_t* answered = item_free + kItemSlots;
  PromptPlace* places = reinterpret_cast<PromptPlace*>(full + kPromptBarriers);  // [kItemSlots], behind `answered`; 16-byte aligned, as the answer is
  uint8_t* answer = reinterpret_cast<uint8_t*>(places + kItemSlots);          // 16 bytes
  uint32_t* bad_key = reinterpret_cast<uint32_t*>(answer + 16);  // [kMaskedTiles][4] keys of the masked tiles whose values are not finite
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t drained;  // all products are done

  // (the same for a warp's lanes, and known to be)
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(&tmem_slot, 512);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_free[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
      mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < kMaskedTiles; ++i) {
      mbar_init(&clean[i], kCleanWarps);
      mbar_init(&dirty[i], 1);
    }
    for (int t = 0; t < 2; ++t) mbar_init(&told[t], 4);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_free[i], kPromptThreads / 32 - 1);  // every warp but the scheduling one
    }
    mbar_init(answered, 1);
    mbar_init(&drained, 1);
    for (int i = 0; i < 4 * kMaskedTiles; ++i) bad_key[i] = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t q_s = smem_u32(smem + Smem::kQ), ring = smem_u32(smem + Smem::kRing);
  PromptItem it;
  bool gave_up = false;  // a bounded wait did
  // the i-th item of this CTA into `it`; false: there is none (or a wait gave up)
  auto next_item = [&](int i) {
    bool got = warp_wait(&item_full[i % kItemSlots], (i / kItemSlots) & 1);
    gave_up |= !got;
    PromptPlace x = {0, 0, -1, 0};
    if (got) {
      const int4 y = *reinterpret_cast<const int4*>(&places[i % kItemSlots]);
      x = {y.x, y.y, y.z, y.w};
    }
    // (always so: a load from shared memory is certain to have been made when its value has been used, and the place is written again
    // after the arrival)
    const bool read = __all_sync(0xFFFFFFFFu, x.len >= -1);
    if (got && read && lane == 0) mbar_arrive(&item_free[i % kItemSlots]);
    prompt_item(p, x, it);
    return x.len >= 0;
  };

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      uint32_t stage = 0, phase = 0;
      int q_use[2] = {0, 0};
      bool ok = true;
      for (int i = 0; ok && next_item(i); ++i) {
        if (lane == 0) {
        auto load_q = [&](auto which) {
          constexpr int t = decltype(which)::value;
          if (it.n_tiles[t] == 0) return;
          ok = ok && mbar_wait(&q_free[t], (q_use[t]++ & 1) ^ 1, nullptr);
          if (!ok) return;
          mbar_arrive_expect_tx(&q_full[t], (HD / 64) * 128u * p.group * p.positions);
          for (int h = 0; h < HD / 64; ++h)
            tma_load_3d(q_s + t * Smem::kOperand + h * kHalfBytes, &tm_q, &q_full[t], h * 64, it.kvh * p.group,
                        it.row0 + it.pos0 + t * p.positions);
        };
        load_q(std::integral_constant<int, 0>{});
        // K(0), V(0), K(1), V(1), ...
        for (int x = 0; x < 2 * it.n && ok; ++x) {
          ok = mbar_wait(&empty[stage], phase ^ 1u, nullptr);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[stage], Smem::kOperand);
          for (int h = 0; h < HD / 64; ++h)
            tma_load_3d(ring + stage * Smem::kOperand + h * kHalfBytes, (x & 1) ? &tm_v : &tm_k, &full[stage], h * 64, it.kvh,
                        it.row0 + (x >> 1) * kKeyTile);
          if (++stage == kStages) stage = 0, phase ^= 1u;
          if (x == 0) load_q(std::integral_constant<int, 1>{});
        }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      }
      gave_up |= !ok;
      if (!ok && lane == 0) {  // (no copy may outlive the CTA)
        for (int s = 0; s < kStages; ++s) mbar_wait(&full[s], (s < static_cast<int>(stage) ? phase : phase ^ 1u), nullptr);
        for (int t = 0; t < 2; ++t)
          if (q_use[t] > 0) mbar_wait(&q_full[t], (q_use[t] - 1) & 1, nullptr);
      }
    } else if (warp == kMmaWarp) {
      const bool leader = elect_one();
      int load = 0;  // ring entries consumed
      int q_use[2] = {0, 0}, p_use[2] = {0, 0};
      uint32_t masked_turns = 0;  // bit m: the parity of clean[m]'s next phase
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && warp_wait(bar, parity);
        tc_fence_after();
      };
      auto full_wait = [&](int i) { wait(&full[i % kStages], (i / kStages) & 1); };
      auto at = [&](int i) { return ring + (i % kStages) * Smem::kOperand; };
      auto commit = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
      };
      const uint64_t q_desc[2] = {flash_desc(q_s, false), flash_desc(q_s + Smem::kOperand, false)};
      for (int i = 0; ok && next_item(i); ++i) {
        if (it.n == 0) continue;
        full_wait(load);
        uint64_t kd = flash_desc(at(load), false);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (it.n_tiles[t] == 0) continue;
          wait(&q_full[t], q_use[t]++ & 1);
          if (!ok) break;
          if (leader) issue_qk<HD>(true, tmem + t * 128, q_desc[t], kd);
          commit(&s_full[t]);
          if (it.n_tiles[t] == 1) commit(&q_free[t]);
        }
        if (ok) commit(&empty[load % kStages]);
        for (int j = 0; j < it.n && ok; ++j) {
          const int vi = load + 2 * j + 1, ki = vi + 1, m = j - it.masked0;
          const bool more = j + 1 < it.n;
          // (the cleaning warps cannot wait on the ring themselves: they would meet their stage in some earlier turn)
          full_wait(vi);
          if (ok && m >= 0 && leader) mbar_arrive(&dirty[m]);
          if (more) full_wait(ki);
          if (m >= 0) {
            wait(&clean[m], masked_turns >> m & 1u);
            masked_turns ^= 1u << m;
          }
          const uint64_t vd = flash_desc(at(vi), true);
          kd = flash_desc(at(ki), false);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || j >= it.n_tiles[t]) continue;
            const uint32_t turn = p_use[t]++ & 1;
            wait(&p_full[2 * t], turn);
            if (ok && leader) issue_pv<HD>(kProbs, tmem + 256 + t * 128, tmem + t * 128, vd, j == 0, 0);
            wait(&p_full[2 * t + 1], turn);
            if (!ok) continue;
            if (leader) issue_pv<HD>(kProbs, tmem + 256 + t * 128, tmem + t * 128, vd, j == 0, 1);
            if (j + 1 < it.n_tiles[t]) {
              if (leader) issue_qk<HD>(true, tmem + t * 128, q_desc[t], kd);
              commit(&s_full[t]);
              if (j + 2 == it.n_tiles[t]) commit(&q_free[t]);
            } else {
              commit(&o_full[t]);
            }
          }
          if (ok) {
            commit(&empty[vi % kStages]);
            if (more) commit(&empty[ki % kStages]);
          }
        }
        load += 2 * it.n;
      }
      gave_up |= !ok;
    } else if (warp >= kCleanWarp) {
      // values of the masked tiles: half of the keys a warp, a key's 16-byte pieces to eight lanes
      const int cw = warp - kCleanWarp;
      int load = 0, was_active[2] = {0, 0}, told_use[2] = {0, 0};  // was_active: row tiles of the last item
      uint32_t turns = 0;  // bit m: the parity of dirty[m]'s next phase
      bool ok = true;
      // (the last warp also keeps the schedule, an item ahead)
      const bool plans = cw == kCleanWarps - 1;
      PromptPlace here = {0, 0, -1, 0}, ahead = here;
      int asked = -1;
      auto publish = [&](int i, const PromptPlace& x) {
        ok = ok && warp_wait(&item_free[i % kItemSlots], ((i / kItemSlots) & 1) ^ 1);
        if (lane == 0) {
          places[i % kItemSlots] = x;
          mbar_arrive(&item_full[i % kItemSlots]);
        }
        __syncwarp();
      };
      if (plans) {
        here = prompt_place(p, static_cast<int>(blockIdx.x));
        publish(0, here);
      }
      for (int i = 0; ok; ++i) {
        if (plans) {
          if (lane == 0) {
            fence_proxy_async_smem();  // (the last answer has been read)
            take_next(answer, answered);
          }
          __syncwarp();
          ok = warp_wait(answered, i & 1);
          asked = i;
          const int id = ok ? taken(answer) : -1;
          __syncwarp();
          ahead.len = -1;
          if (id >= 0) ahead = prompt_place(p, id);
          publish(i + 1, ahead);
          prompt_item(p, here, it);
          here = ahead;
        } else if (!next_item(i)) {
          break;
        }
        if (it.n == 0) {
          if (plans && here.len < 0) break;
          continue;
        }
        // the words of the last item have been read (by the row tiles that it had: another's softmax may be items ahead)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (was_active[t]) ok = ok && mbar_wait(&told[t], told_use[t]++ & 1, nullptr);
          was_active[t] = it.n_tiles[t] > 0;
        }
        if (lane < 2 * kMaskedTiles) bad_key[(lane >> 1) * 4 + cw * 2 + (lane & 1)] = 0;
        __syncwarp();
        // (where a wait gives up the item goes on without waiting: lanes give up one by one, the warp's votes need them all)
        for (int j = it.masked0; j < it.n; ++j) {
          const int m = j - it.masked0;
          ok = ok && mbar_wait(&dirty[m], turns >> m & 1u, nullptr);
          turns ^= 1u << m;
          // (the swizzle stays within a key's 128 bytes)
          uint8_t* v = smem + Smem::kRing + ((load + 2 * j + 1) % kStages) * Smem::kOperand + cw * 64 * 128 + lane * 16;
          const int valid = it.len - j * kKeyTile - cw * 64 - (lane >> 3);  // of keys lane / 8, + 4, + 8, ...
          // an exponent of ones carries into its half's top bit
          uint32_t seen[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            seen[x] = 0;
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) {
              const uint4 w = *reinterpret_cast<const uint4*>(v + h * kHalfBytes + x * 512);
              seen[x] |= ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                         ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
            }
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const bool nan = (seen[x] & 0x80008000u) != 0, behind = 4 * x >= valid;
            if (nan || behind) {
#pragma unroll
              for (int h = 0; h < HD / 64; ++h) *reinterpret_cast<uint4*>(v + h * kHalfBytes + x * 512) = make_uint4(0, 0, 0, 0);
              const int key = cw * 64 + 4 * x + (lane >> 3);
              if (!behind) atomicOr(&bad_key[m * 4 + (key >> 5)], 1u << (key & 31));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&clean[m]);
        }
        load += 2 * it.n;
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (plans && here.len < 0) break;
      }
      if (!ok && asked >= 0) mbar_wait(answered, asked & 1, nullptr);  // (the answer is a write to this CTA, too)
      gave_up |= !ok;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // softmax: warpgroup t, a row a thread
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + 256 + t * 128 + lanes;
    float c = 0.0f;
    int s_use = 0, o_use = 0;
    bool ok = true;
    auto scale = [&](int) { return make_float2(c, c); };
    auto ready = [&](int half) {
      if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
    };
    for (int i = 0; ok && next_item(i); ++i) {
      if (it.n == 0) continue;
      const int n = t == 0 ? it.n_tiles[0] : it.n_tiles[1];
      const int from = it.pos0 + t * p.positions, pos = from + over_group(r, p.inverse);
      // (a row of the tile without a query gets its S from whatever stands in Q's place, the next sequence or an earlier item:
      // with a factor of 0 and a maximum of 0 it has no say in when the warp's rows are rescaled, whatever S is)
      const bool query = r < p.group * p.positions && pos < it.len;
      SoftmaxRow row;
      c = query ? p.c : 0.0f;
      row.m = query ? -INFINITY : 0.0f;
      for (int j = 0; j < n && ok; ++j) {
        ok = warp_wait(&s_full[t], s_use++ & 1);
        if (!ok) break;
        tc_fence_after();
        const int seen = pos + 1 - j * kKeyTile;  // of this tile's keys, by this row
        const uint32_t see[4] = {first_bits(seen, 0), first_bits(seen, 1), first_bits(seen, 2), first_bits(seen, 3)};
        if ((j + 1) * kKeyTile > from + 1)
          softmax_tile<HD, kProbs, true, NEGATIVE>(s_at, o_at, j == 0, scale, scale, scale, see, row, ready);
        else
          softmax_tile<HD, kProbs, false, NEGATIVE>(s_at, o_at, j == 0, scale, scale, scale, see, row, ready);
      }
      bool poison = false;
      if (n > 0) {
        ok = ok && warp_wait(&o_full[t], o_use++ & 1);
        tc_fence_after();
        // rows that see a key whose value is not finite (an item's cleaning is behind its o_full)
        for (int j = it.masked0; j < n; ++j)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (bad_key[(j - it.masked0) * 4 + w] & first_bits(pos + 1 - j * kKeyTile, w)) poison = true;
      }
      // (the vote uses the words, so that they have been read before they are cleared for the next item)
      poison = __ballot_sync(0xFFFFFFFFu, poison) >> lane & 1u;
      if (lane == 0 && n > 0) mbar_arrive(&told[t]);
      if (n > 0 && ok) {
        const bool live = r < p.group * p.positions && pos < it.len;
        const float inv = poison ? NAN : row.l == 0.0f ? 0.0f : 1.0f / row.l;
#pragma unroll
        for (int x = 0; x < HD; x += 64) {
          uint32_t v[64];
          tmem_ld32(o_at + x, v);
          tmem_ld32(o_at + x + 32, v + 32);
          tmem_wait_ld();
          tmem_landed32(v);
          tmem_landed32(v + 32);
          uint4 w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            w[k].x = pack_p(__uint_as_float(v[8 * k]) * inv, __uint_as_float(v[8 * k + 1]) * inv);
            w[k].y = pack_p(__uint_as_float(v[8 * k + 2]) * inv, __uint_as_float(v[8 * k + 3]) * inv);
            w[k].z = pack_p(__uint_as_float(v[8 * k + 4]) * inv, __uint_as_float(v[8 * k + 5]) * inv);
            w[k].w = pack_p(__uint_as_float(v[8 * k + 6]) * inv, __uint_as_float(v[8 * k + 7]) * inv);
          }
          store_rows(smem + Smem::kOut + warp * 4096, w, [&](int z) -> __nv_bfloat16* {
            const int y = (warp & 3) * 32 + z, ys = over_group(y, p.inverse), at = from + ys;
            return y < p.group * p.positions && at < it.len
                       ? p.out + static_cast<int64_t>(it.row0 + at) * p.out_row_stride +
                             (it.kvh * p.group + y - ys * p.group) * p.out_head_stride + x
                       : nullptr;
          });
        }
        tc_fence_before();  // (O has been read before the next item's first product writes it)
        if (live && p.lse)
          p.lse[static_cast<int64_t>(it.row0 + pos) * p.n_q + it.kvh * p.group + r - (pos - from) * p.group] = row.l == 0.0f ? -INFINITY : (row.m + log2f(row.l)) * kLn2;
      }
    }
    gave_up |= !ok;
  }
  if (gave_up && p.status) atomicOr(p.status, DT_KV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    // (where a wait gave up: no product may outlive its operands and tensor memory)
    if (elect_one()) tc_commit(&drained);
    mbar_wait(&drained, 0, nullptr);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool NEGATIVE>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PromptParams& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_prompt<HD, NEGATIVE>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptSmem<HD>::kBytes);
  if (e != cudaSuccess) return e;
  const int items = p.slots * p.n_kv;
  k_prompt<HD, NEGATIVE><<<items, kPromptThreads, PromptSmem<HD>::kBytes, st>>>(q, k, v, p);
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
  if (!kv_rows_apart(a.n_rows, a.n_q, a.head_dim, a.out_row_stride, a.out_head_stride))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: rows of out overlap", who);
  PromptParams p = {};
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  p.row_start = a.row_start;
  p.n_rows = a.n_rows;
  p.out_row_stride = a.out_row_stride;
  p.out_head_stride = a.out_head_stride;
  p.n_seq = a.n_seq;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.group = a.n_q / a.n_kv;
  p.positions = 128 / p.group;
  p.inverse = group_inverse(p.group);
  const int64_t slots = a.n_rows / (2 * p.positions) + a.n_seq;
  if (slots * a.n_kv > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: too many rows and heads for one launch", who);
  p.slots = static_cast<int>(slots);
  p.c = a.scale * kLog2e;
  CUtensorMap q, k, v;
  if (!kv_tmap_heads(&q, a.q, a.head_dim, a.n_q, a.n_rows, a.q_head_stride, a.q_row_stride, p.group, p.positions) ||
      !kv_tmap_heads(&k, a.k, a.head_dim, a.n_kv, a.n_rows, a.k_head_stride, a.k_row_stride, 1, kKeyTile) ||
      !kv_tmap_heads(&v, a.v, a.head_dim, a.n_kv, a.n_rows, a.v_head_stride, a.v_row_stride, 1, kKeyTile))
    return kv_fail(DT_ERR_SHAPE, "%s: strides that a tensor map does not take (zero, or 2^40 bytes and more)", who);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.c < 0.0f) return kv_launched(who, a.head_dim == 64 ? launch<64, true>(q, k, v, p, st) : launch<128, true>(q, k, v, p, st));
  return kv_launched(who, a.head_dim == 64 ? launch<64, false>(q, k, v, p, st) : launch<128, false>(q, k, v, p, st));
}
