// dt_cache_attention for many query rows per key/value head (slots * group > 16:
// drafted trees), on the tensor cores.
//
// Rows of a tile: 128 rows = (128 / group) slots x the group's heads.  A CTA takes
// two tiles at a time over a stretch of key tiles (cached tokens, then the new
// ones), see kv_flash.cuh for S, P and O.  An odd last row tile goes alone.
//
// What bounds it: at 65 slots and 4 heads a group a cached key is worth 260 * 512
// flops for 256 bytes, twice the tensor cores' balance, so tensor time, with the
// softmax and the conversion of the cache beside it; with one tile of rows it is
// about the cache's bytes.  A single row tile would leave the tensor core idle
// during its softmax, so it is taken twice, over the even and the odd key tiles of
// its stretch, and joined like two pieces.
//
// Cached keys and values come to shared memory as fp16 (e4m3 is exact in it): one
// warp looks up page numbers and scales and fetches whole pages a tile ahead (a
// page of a head is contiguous: one bulk copy), four converting warps turn them
// into the layout that the products read.  Scales stay in 32 bits: the key's multiplies the logit, the value's the weight,
// which the product takes in fp16 (11 bits of P where bf16 would keep 8) and a unit of the row's own (kv_flash.cuh).  Q comes to fp16 by a
// power of two per row (exact to 2^-40 of the row's maximum).  New tokens are bf16, whose range fp16 has not, and taken as they
// are: Q is laid out once more in bf16 before a stretch's first tile of them, under the last product with P, and P is the
// sum of two bf16.  So nothing shares a power of two with what only stands beside it (with one for all of a tile's new
// tokens, an unseen one of 1e30 wiped out the others).  With bf16 throughout and P as two bf16 in every tile the
// wide tree took 417 to 457 us, with that for new tiles only but Q and K in bf16 everywhere some 35 us more than now.
//
// Split.  The work is the list of (key/value head, request, row tiles, key tile),
// cut into equal pieces, one for each SM.  A tile of new keys counts kNewCost times,
// for itself and for what the end of a stretch costs.  A stretch that several pieces share is joined by the CTA that finishes
// last, in the order of keys.
//
// Measured: 32 trees of 65 slots (4 rows of each head streamed by the other kernel)
// over up to 4k cached tokens, 32 heads over 8, 209 us; one of 513 slots over 32k 310
// us (likewise; 335 with a row tile for the rows left over), 0.89 PFLOP/s.  Where the time goes: the products 2048 cycles of a pair of row
// tiles' 4 600 a key tile, the rest the softmax between them and shared memory (Q, K
// and V are read by both tiles' products, and written by the conversion); and what a
// stretch costs besides, its Q and its join, some 30 000 cycles, two or three times
// a CTA.  Reading the next stretch's Q and new tokens into L2 ahead changes nothing.
#pragma once

#include "kv_decode.cuh"
#include "kv_flash.cuh"

namespace dt {

constexpr int kTreeStages = 4;   // K and V tiles, alternating
constexpr int kTreeSlots = 4;    // what goes with a key tile: its scales and masks
constexpr int kTreeMmaWarp = 8, kTreeFetchWarp = 9, kTreeConvWarp = 12, kTreeConvWarps = 4;  // (10 and 11: none)
constexpr int kConvThreads = 32 * kTreeConvWarps;
constexpr int kTreeThreads = 32 * (kTreeConvWarp + kTreeConvWarps);
// Registers: 512 threads start with 128; the softmax's 256 go to 144, the others' to 112.  What a role spills would go
// to L2, there being no L1 left beside the shared memory (nothing now; us for 32 trees and for the wide one when something did: 136 and 120:
// 217 and 339; 144 and 112: 215 and 336; 152 and 104: 220 and 344; 160 and 96: 217 and 342).
constexpr int kTreeSoftmaxRegs = 144, kTreeOtherRegs = 112;
static_assert(2 * kTreeSoftmaxRegs + 2 * kTreeOtherRegs <= 4 * 128, "");

struct TreeParams {
  dt_kv_cache c;
  dt_cache_attention_args a;
  int group, shift;
  int per_tile;     // slots of a row tile
  uint32_t inverse; // group_inverse(group)
  int pairs, odd;   // pairs of row tiles, and whether one is left
  int fresh_tiles;  // key tiles of new tokens
  unsigned* done;   // [n_req * n_kv * (pairs + odd)] zero between launches
  float* part;      // [2 * pieces][2 tiles][HD / 4][128][4], then [2 * pieces][2][128][2]
};

// (2, 3, 4, 5, 6: 220, 213, 219, 209, 209 us for 32 trees, 328, 324, 324, 335, 340 for the wide one, 80, 74, 57, 55, 60 for
// 4 trees over 4k tokens)
constexpr int kNewCost = 5;

// What a row tile or a pair of them costs over a request's keys, at least 1.
DT_DEVINL int tree_cost(int len, int max_len, int fresh) {
  len = min(max(len, 0), max_len);
  return max(1, (len + kKeyTile - 1) / kKeyTile + fresh * kNewCost);
}
struct TreeUnits {
  int max_len, fresh, row_tiles;  // row_tiles: pairs and the odd one
  DT_DEVINL int operator()(int len) const { return row_tiles * tree_cost(len, max_len, fresh); }
};

// A stretch of key tiles of one (head, request, pair of row tiles or single one).
struct TreeSegment {
  int req, kvh, pair, tiles;  // tiles: row tiles, 2 or 1
  int first, units;           // in the work
  int key_begin, key_end;     // key tiles of this stretch
  int len, cached;            // tokens and key tiles in the cache
};

// Walks a piece's segments; every role of a CTA walks the same ones.
struct TreeWalk {
  int u, u_end, req, kvh, local, base;  // local: unit inside (req, kvh), whose first unit is base
  DT_DEVINL bool next(const TreeParams& p, TreeSegment& s) {
    if (u >= u_end) return false;
    const int max_len = p.a.max_blocks << p.shift;
    const int len = min(max(p.a.length[req], 0), max_len);
    const int cost = tree_cost(len, max_len, p.fresh_tiles);
    s.req = req;
    s.kvh = kvh;
    s.len = len;
    s.cached = (len + kKeyTile - 1) / kKeyTile;
    s.pair = local / cost;
    s.tiles = s.pair < p.pairs ? 2 : 1;
    s.first = base + s.pair * cost;
    s.units = cost;
    const int stop = min(u_end, s.first + cost);
    // a key tile belongs to the piece that its first unit is in; a stretch inside a new tile holds none
    auto tiles_before = [&](int x) {
      const int fresh = x - s.cached;
      return fresh <= 0 ? x : s.cached + (fresh + kNewCost - 1) / kNewCost;
    };
    s.key_begin = tiles_before(u - s.first);
    s.key_end = stop == s.first + cost ? max(1, s.cached + p.fresh_tiles) : tiles_before(stop - s.first);
    const int total = (p.pairs + p.odd) * cost;
    local += stop - u;
    u = stop;
    if (local == total) {
      local = 0;
      base += total;
      if (++req == p.a.n_req) req = 0, ++kvh;
    }
    return true;
  }
};

// Walks a piece's key tiles, segment after segment.
// Which of a stretch's key tiles is the first of new tokens (0 and less: all of them are).
DT_DEVINL int first_new_tile(const TreeParams& p, const TreeSegment& s) {
  return p.a.k_new ? s.cached - s.key_begin : 1 << 30;
}

enum { kTileNone = 0, kTileCached = 1, kTileNew = 2 };
struct TreeKeyTile {
  int kind;
  int key0, req, kvh, len;   // key0: its first cached token, or new token
};
struct TreeTileWalk {
  TreeWalk walk;
  TreeSegment sg;
  int key;
  DT_DEVINL void next(const TreeParams& p, TreeKeyTile& t) {
    t.kind = kTileNone;
    while (sg.tiles == 0 || key >= sg.key_end) {
      if (!walk.next(p, sg)) {
        sg.tiles = 0;
        return;
      }
      key = sg.key_begin;
    }
    // (a request without a key at all still has a tile: a cached one of no tokens)
    const bool fresh = p.a.k_new && key >= sg.cached;
    t.kind = fresh ? kTileNew : kTileCached;
    t.key0 = (fresh ? key - sg.cached : key) * kKeyTile;
    t.req = sg.req;
    t.kvh = sg.kvh;
    t.len = sg.len;
    ++key;
  }
};

// `bytes` (a multiple of 16) of contiguous global memory to shared memory.
DT_DEVINL void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// What goes with a key tile.
struct alignas(8) TreeTile {
  float k_scale[8], v_scale[8], v_log[8];  // of 16 keys each, and the value scale's logarithm
  uint32_t seen[4];   // cached keys that exist (new ones: the keys below slots)
  uint32_t bad[4];    // keys whose values are not finite (new ones only)
  int plain;          // all keys exist
};

// full, empty; q_full, s_full, o_full, st_full, st_free of two each, p_full of four
constexpr int kTreeBarriers = 2 * kTreeStages + 5 * 2 + 4;

template <int HD>
struct TreeSmem {
  static constexpr uint32_t kOperand = kOperandBytes<HD>;
  static constexpr uint32_t kQ = 0, kRing = 2 * kOperand, kStaging = kRing + kTreeStages * kOperand;
  static constexpr uint32_t kStagingBytes = 2 * kKeyTile * HD;  // K, V: [key][channel] in 8 bits
  static constexpr uint32_t kBars = kStaging + kStagingBytes, kTiles = kBars + kTreeBarriers * 8;
  static constexpr uint32_t kBytes = kTiles + kTreeSlots * sizeof(TreeTile) + 1024;  // + alignment
  static_assert(kTiles % alignof(TreeTile) == 0 && kBytes + kStaticBytes <= kSmemBytes, "");
};

// 16 bytes of global memory to shared memory, without a register; zeros where not `there`.
DT_DEVINL void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
DT_DEVINL void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

DT_DEVINL int by_group(const TreeParams& p, int y) { return over_group(y, p.inverse); }

template <int HD>
__global__ void __launch_bounds__(kTreeThreads, 1) k_tree(const TreeParams p) {
  using Smem = TreeSmem<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem::kBars);
  uint64_t* empty = full + kTreeStages;
  uint64_t* q_full = empty + kTreeStages;  // [2]
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;           // [2][2] halves of P
  uint64_t* o_full = p_full + 4;
  uint64_t* st_full = o_full + 2;   // [2] K, V in the staging place
  uint64_t* st_free = st_full + 2;  // [2]
  TreeTile* tiles = reinterpret_cast<TreeTile*>(full + kTreeBarriers);  // [kTreeSlots], behind st_free
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t drained;  // all products are done
  __shared__ int scratch[4], s_start[128 + 1], s_last;

  // (the same for a warp's lanes, and known to be)
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const dt_cache_attention_args& a = p.a;
  const int n_kv = p.c.n_kv;

  if (warp == kTreeMmaWarp) tmem_alloc(&tmem_slot, 512);
  if (tid == 0) {
    for (int s = 0; s < kTreeStages; ++s) {
      mbar_init(&full[s], kTreeConvWarps);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 4);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&st_full[t], 1);
      mbar_init(&st_free[t], kTreeConvWarps);
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  // (the rows left over, if any, may start on the SMs that this kernel leaves first)
  dt_grid_release();
  const TreeUnits units = {a.max_blocks << p.shift, p.fresh_tiles, p.pairs + p.odd};
  TileRow<128, TreeUnits> row_of = {a.length, a.n_req, units, 0, s_start};
  row_of.sum(scratch);  // (ends with a barrier)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int work = row_of.total() * n_kv, pieces = min(work, static_cast<int>(gridDim.x)), piece = blockIdx.x;
  if (piece < pieces) {
    const Cut cut(work, pieces);
    TreeWalk start;
    start.u = cut.begin(piece);
    start.u_end = cut.begin(piece + 1);
    start.kvh = start.u / row_of.total();
    {
      int first;
      const int index = start.u - start.kvh * row_of.total();
      row_of.find(index, start.req, first);
      start.local = index - first;
      start.base = start.u - start.local;
    }
    TreeWalk walk = start;
    TreeSegment sg = {};
    const uint32_t q_s = smem_u32(smem + Smem::kQ), ring = smem_u32(smem + Smem::kRing);

    bool gave_up = false;  // a bounded wait did
    if (warp >= kTreeMmaWarp) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTreeOtherRegs));
      if (warp == kTreeMmaWarp) {
        const bool leader = elect_one();
        int count = 0;  // key tiles so far
        int p_use[2] = {0, 0}, q_use[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          ok = ok && warp_wait(bar, parity);
          tc_fence_after();
        };
        auto full_wait = [&](int i) { wait(&full[i % kTreeStages], (i / kTreeStages) & 1); };
        auto at = [&](int i) { return ring + (i % kTreeStages) * Smem::kOperand; };
        auto commit = [&](uint64_t* bar) {
          if (leader) tc_commit(bar);
        };
        const uint64_t q_desc[2] = {flash_desc(q_s, false), flash_desc(q_s + Smem::kOperand, false)};
        auto pv = [&](int t, int i, bool fresh, bool first, bool last) {  // ring entry i into O of slot t
          const uint32_t turn = p_use[t]++ & 1;
          const uint64_t vd = flash_desc(at(i), true);
          wait(&p_full[2 * t], turn);
          if (ok && leader) issue_pv<HD>(fresh ? kWeightPairs : kWeights, tmem + 256 + t * 128, tmem + t * 128, vd, first, 0);
          wait(&p_full[2 * t + 1], turn);
          if (ok && leader) issue_pv<HD>(fresh ? kWeightPairs : kWeights, tmem + 256 + t * 128, tmem + t * 128, vd, first, 1);
          if (ok && last) commit(&o_full[t]);
        };
        auto qk = [&](int t, int i, bool fresh, bool new_q) {  // new_q: Q of slot t is laid out (again) for this tile
          if (new_q) wait(&q_full[t], q_use[t]++ & 1);
          if (!ok) return;
          if (leader) issue_qk<HD>(fresh, tmem + t * 128, q_desc[t], flash_desc(at(i), false));
          commit(&s_full[t]);
        };
        auto release = [&](int i) {
          if (ok) commit(&empty[i % kTreeStages]);
        };
        while (ok && walk.next(p, sg)) {
          const int n = sg.key_end - sg.key_begin;
          if (n == 0) continue;
          const int first_new = first_new_tile(p, sg);
          full_wait(2 * count);
          qk(0, 2 * count, first_new <= 0, true);
          if (sg.tiles == 2) {
            qk(1, 2 * count, first_new <= 0, true);
            release(2 * count);
            for (int j = 0; j < n && ok; ++j, ++count) {
              const int vi = 2 * count + 1, ki = vi + 1;
              const bool more = j + 1 < n;
              full_wait(vi);
              if (more) full_wait(ki);
  #pragma unroll
              for (int t = 0; t < 2; ++t) {
                pv(t, vi, j >= first_new, j == 0, !more);
                if (more) qk(t, ki, j + 1 >= first_new, j + 1 == first_new);
              }
              release(vi);
              if (more) release(ki);
            }
          } else {
            release(2 * count);
  #pragma unroll 1
            for (int j0 = 0; j0 < n && ok; j0 += 2) {
  #pragma unroll
              for (int t = 0; t < 2; ++t) {
                const int j = j0 + t;
                if (j >= n) break;
                const int vi = 2 * (count + j) + 1, ki = vi + 1;
                if (j + 1 < n) {
                  full_wait(ki);
                  qk(t ^ 1, ki, j + 1 >= first_new, j == 0 || (j + 1 >= first_new && j - 1 < first_new));
                  release(ki);
                }
                full_wait(vi);
                pv(t, vi, j >= first_new, j0 == 0, j + 2 >= n);
                release(vi);
              }
            }
            count += n;
          }
        }
        gave_up = !ok;
      } else if (warp == kTreeFetchWarp) {
        // --- pages to the staging place, a tile ahead of their conversion; page numbers and scales another tile ahead
        struct Page {  // of 16 keys, held by lanes 0..7
          int id;
          float ks, vs;
        };
        TreeKeyTile cur, nxt;
        TreeTileWalk tw = {walk, {}, 0};
        auto pages_of = [&](const TreeKeyTile& t) {
          Page g = {-1, 1.0f, 0.0f};
          const int tok = t.key0 + lane * 16;
          if (t.kind == kTileCached && lane < 8 && tok < t.len) {
            g.id = __ldg(a.block_table + static_cast<size_t>(t.req) * a.max_blocks + (tok >> p.shift));
            if (g.id < 0 || g.id >= p.c.n_pages) {
              if (a.status) atomicOr(a.status, DT_KV_BAD_INDEX);
              g.id = -1;
            } else {
              const size_t at = static_cast<size_t>(g.id) * n_kv + t.kvh;
              g.ks = __ldg(p.c.k_scale + at);
              g.vs = __ldg(p.c.v_scale + at);
            }
          }
          return g;
        };
        const int copy_keys = min(1 << p.shift, kKeyTile);
        tw.next(p, cur);
        Page gc = pages_of(cur);
        bool ok = true;
        int fetched[2] = {0, 0};
        for (int count = 0; cur.kind != kTileNone && ok; ++count) {
          tw.next(p, nxt);
          const Page gn = pages_of(nxt);
          TreeTile& info = tiles[count % kTreeSlots];
          const bool copies = cur.kind == kTileCached && lane < 8 && gc.id >= 0 && (lane * 16 & (copy_keys - 1)) == 0;
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, copies)) * copy_keys * HD;
          const uint32_t there = __ballot_sync(0xFFFFFFFFu, gc.id >= 0);
          const size_t at = copies ? (static_cast<size_t>(gc.id) * n_kv + cur.kvh << p.shift) * HD : 0;
  #pragma unroll
          for (int which = 0; which < 2; ++which) {
            ok = ok && warp_wait(&st_free[which], (count & 1) ^ 1);
            if (!ok) break;
            // (the place is free: the tile four before this one is behind its softmax, too)
            if (which == 0) {
              const bool plain = __all_sync(0xFFFFFFFFu, lane >= 8 || gc.id >= 0) && cur.len - cur.key0 >= kKeyTile;
              if (lane < 8) info.k_scale[lane] = gc.ks, info.v_scale[lane] = gc.vs, info.v_log[lane] = lg2(gc.vs);
              if (lane == 0) info.plain = plain;
              if (lane < 4) {
                const uint32_t two = there >> (2 * lane);
                info.seen[lane] = cur.kind == kTileNew ? first_bits(a.slots - cur.key0, lane)
                                                       : first_bits(cur.len - cur.key0, lane) & (((two & 1) ? 0xFFFFu : 0u) | ((two & 2) ? 0xFFFF0000u : 0u));
                info.bad[lane] = 0;
              }
              __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(&st_full[which], bytes);
            ++fetched[which];
            __syncwarp();
            if (copies)
              bulk_load(smem_u32(smem + Smem::kStaging) + which * kKeyTile * HD + lane * 16 * HD,
                        static_cast<const uint8_t*>(which ? p.c.v : p.c.k) + at, copy_keys * HD, &st_full[which]);
          }
          cur = nxt;
          gc = gn;
        }
        // (where a wait gave up: no copy may outlive the CTA)
        if (!ok)
          for (int which = 0; which < 2; ++which)
            if (fetched[which] > 0) mbar_wait(&st_full[which], (fetched[which] - 1) & 1, nullptr);
        gave_up = !ok;
      } else if (warp >= kTreeConvWarp) {
        // --- conversion
        constexpr int kLanes = HD / 16;               // threads of a key's row (16 bytes each)
        constexpr int kPassRows = kConvThreads / kLanes;
        constexpr int kPasses = kKeyTile / kPassRows;  // pieces of a thread
        const int ct = tid - kTreeConvWarp * 32, cc = ct % kLanes, cr = ct / kLanes;
        auto arrive = [&](int i) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[i % kTreeStages]);
        };
        // (where a wait gives up the loop goes on without waiting: other warps may stand at its named barrier)
        bool ok = true;
        auto room = [&](int i) { ok = ok && mbar_wait(&empty[i % kTreeStages], ((i / kTreeStages) & 1) ^ 1, nullptr); };
        // a cached tile's K or V out of the staging place.  The two halves of a row's threads begin with different
        // halves of their 16 bytes, so that their stores meet different banks.
        const bool swap = HD == 128 && (cc & 4);
        const int chunk0 = 2 * cc + (swap ? 1 : 0);
        const int place = (chunk0 >> 3) * kHalfBytes + cr * 128, piece0 = ((chunk0 & 7) ^ (cr & 7)) << 4;
        const uint8_t* st0 = smem + Smem::kStaging + ct * 16 + (swap ? 8 : 0);
        const int st1 = swap ? -8 : 8;
        // (passes are multiples of 8 rows apart: the swizzle is the same)
        auto convert = [&](const TreeTile& info, int count, int which) {
          const bool plain = info.plain;
          const uint8_t* st = st0 + which * kKeyTile * HD;
          uint8_t* op = smem + Smem::kRing + ((2 * count + which) % kTreeStages) * Smem::kOperand + place;
          constexpr int kBatch = 4;
  #pragma unroll 1
          for (int k0 = 0; k0 < kPasses; k0 += kBatch) {
            uint2 w[kBatch][2];
  #pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const uint8_t* x = st + (k0 + k) * kConvThreads * 16;
              w[k][0] = *reinterpret_cast<const uint2*>(x);
              w[k][1] = *reinterpret_cast<const uint2*>(x + st1);
            }
            if (k0 == 0) room(2 * count + which);
            uint32_t h[kBatch][8];
  #pragma unroll
            for (int k = 0; k < kBatch; ++k)
  #pragma unroll
              for (int y = 0; y < 2; ++y) {
                e4m3x4_to_f16x2x2(w[k][y].x, h[k][4 * y], h[k][4 * y + 1]);
                e4m3x4_to_f16x2x2(w[k][y].y, h[k][4 * y + 2], h[k][4 * y + 3]);
              }
            if (!plain) {
  #pragma unroll
              for (int k = 0; k < kBatch; ++k) {
                const int row = (k0 + k) * kPassRows + cr;
                const bool seen = info.seen[row >> 5] >> (row & 31) & 1u;  // (what no row sees may be NaN, or not there)
  #pragma unroll
                for (int x = 0; x < 8; ++x) h[k][x] = seen ? h[k][x] : 0u;
              }
            }
  #pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              uint8_t* to = op + (k0 + k) * kPassRows * 128;
              *reinterpret_cast<uint4*>(to + piece0) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
              *reinterpret_cast<uint4*>(to + (piece0 ^ 16)) = make_uint4(h[k][4], h[k][5], h[k][6], h[k][7]);
            }
          }
          arrive(2 * count + which);
          // The staging place goes back here, and no earlier: a load from shared memory is certain to have been made when
          // its value has been used.  (Handed back between the loads and the wait for room, it was overwritten by the
          // next page's copy now and then before they had read it.)
          if (lane == 0) mbar_arrive(&st_free[which]);
        };
        // A new tile, bf16 as it comes, all of it in flight at once.  Values that are not finite become zeros and
        // their keys are noted, for the rows that see them: before K is handed over, since S tells the softmax that
        // the notes are there.
        constexpr int kL = HD / 8, kR = kConvThreads / kL, kP = kKeyTile / kR;  // threads of a row, rows at a time, pieces of a thread
        const int c8 = ct % kL, r8 = ct / kL;
        auto convert_new = [&](const TreeKeyTile& t, TreeTile& info, int count) {
          // (rows are multiples of 8 apart: the swizzle is the same)
          const uint32_t place_new = (c8 >> 3) * kHalfBytes + r8 * 128 + (((c8 & 7) ^ (r8 & 7)) << 4);
          uint8_t* op[2];
  #pragma unroll
          for (int which = 0; which < 2; ++which) {
            const int64_t row_stride = which ? a.v_row_stride : a.k_row_stride;
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(which ? a.v_new : a.k_new) + t.kvh * (which ? a.v_head_stride : a.k_head_stride) + c8 * 8;
            op[which] = smem + Smem::kRing + ((2 * count + which) % kTreeStages) * Smem::kOperand + place_new;
            room(2 * count + which);
  #pragma unroll 4
            for (int k = 0; k < kP; ++k) {
              const int b = t.key0 + k * kR + r8;
              copy16(smem_u32(op[which] + k * kR * 128), x + (static_cast<int64_t>(t.req) * a.slots + min(b, a.slots - 1)) * row_stride, b < a.slots);
            }
          }
          copies_landed();
  #pragma unroll 4
          for (int k = 0; k < kP; ++k) {
            uint4* at = reinterpret_cast<uint4*>(op[1] + k * kR * 128);
            const uint4 w = *at;
            // (an exponent of ones carries into its half's top bit)
            const uint32_t odd = ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                                 ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
            if (odd & 0x80008000u) {
              *at = make_uint4(0, 0, 0, 0);
              atomicOr(&info.bad[(k * kR + r8) >> 5], 1u << ((k * kR + r8) & 31));
            }
          }
          arrive(2 * count);
          arrive(2 * count + 1);
        };
        TreeKeyTile cur;
        TreeTileWalk tw = {walk, {}, 0};
        for (int count = 0; tw.next(p, cur), cur.kind != kTileNone; ++count) {
          TreeTile& info = tiles[count % kTreeSlots];
          ok = ok && mbar_wait(&st_full[0], count & 1, nullptr);
          if (cur.kind == kTileCached) {
  #pragma unroll 1
            for (int which = 0; which < 2; ++which) {
              if (which) ok = ok && mbar_wait(&st_full[1], count & 1, nullptr);
              convert(info, count, which);
            }
          } else {
            ok = ok && mbar_wait(&st_full[1], count & 1, nullptr);
            __syncwarp();
            if (lane == 0) mbar_arrive(&st_free[0]), mbar_arrive(&st_free[1]);
            convert_new(cur, info, count);
          }
        }
        gave_up = !ok;
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTreeSoftmaxRegs));
      // --- softmax: warpgroup t, a row a thread
      const int t = warp >> 2, r = tid & 127;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + 256 + t * 128 + lanes;
      float* stats = p.part + static_cast<size_t>(2 * pieces) * 2 * 128 * HD;
      int count = 0, s_use = 0, o_use = 0;
      bool ok = true;
      auto ready = [&](int half) {
        if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
      };
      while (walk.next(p, sg)) {
        const int n = sg.key_end - sg.key_begin;
        // a single row tile is both slots': t takes every other key tile
        const bool split = sg.tiles == 1;
        const int steps = split ? (n + 1 - t) / 2 : n, tile = sg.pair * 2 + (split ? 0 : t);
        const int slot = tile * p.per_tile + by_group(p, r), head = sg.kvh * p.group + r - by_group(p, r) * p.group;
        const bool live = r < p.per_tile * p.group && slot < a.slots;
        const int64_t row = static_cast<int64_t>(sg.req) * a.slots + slot;
        SoftmaxRow sm;
        bool poison = false;  // the row sees a new token's value that is not finite: O is NaN, the sum is not
        const int first_new = first_new_tile(p, sg);
        float c = 0.0f;  // what makes a power of two of a raw logit, but for the key's scale
        // Q, HD / 8 lanes a row: to fp16 by a power of two of the row's own, or as it comes; with the scale's sign
        auto load_q = [&](bool bf16) {
          constexpr int kL = HD / 8, kR = 32 / kL, kN = 32 / kR;  // lanes of a row, rows at a time, times
          uint8_t* op = smem + Smem::kQ + t * Smem::kOperand;
          const int cx = lane % kL, rx = lane / kL;
          const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
          const float unit = fabsf(a.scale) * kLog2e;
          c = unit;
#pragma unroll 8
          for (int i = 0; i < kN; ++i) {
            const int y = (warp & 3) * 32 + i * kR + rx, ys = by_group(p, y), sl = tile * p.per_tile + ys;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (y < p.per_tile * p.group && sl < a.slots)
              w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                       (static_cast<int64_t>(sg.req) * a.slots + sl) * a.q_row_stride +
                                                       (sg.kvh * p.group + y - ys * p.group) * a.q_head_stride) + cx);
            uint32_t h[4] = {w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip};
            if (!bf16) {
              float amax = 0.0f;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(h[z] << 16)), fabsf(__uint_as_float(h[z] & 0xFFFF0000u))));
#pragma unroll
              for (int o = 1; o < kL; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
              int k = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
              k = min(max(k, -100), 127);
              const float up = __uint_as_float(static_cast<uint32_t>(14 - k + 127) << 23);
#pragma unroll
              for (int z = 0; z < 4; ++z)
                h[z] = pack_f16(__uint_as_float(h[z] << 16) * up, __uint_as_float(h[z] & 0xFFFF0000u) * up);
              const int mine = __shfl_sync(0xFFFFFFFFu, k, (lane % kR) * kL);
              if (lane / kR == i) c = unit * __uint_as_float(static_cast<uint32_t>(mine - 14 + 127) << 23);
            }
            *reinterpret_cast<uint4*>(op + (cx >> 3) * kHalfBytes + y * 128 + (((cx & 7) ^ (y & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[t]);
        };
        {
          for (int i = 0; i < steps; ++i) {
            const int j = split ? 2 * i + t : i, key = sg.key_begin + j;
            const bool fresh = j >= first_new;
            // (this row tile's last product with Q, that of its last step, is done: S has been read)
            if (i == 0 || (fresh && j - (split ? 2 : 1) < first_new)) load_q(fresh);
            uint32_t see[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
            if (fresh) {  // which of the new tokens this row sees, while the product runs
              const int b0 = (key - sg.cached) * kKeyTile;
              if (!a.mask) {
#pragma unroll
                for (int w = 0; w < 4; ++w) see[w] = first_bits(slot + 1 - b0, w);
              } else {
                // the warp's slots, eight at a time: a byte a lane, 32 bytes to a word by ballot
                const int s0 = tile * p.per_tile + by_group(p, (warp & 3) * 32);
                const int s1 = tile * p.per_tile + by_group(p, (warp & 3) * 32 + 31);
                const uint8_t* mask = a.mask + static_cast<int64_t>(sg.req) * a.slots * a.slots + b0 + lane;
                for (int x = s0; x <= s1; x += 8) {
                  uint8_t byte[8][4];
#pragma unroll
                  for (int y = 0; y < 8; ++y)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                      byte[y][w] = x + y <= s1 && x + y < a.slots && b0 + 32 * w + lane < a.slots
                                       ? __ldg(mask + static_cast<int64_t>(x + y) * a.slots + 32 * w) : 0;
#pragma unroll
                  for (int y = 0; y < 8; ++y)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                      const uint32_t word = __ballot_sync(0xFFFFFFFFu, byte[y][w] != 0);
                      if (slot == x + y) see[w] = word;
                    }
                }
              }
              if (!live) see[0] = see[1] = see[2] = see[3] = 0;
            }
            ok = ok && warp_wait(&s_full[t], s_use++ & 1);
            if (!ok) break;
            tc_fence_after();
            const TreeTile& info = tiles[(count + j) % kTreeSlots];
            bool all = true;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              see[w] &= info.seen[w];
              poison |= (see[w] & info.bad[w]) != 0;
              all &= see[w] == 0xFFFFFFFFu;
            }
            const bool masked = !__all_sync(0xFFFFFFFFu, all);
            auto scale = [&](int w) {
              const float2 x = *reinterpret_cast<const float2*>(&info.k_scale[2 * w]);
              return make_float2(c * x.x, c * x.y);
            };
            auto value = [&](int w) { return *reinterpret_cast<const float2*>(&info.v_scale[2 * w]); };
            auto value_log = [&](int w) { return *reinterpret_cast<const float2*>(&info.v_log[2 * w]); };
            if (fresh) softmax_tile<HD, kWeightPairs, true, false>(s_at, o_at, i == 0, scale, value, value_log, see, sm, ready);
            else if (masked) softmax_tile<HD, kWeights, true, false>(s_at, o_at, i == 0, scale, value, value_log, see, sm, ready);
            else softmax_tile<HD, kWeights, false, false>(s_at, o_at, i == 0, scale, value, value_log, see, sm, ready);
          }
          if (steps > 0) ok = ok && warp_wait(&o_full[t], o_use++ & 1);
          tc_fence_after();
        }
        count += n;

        // --- the end of a stretch: the answer, or a part of it
        const int c_first = cut.of(sg.first), c_last = cut.of(sg.first + sg.units - 1);
        const bool alone = c_first == c_last && !split;
        auto out_of = [&](int z, int x) -> __nv_bfloat16* {  // row z of the warp, channel x
          const int y = (warp & 3) * 32 + z, ys = by_group(p, y), sl = tile * p.per_tile + ys;
          return y < p.per_tile * p.group && sl < a.slots
                     ? static_cast<__nv_bfloat16*>(a.out) + (static_cast<int64_t>(sg.req) * a.slots + sl) * a.out_row_stride +
                           (sg.kvh * p.group + y - ys * p.group) * a.out_head_stride + x
                     : nullptr;
        };
        auto finish_lse = [&](float top, float sum) {
          if (live && a.lse) a.lse[row * a.n_q + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        };
        {
          const float unit = ex2(sm.u - sm.m), inv = sm.u == -INFINITY || sm.l == 0.0f ? 0.0f : alone ? unit / sm.l : unit;  // (O to the sum's unit)
          const size_t mine = static_cast<size_t>(2 * piece + (piece == c_first)) * 2 + t;
          const bool nan = sm.l != sm.l || poison, none = steps == 0;  // (none: nothing was put into O)
#pragma unroll
          for (int x = 0; x < HD; x += 64) {
            uint32_t v[64];
            tmem_ld32(o_at + x, v);
            tmem_ld32(o_at + x + 32, v + 32);
            tmem_wait_ld();
            tmem_landed32(v);
            tmem_landed32(v + 32);
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = none ? 0u : __float_as_uint(nan ? NAN : __uint_as_float(v[i]) * inv);
            if (alone) {
              uint4 w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                w[k].x = pack_p(__uint_as_float(v[8 * k]), __uint_as_float(v[8 * k + 1]));
                w[k].y = pack_p(__uint_as_float(v[8 * k + 2]), __uint_as_float(v[8 * k + 3]));
                w[k].z = pack_p(__uint_as_float(v[8 * k + 4]), __uint_as_float(v[8 * k + 5]));
                w[k].w = pack_p(__uint_as_float(v[8 * k + 6]), __uint_as_float(v[8 * k + 7]));
              }
              // (through the row tile's own Q, which the next segment's replaces after this)
              store_rows(smem + Smem::kQ + t * Smem::kOperand + (warp & 3) * 4096, w, [&](int z) { return out_of(z, x); });
            } else {
#pragma unroll
              for (int i = 0; i < 64; i += 4)
                __stcg(reinterpret_cast<float4*>(p.part) + (mine * (HD / 4) + (x + i) / 4) * 128 + r,
                       make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])));
            }
          }
          if (alone) finish_lse(sm.m, sm.l);
          else __stcg(reinterpret_cast<float2*>(stats) + mine * 128 + r, make_float2(sm.m, sm.l));
          tc_fence_before();  // (O is read before the next segment's first product writes it)
        }
        if (!alone) {
          const bool own = c_first == c_last;  // (a split row tile of one piece: both parts are this CTA's)
          if (!own) __threadfence();
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (own) {
            if (tid == 0) s_last = 1;
          } else if (tid == 0) {
            unsigned* done = p.done + (static_cast<size_t>(sg.req) * n_kv + sg.kvh) * (p.pairs + p.odd) + sg.pair;
            s_last = atomicAdd(done, 1u) == static_cast<unsigned>(c_last - c_first);
            if (s_last) *done = 0u;  // ready for the next call
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (s_last && !(split && t == 1)) {
            if (!own) __threadfence();
            // parts in the order of keys: of each piece that of this row tile, or both slots' of a split one
            const int parts = (c_last - c_first + 1) << (split ? 1 : 0);
            auto part_of = [&](int x) {
              const int pc = c_first + (split ? x >> 1 : x);
              return static_cast<size_t>(2 * pc + (pc == c_first)) * 2 + (split ? x & 1 : t);
            };
            float top = -INFINITY, sum = 0.0f;
            for (int x = 0; x < parts; ++x) top = fmaxf(top, __ldcg(reinterpret_cast<const float2*>(stats) + part_of(x) * 128 + r).x);
            const float base = top == -INFINITY ? 0.0f : top;
            for (int x = 0; x < parts; ++x) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(stats) + part_of(x) * 128 + r);
              sum += ml.y * ex2(ml.x - base);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int x = 0; x < HD; x += 64) {
              float4 o[16] = {};
              for (int k = 0; k < parts; ++k) {
                const float f = ex2(__ldcg(reinterpret_cast<const float2*>(stats) + part_of(k) * 128 + r).x - base);
                const float4* y = reinterpret_cast<const float4*>(p.part) + (part_of(k) * (HD / 4) + x / 4) * 128 + r;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float4 z = __ldcg(y + i * 128);
                  o[i].x += z.x * f, o[i].y += z.y * f, o[i].z += z.z * f, o[i].w += z.w * f;
                }
              }
              uint4 w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                w[k] = make_uint4(pack_p(o[2 * k].x * inv, o[2 * k].y * inv), pack_p(o[2 * k].z * inv, o[2 * k].w * inv),
                                  pack_p(o[2 * k + 1].x * inv, o[2 * k + 1].y * inv),
                                  pack_p(o[2 * k + 1].z * inv, o[2 * k + 1].w * inv));
              store_rows(smem + Smem::kQ + t * Smem::kOperand + (warp & 3) * 4096, w, [&](int z) { return out_of(z, x); });
            }
            finish_lse(top, sum);
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");  // (s_last has been read)
        }
      }
      gave_up = !ok;
    }
    if (gave_up && a.status) atomicOr(a.status, DT_KV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTreeMmaWarp) {
    // (where a wait gave up: no product may outlive its operands and tensor memory)
    if (elect_one()) tc_commit(&drained);
    mbar_wait(&drained, 0, nullptr);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Grid: a CTA for each SM, and no more than units there can be.
inline int tree_grid(long long max_units) { return static_cast<int>(max_units < kSms ? max_units : kSms); }
inline size_t tree_workspace(int head_dim) {
  return kCounterBytes + static_cast<size_t>(2 * kSms) * 2 * 128 * (head_dim + 2) * 4;
}

template <int HD>
cudaError_t launch_tree(const TreeParams& p, int grid, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_tree<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeSmem<HD>::kBytes);
  if (e != cudaSuccess) return e;
  k_tree<HD><<<grid, kTreeThreads, TreeSmem<HD>::kBytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dt
