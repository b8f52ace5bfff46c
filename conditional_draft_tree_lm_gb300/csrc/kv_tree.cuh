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
// about the cache's bytes.
//
// Cached keys and values come to shared memory as fp16 (e4m3 is exact in it) by
// four converting warps: 8-bit pieces are copied a tile ahead (cp.async, into
// slots of the copying thread's own), converted, and stored in the layout that the
// products read.  What a page's scale would change stays exact in 32 bits: the
// key's scale multiplies the logit, the value's is folded into V relative to the
// largest scale so far, O being in units of that one (exact for powers of two).
// Q is brought to fp16 by a power of two per row, new keys and values by one per
// tile.  fp16 keeps 11 bits of P where bf16 would keep 8.
//
// Split.  The work is the list of (key/value head, request, row tiles, key tile),
// cut into equal pieces, one for each SM; a unit is a key tile for two row tiles
// and two key tiles for one.  A stretch that several pieces share is joined by the
// CTA that finishes last, in the order of keys.
#pragma once

#include "kv_decode.cuh"
#include "kv_flash.cuh"

namespace dt {

constexpr int kTreeStages = 4;   // K and V tiles, alternating
constexpr int kTreeSlots = 4;    // what goes with a key tile: its scales and masks
constexpr int kTreeMmaWarp = 8, kTreeConvWarp = 9, kTreeConvWarps = 4;
constexpr int kConvThreads = 32 * kTreeConvWarps;
constexpr int kTreeThreads = 32 * (kTreeConvWarp + kTreeConvWarps);

struct TreeParams {
  dt_kv_cache c;
  dt_cache_attention_args a;
  int group, shift;
  int per_tile;     // slots of a row tile
  int pairs, odd;   // pairs of row tiles, and whether one is left
  int fresh_tiles;  // key tiles of new tokens
  unsigned* done;   // [n_req * n_kv * (pairs + odd)] zero between launches
  float* part;      // [2 * pieces][2 tiles][HD / 4][128][4], then [2 * pieces][2][128][2]
};

// The key tiles of a request, and its units over all its row tiles.
DT_DEVINL int tree_key_tiles(int len, int max_len, int fresh) {
  len = min(max(len, 0), max_len);
  return max(1, (len + kKeyTile - 1) / kKeyTile + fresh);
}
struct TreeUnits {
  int max_len, fresh, pairs, odd;
  DT_DEVINL int operator()(int len) const {
    const int kt = tree_key_tiles(len, max_len, fresh);
    return pairs * kt + odd * ((kt + 1) / 2);
  }
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
    const int kt = tree_key_tiles(len, max_len, p.fresh_tiles), half = (kt + 1) / 2;
    s.req = req;
    s.kvh = kvh;
    s.len = len;
    s.cached = (len + kKeyTile - 1) / kKeyTile;
    s.pair = min(local / kt, p.pairs);
    s.tiles = s.pair < p.pairs ? 2 : 1;
    const int in_req = s.pair * kt;
    s.first = base + in_req;
    s.units = s.tiles == 2 ? kt : half;
    const int stop = min(u_end, s.first + s.units);
    const int per = 3 - s.tiles;  // key tiles of a unit
    s.key_begin = (u - s.first) * per;
    s.key_end = min(kt, (stop - s.first) * per);
    const int total = p.pairs * kt + p.odd * half;
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

template <int HD>
struct TreeSmem {
  static constexpr uint32_t kOperand = kOperandBytes<HD>;
  static constexpr uint32_t kQ = 0, kRing = 2 * kOperand, kStaging = kRing + kTreeStages * kOperand;
  static constexpr uint32_t kStagingBytes = 2 * kKeyTile * HD;  // K, V: [piece][thread] of 16 bytes
  static constexpr uint32_t kBars = kStaging + kStagingBytes;
  static constexpr uint32_t kBytes = kBars + 512 + 1024;  // + alignment
};

// What the converting warps leave with a key tile for the softmax.
struct TreeTile {
  float k_scale[8];   // of 16 keys each
  uint32_t seen[4];   // cached keys that exist (new ones: the keys below slots)
  uint32_t bad[4];    // keys whose values are not finite (new ones only)
  float ratio, vref;  // O's unit before / after this tile, and after
};

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
  TreeTile* tiles = reinterpret_cast<TreeTile*>(o_full + 2);  // [kTreeSlots]
  __shared__ uint32_t tmem_slot;
  __shared__ int scratch[4], s_start[128 + 1], s_last;
  __shared__ float s_max[2][kTreeConvWarps];

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
    }
    fence_mbar_init();
  }
  tc_fence_before();
  const TreeUnits units = {a.max_blocks << p.shift, p.fresh_tiles, p.pairs, p.odd};
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

    if (warp == kTreeMmaWarp) {
      const bool leader = elect_one();
      int count = 0;  // key tiles so far
      int s_use[2] = {0, 0}, segs[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, nullptr));
        tc_fence_after();
      };
      auto full_wait = [&](int i) { wait(&full[i % kTreeStages], (i / kTreeStages) & 1); };
      auto at = [&](int i) { return ring + (i % kTreeStages) * Smem::kOperand; };
      auto commit = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
      };
      const uint64_t q_desc[2] = {flash_desc(q_s, false), flash_desc(q_s + Smem::kOperand, false)};
      while (ok && walk.next(p, sg)) {
        const int n = sg.key_end - sg.key_begin;
        full_wait(2 * count);
        uint64_t kd = flash_desc(at(2 * count), false);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= sg.tiles) continue;
          wait(&q_full[t], segs[t]++ & 1);
          if (!ok) break;
          if (leader) issue_qk<HD, false>(tmem + t * 128, q_desc[t], kd);
          commit(&s_full[t]);
        }
        if (ok) commit(&empty[(2 * count) % kTreeStages]);
        for (int j = 0; j < n && ok; ++j, ++count) {
          const int vi = 2 * count + 1, ki = 2 * count + 2;
          const bool more = j + 1 < n;
          full_wait(vi);
          if (more) full_wait(ki);
          const uint64_t vd = flash_desc(at(vi), true);
          kd = flash_desc(at(ki), false);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || t >= sg.tiles) continue;
            const uint32_t turn = s_use[t]++ & 1;
            wait(&p_full[2 * t], turn);
            if (ok && leader) issue_pv<HD, false>(tmem + 256 + t * 128, tmem + t * 128, vd, j == 0, 0);
            wait(&p_full[2 * t + 1], turn);
            if (!ok) continue;
            if (leader) issue_pv<HD, false>(tmem + 256 + t * 128, tmem + t * 128, vd, j == 0, 1);
            if (more) {
              if (leader) issue_qk<HD, false>(tmem + t * 128, q_desc[t], kd);
              commit(&s_full[t]);
            } else {
              commit(&o_full[t]);
            }
          }
          if (ok) {
            commit(&empty[vi % kTreeStages]);
            if (more) commit(&empty[ki % kTreeStages]);
          }
        }
      }
    } else if (warp >= kTreeConvWarp) {
      // --- conversion: tile after tile, the next one's 8-bit pieces in flight, the one's after that page numbers too
      constexpr int kLanes = HD / 16;               // threads of a key's row (16 bytes each)
      constexpr int kPassRows = kConvThreads / kLanes;
      constexpr int kPasses = kKeyTile / kPassRows;  // pieces of a thread
      const int ct = tid - kTreeConvWarp * 32, cw = ct >> 5, cc = ct % kLanes, cr = ct / kLanes;
      struct Tile {
        int kind, key0, req, kvh, len;  // kind: 0 none, 1 cached, 2 new, + 4 for the first of a segment
      };
      int key = 0;
      auto advance = [&](Tile& t) {
        if (key >= sg.key_end || sg.tiles == 0) {
          if (!walk.next(p, sg)) {
            sg.tiles = 0;
            t.kind = 0;
            return;
          }
          key = sg.key_begin;
        }
        const bool cached = key < sg.cached;
        // (a request without a key at all still has a tile: a cached one of length 0)
        t.kind = (cached || !a.k_new ? 1 : 2) + (key == sg.key_begin ? 4 : 0);
        t.key0 = (cached || !a.k_new ? key : key - sg.cached) * kKeyTile;
        t.req = sg.req;
        t.kvh = sg.kvh;
        t.len = sg.len;
        ++key;
      };
      struct Page {  // of 16 keys, held by lanes 0..7 of every warp
        int id;
        float ks, vs;
      };
      auto pages_of = [&](const Tile& t) {
        Page g = {-1, 0.0f, 0.0f};
        const int tok = t.key0 + lane * 16;
        if ((t.kind & 3) == 1 && lane < 8 && tok < t.len) {
          g.id = __ldg(a.block_table + static_cast<size_t>(t.req) * a.max_blocks + (tok >> p.shift));
          if (g.id < 0 || g.id >= p.c.n_pages) {
            if (a.status && cw == 0) atomicOr(a.status, DT_KV_BAD_INDEX);
            g.id = -1;
          } else {
            const size_t at = static_cast<size_t>(g.id) * n_kv + t.kvh;
            g.ks = __ldg(p.c.k_scale + at);
            g.vs = __ldg(p.c.v_scale + at);
          }
        }
        return g;
      };
      uint8_t* staging = smem + Smem::kStaging;
      auto fetch = [&](const Tile& t, const Page& g, const void* codes, int which) {
        if ((t.kind & 3) == 1) {
#pragma unroll
          for (int i = 0; i < kPasses; ++i) {
            const int row = i * kPassRows + cr;
            const int id = __shfl_sync(0xFFFFFFFFu, g.id, row >> 4);
            if (id >= 0) {
              const size_t at = (((static_cast<size_t>(id) * n_kv + t.kvh) << p.shift) + ((t.key0 + row) & ((1 << p.shift) - 1))) * HD + cc * 16;
              cp_async16(smem_u32(staging + ((which * kPasses + i) * kConvThreads + ct) * 16), static_cast<const uint8_t*>(codes) + at);
            }
          }
        }
        cp_commit();
      };
      // 8 halves to their place: key `row`, channels 8 * chunk ..
      auto put = [&](uint8_t* op, int row, int chunk, const uint4& w) {
        *reinterpret_cast<uint4*>(op + (chunk >> 3) * kHalfBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = w;
      };
      auto arrive = [&](int i) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[i % kTreeStages]);
      };
      // a cached tile's K or V out of the staging place, values multiplied by a factor per 16 keys
      auto convert = [&](const Tile& t, const Page& g, int which, float inv) {
        uint4 w[kPasses];
#pragma unroll
        for (int k = 0; k < kPasses; ++k)
          w[k] = *reinterpret_cast<const uint4*>(staging + ((which * kPasses + k) * kConvThreads + ct) * 16);
        return [=](uint8_t* op) {
#pragma unroll
          for (int k = 0; k < kPasses; ++k) {
            const int row = k * kPassRows + cr;
            const int id = __shfl_sync(0xFFFFFFFFu, g.id, row >> 4);
            const float f = which ? __shfl_sync(0xFFFFFFFFu, g.vs, row >> 4) * inv : 1.0f;
            const uint32_t in[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint32_t h[8];
            const __half2 f2 = __float2half2_rn(f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              e4m3x4_to_f16x2x2(in[x], h[2 * x], h[2 * x + 1]);
              if (which) {
                __half2* y = reinterpret_cast<__half2*>(&h[2 * x]);
                y[0] = __hmul2(y[0], f2);
                y[1] = __hmul2(y[1], f2);
              }
            }
            const bool live = id >= 0 && t.key0 + row < t.len;
            const uint4 lo = live ? make_uint4(h[0], h[1], h[2], h[3]) : make_uint4(0, 0, 0, 0);
            const uint4 hi = live ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(0, 0, 0, 0);
            // the two halves of a row's threads start with different chunks: no bank conflict
            const bool swap = HD == 128 && (cc & 4);
            put(op, row, 2 * cc + (swap ? 1 : 0), swap ? hi : lo);
            put(op, row, 2 * cc + (swap ? 0 : 1), swap ? lo : hi);
          }
        };
      };
      // a new tile's K or V, bf16: its largest finite magnitude first, then fp16 by a power of two
      auto convert_new = [&](const Tile& t, int which, float& vref, float& scale, uint32_t* bad, uint8_t* op) {
        constexpr int kL = HD / 8, kR = kConvThreads / kL, kP = kKeyTile / kR;
        const int c8 = ct % kL, r8 = ct / kL;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(which ? a.v_new : a.k_new);
        const int64_t rs = which ? a.v_row_stride : a.k_row_stride, hs = which ? a.v_head_stride : a.k_head_stride;
        float top = 0.0f;
        auto piece_of = [&](int k) {
          const int b = t.key0 + k * kR + r8;
          return b < a.slots ? __ldg(reinterpret_cast<const uint4*>(x + (static_cast<int64_t>(t.req) * a.slots + b) * rs +
                                                                    t.kvh * hs + c8 * 8))
                             : make_uint4(0, 0, 0, 0);
        };
        // (read twice, the second time from L1: a tile would take 64 registers)
#pragma unroll 4
        for (int k = 0; k < kP; ++k) {
          const uint4 w = piece_of(k);
          const uint32_t in[4] = {w.x, w.y, w.z, w.w};
          bool odd = false;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float lo = fabsf(__uint_as_float(in[y] << 16)), hi = fabsf(__uint_as_float(in[y] & 0xFFFF0000u));
            const bool fl = lo <= 3.402823466e38f, fh = hi <= 3.402823466e38f;
            odd |= !fl || !fh;
            top = fmaxf(top, fmaxf(fl ? lo : 0.0f, fh ? hi : 0.0f));
          }
          // the key's value takes no part in the product, the rows that see it become NaN
          if (which && odd) atomicOr(&bad[(k * kR + r8) >> 5], 1u << ((k * kR + r8) & 31));
        }
        top = warp_max(top);
        if (lane == 0) s_max[which][cw] = top;
        asm volatile("bar.sync 2, %0;" ::"n"(kConvThreads) : "memory");
#pragma unroll
        for (int k = 0; k < kTreeConvWarps; ++k) top = fmaxf(top, s_max[which][k]);
        asm volatile("bar.sync 2, %0;" ::"n"(kConvThreads) : "memory");
        scale = kv_pow2_scale(top);
        if (which) vref = fmaxf(vref, scale), scale = vref;
        const float inv = 1.0f / scale;
#pragma unroll 4
        for (int k = 0; k < kP; ++k) {
          const int row = k * kR + r8;
          const uint4 w = piece_of(k);
          const uint32_t in[4] = {w.x, w.y, w.z, w.w};
          uint32_t h[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            h[y] = pack_f16(__uint_as_float(in[y] << 16) * inv, __uint_as_float(in[y] & 0xFFFF0000u) * inv);
          const bool zero = which && (bad[row >> 5] >> (row & 31) & 1u);
          put(op, row, c8, zero ? make_uint4(0, 0, 0, 0) : make_uint4(h[0], h[1], h[2], h[3]));
        }
      };

      sg.tiles = 0;
      Tile cur, nxt, nx2;
      advance(cur);
      Page gc = pages_of(cur);
      advance(nxt);
      Page gn = pages_of(nxt);
      fetch(cur, gc, p.c.k, 0);
      fetch(cur, gc, p.c.v, 1);
      float vref = 0.0f;
      // (where a wait gives up the loop goes on without waiting: other warps may stand at its named barrier)
      bool ok = true;
      auto room = [&](int i) { ok = ok && mbar_wait(&empty[i % kTreeStages], ((i / kTreeStages) & 1) ^ 1, nullptr); };
      for (int count = 0; cur.kind; ++count) {
        advance(nx2);
        const Page g2 = pages_of(nx2);
        TreeTile& info = tiles[count % kTreeSlots];
        const int ki = 2 * count, vi = ki + 1;
        if (cur.kind & 4) vref = 1.17549435e-38f;
        const float before = vref;
        uint8_t* k_op = smem + Smem::kRing + (ki % kTreeStages) * Smem::kOperand;
        uint8_t* v_op = smem + Smem::kRing + (vi % kTreeStages) * Smem::kOperand;
        if ((cur.kind & 3) == 1) {
          cp_wait<1>();
          auto store_k = convert(cur, gc, 0, 1.0f);
          fetch(nxt, gn, p.c.k, 0);
          room(ki);
          float top = lane < 8 ? gc.vs : 0.0f;
          top = warp_max(top);
          vref = fmaxf(vref, top);
          if (cw == 0) {
            if (lane < 8) info.k_scale[lane] = gc.ks;
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, lane < 8 && gc.id >= 0);
            if (lane < 4) {
              const uint32_t two = there >> (2 * lane);
              info.seen[lane] = first_bits(cur.len - cur.key0, lane) & (((two & 1) ? 0xFFFFu : 0u) | ((two & 2) ? 0xFFFF0000u : 0u));
              info.bad[lane] = 0;
            }
            if (lane == 0) {
              info.ratio = (cur.kind & 4) ? 1.0f : before / vref;
              info.vref = vref;
            }
          }
          store_k(k_op);
          arrive(ki);
          cp_wait<1>();
          auto store_v = convert(cur, gc, 1, 1.0f / vref);
          fetch(nxt, gn, p.c.v, 1);
          room(vi);
          store_v(v_op);
          arrive(vi);
        } else {
          // (the groups of this tile hold nothing; the next tile's take their places in the count)
          cp_wait<0>();
          fetch(nxt, gn, p.c.k, 0);
          room(ki);
          if (ct < 4) info.bad[ct] = 0;
          float scale;
          convert_new(cur, 0, vref, scale, info.bad, k_op);  // (its barriers order the zeros before)
          if (ct < 8) info.k_scale[ct] = scale;
          if (ct < 4) info.seen[ct] = first_bits(a.slots - cur.key0, ct);
          // the values before the keys are handed over: the tile's ratio goes with the keys
          room(vi);
          convert_new(cur, 1, vref, scale, info.bad, v_op);
          if (ct == 0) {
            info.ratio = (cur.kind & 4) ? 1.0f : before / vref;
            info.vref = vref;
          }
          fetch(nxt, gn, p.c.v, 1);
          arrive(ki);
          arrive(vi);
        }
        cur = nxt;
        gc = gn;
        nxt = nx2;
        gn = g2;
      }
      cp_wait<0>();
    } else {
      // --- softmax: warpgroup t, a row a thread
      const int t = warp >> 2, r = tid & 127;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + 256 + t * 128 + lanes;
      float* stats = p.part + static_cast<size_t>(2 * pieces) * 2 * 128 * HD;
      int count = 0, s_use = 0, o_use = 0;
      bool ok = true;
      // (where a wait gives up, likewise)
      while (walk.next(p, sg)) {
        const int n = sg.key_end - sg.key_begin;
        const int slot = (sg.pair * 2 + t) * p.per_tile + r / p.group, head = sg.kvh * p.group + r % p.group;
        const bool live = t < sg.tiles && r < p.per_tile * p.group && slot < a.slots;
        const int64_t row = static_cast<int64_t>(sg.req) * a.slots + slot;
        float m = -INFINITY, l = 0.0f, vref = 0.0f;
        if (t < sg.tiles) {
          // Q to fp16 by a power of two of the row's own
          float c;
          {
            float amax = 0.0f;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row * a.q_row_stride + head * a.q_head_stride;
            auto piece_of = [&](int i) {
              return live ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
            };
#pragma unroll 8
            for (int i = 0; i < HD / 8; ++i) {
              const uint4 w = piece_of(i);
              const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int y = 0; y < 4; ++y)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(in[y] << 16)), fabsf(__uint_as_float(in[y] & 0xFFFF0000u))));
            }
            int k = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
            k = min(max(k, -100), 127);
            const float up = __uint_as_float(static_cast<uint32_t>(14 - k + 127) << 23);
            c = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(k - 14 + 127) << 23);
            uint8_t* op = smem + Smem::kQ + t * Smem::kOperand;
#pragma unroll 8
            for (int i = 0; i < HD / 8; ++i) {
              const uint4 w = piece_of(i);
              const uint32_t in[4] = {w.x, w.y, w.z, w.w};
              uint32_t h[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                h[y] = pack_f16(__uint_as_float(in[y] << 16) * up, __uint_as_float(in[y] & 0xFFFF0000u) * up);
              *reinterpret_cast<uint4*>(op + (i >> 3) * kHalfBytes + r * 128 + (((i & 7) ^ (r & 7)) << 4)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[t]);
          }
          bool poison = false;
          for (int j = 0; j < n; ++j) {
            const int key = sg.key_begin + j;
            const bool fresh = a.k_new && key >= sg.cached;
            uint32_t see[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
            if (fresh) {  // which of the new tokens this row sees, while the product runs
              const int b0 = (key - sg.cached) * kKeyTile;
              const uint8_t* mask = a.mask ? a.mask + row * a.slots + b0 : nullptr;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                if (!live) {
                  see[w] = 0;
                } else if (!mask) {
                  see[w] = first_bits(slot + 1 - b0, w);
                } else {
                  uint32_t x = 0;
                  for (int i = 0; i < 32; ++i)
                    if (b0 + w * 32 + i < a.slots) x |= (mask[w * 32 + i] != 0 ? 1u : 0u) << i;
                  see[w] = x;
                }
              }
            }
            ok = ok && mbar_wait(&s_full[t], s_use++ & 1, nullptr);
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
            vref = info.vref;
            const float ratio = info.ratio;
            // the largest logit that is seen, 16 keys (of one scale) at a time
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t s[32];
              tmem_ld32(s_at + 32 * w, s);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float ck = c * info.k_scale[2 * w + h];
                float hi = -INFINITY, lo = INFINITY;
                if (!masked) {
                  if (c >= 0.0f) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) hi = fmaxf(hi, __uint_as_float(s[16 * h + i]));
                    top = fmaxf(top, hi * ck);
                  } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) lo = fminf(lo, __uint_as_float(s[16 * h + i]));
                    top = fmaxf(top, lo * ck);
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    if (see[w] >> (16 * h + i) & 1u) top = fmaxf(top, __uint_as_float(s[16 * h + i]) * ck);
                }
              }
            }
            if (__any_sync(0xFFFFFFFFu, top > m + 8.0f || ratio != 1.0f)) {
              const float m2 = fmaxf(m, top), f = m2 == -INFINITY ? 1.0f : ex2(m - m2);
              if (j > 0) rescale_o<HD>(o_at, f * ratio);
              l *= f;
              m = m2;
            }
            const float base = m == -INFINITY ? 0.0f : m;
            float sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t s[32], pk[16];
              tmem_ld32(s_at + 32 * w, s);
              const float ck[2] = {c * info.k_scale[2 * w], c * info.k_scale[2 * w + 1]};
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float e0 = ex2(fmaf(__uint_as_float(s[2 * i]), ck[i >> 3], -base));
                float e1 = ex2(fmaf(__uint_as_float(s[2 * i + 1]), ck[i >> 3], -base));
                if (masked) {
                  if (!(see[w] >> (2 * i) & 1u)) e0 = 0.0f;
                  if (!(see[w] >> (2 * i + 1) & 1u)) e1 = 0.0f;
                }
                sum[(2 * i) & 3] += e0;
                sum[(2 * i + 1) & 3] += e1;
                pk[i] = pack_f16(e0, e1);
              }
              tmem_st16(s_at + 16 * w, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t]), mbar_arrive(&p_full[2 * t + 1]);
          }
          if (poison) l = NAN;
          if (ok) ok = mbar_wait(&o_full[t], o_use++ & 1, nullptr);
          tc_fence_after();
        }
        count += n;

        // --- the end of a stretch: the answer, or a part of it
        const int c_first = cut.of(sg.first), c_last = cut.of(sg.first + sg.units - 1);
        const bool alone = c_first == c_last;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * a.out_row_stride + head * a.out_head_stride;
        auto finish_lse = [&](float top, float sum) {
          if (live && a.lse) a.lse[row * a.n_q + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        };
        if (t < sg.tiles) {
          const float inv = alone ? (l == 0.0f ? 0.0f : vref / l) : vref;
          const size_t mine = static_cast<size_t>(2 * piece + (piece == c_first)) * 2 + t;
          // (O in units of vref; where nothing was seen, it is zeros, or in a first tile never NaN: V is finite then)
#pragma unroll
          for (int x = 0; x < HD; x += 32) {
            uint32_t v[32];
            tmem_ld32(o_at + x, v);
            tmem_wait_ld();
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[i]) * inv;
            if (l != l) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = NAN;
            }
            if (alone) {
              if (live) {
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                  *reinterpret_cast<uint4*>(out + x + i) = make_uint4(pack_p<true>(o[i], o[i + 1]), pack_p<true>(o[i + 2], o[i + 3]),
                                                                      pack_p<true>(o[i + 4], o[i + 5]), pack_p<true>(o[i + 6], o[i + 7]));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                __stcg(reinterpret_cast<float4*>(p.part) + (mine * (HD / 4) + (x + i) / 4) * 128 + r,
                       make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
            }
          }
          if (alone) finish_lse(m, l);
          else __stcg(reinterpret_cast<float2*>(stats) + mine * 128 + r, make_float2(m, l));
          tc_fence_before();  // (O is read before the next segment's first product writes it)
        }
        if (!alone) {
          __threadfence();
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (tid == 0) {
            unsigned* done = p.done + (static_cast<size_t>(sg.req) * n_kv + sg.kvh) * (p.pairs + p.odd) + sg.pair;
            s_last = atomicAdd(done, 1u) == static_cast<unsigned>(c_last - c_first);
            if (s_last) *done = 0u;  // ready for the next call
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (s_last && t < sg.tiles) {
            __threadfence();
            auto part_of = [&](int x) { return static_cast<size_t>(2 * x + (x == c_first)) * 2 + t; };
            float top = -INFINITY, sum = 0.0f;
            for (int x = c_first; x <= c_last; ++x) top = fmaxf(top, __ldcg(reinterpret_cast<const float2*>(stats) + part_of(x) * 128 + r).x);
            const float base = top == -INFINITY ? 0.0f : top;
            for (int x = c_first; x <= c_last; ++x) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(stats) + part_of(x) * 128 + r);
              sum += ml.y * ex2(ml.x - base);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int c8 = 0; c8 < HD / 8; ++c8) {
              float o[8] = {};
              for (int x = c_first; x <= c_last; ++x) {
                const float f = ex2(__ldcg(reinterpret_cast<const float2*>(stats) + part_of(x) * 128 + r).x - base);
                const float4* y = reinterpret_cast<const float4*>(p.part) + (part_of(x) * (HD / 4) + 2 * c8) * 128 + r;
                const float4 y0 = __ldcg(y), y1 = __ldcg(y + 128);
                o[0] += y0.x * f, o[1] += y0.y * f, o[2] += y0.z * f, o[3] += y0.w * f;
                o[4] += y1.x * f, o[5] += y1.y * f, o[6] += y1.z * f, o[7] += y1.w * f;
              }
              if (live)
                *reinterpret_cast<uint4*>(out + 8 * c8) = make_uint4(pack_p<true>(o[0] * inv, o[1] * inv), pack_p<true>(o[2] * inv, o[3] * inv),
                                                                     pack_p<true>(o[4] * inv, o[5] * inv), pack_p<true>(o[6] * inv, o[7] * inv));
            }
            finish_lse(top, sum);
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");  // (s_last has been read)
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTreeMmaWarp) {
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
