// dt_cache_attention for few query rows per key/value head (slots * group <= 16:
// single tokens, short drafts; or as few rows behind a tree's full row tiles):
// streaming the 8-bit cache once.
//
// Per key/value head the group's rows share every cached key, so a call reads
// len * 2 * head_dim bytes for 4 * rows * len * head_dim flops: at most 32 flops
// a byte here, far below the tensor cores' balance, so it is bound by the cache's
// bytes (HBM), or by latency when the whole call is a few microseconds.
//
// Split.  The work is the list of (key/value head, request, tile of 128 tokens),
// cut into pieces of equal length, one or more for each CTA of a grid that fits
// the GPU at once; the cut depends on the lengths only, however ragged they are.
// Every CTA finds its place by summing the lengths itself (no extra launch, no
// host copy of lengths).  A (request, head) that several pieces share is joined by
// the CTA that finishes last, in the order of tiles, so results do not depend on
// timing.  What a new (request, head) costs is a chain of memory latencies (page
// numbers, scales, Q, the first tiles, the join's fence and parts), so the next
// one's first steps are put in flight before the last one is joined.
//
// A warp takes steps of two times 16 keys (two, so that their chains of products
// overlap) from a ring of its own in shared memory, which one of its lanes keeps
// filled by TMA (copies by the threads themselves, 16 bytes each, stopped at 4.9
// TB/s whatever their number in flight; with TMA the same stream runs at 6.5).  The
// 128-byte swizzle spreads a fragment's rows over the banks:
//   S^T[key, row] = K (A, 16 keys) Q^T (B, 8 rows): a thread supplies 4 adjacent
//     channels of keys lane/4 and lane/4 + 8 per product; which channel is which k
//     is free as long as Q uses the same order, so 16-byte pieces feed four products.
//   O^T[channel, row] = V^T (A) P^T (B): S^T's fragment, rounded to fp16 and
//     transposed by movmatrix, is the B fragment; a thread supplies 16 adjacent
//     channels of 4 keys, two keys' bytes interleaved by a byte permute.
// e4m3 goes to fp16 exactly (one conversion for two values).  The page scales stay
// outside: the key's multiplies the logit, the value's is folded into P, in a
// unit of the row's own that follows the keys (move_unit).  Q is brought to fp16 by a power of two per
// row (exact to 2^-40 of the row's maximum), P is held in fp16: 11 bits, where
// bf16 would give 8.  Maxima, sums and O are 32 bits.  New tokens' keys and values
// take the same products in bf16 (row by row with plain multiplications: 15 us more
// for 32 trees of 65 slots, 40 us for a tree of 513).
//
// Measured: 32 tokens over caches of up to 16k tokens (671 MB) 109 us, 6.2 TB/s, 91 %
// of the measured copy bandwidth; one token over 2k 7.7 us, a chain of latencies.
#pragma once

#include <cuda.h>

#include "kv.cuh"

namespace dt {

constexpr int kDecodeMaxRows = 16;
constexpr int kDecodeThreads = 128;
constexpr int kDecodeWarps = kDecodeThreads / 32;
constexpr int kDecodeTile = 32 * kDecodeWarps;  // tokens: a step of every warp
constexpr int kDecodeCtas = 2;                  // per SM

// The workspace starts with the joins' counters, at the same place for every call
// (so that no call's parts lie over another's counters), the parts follow.
constexpr size_t kCounterBytes = size_t(1) << 20;
constexpr int kMaxJoins = static_cast<int>(kCounterBytes / 4);

struct DecodeParams {
  dt_kv_cache c;
  dt_cache_attention_args a;
  int group, rows, shift;  // rows: of the slots from slot0 on, times group
  int slot0;
  int box;                 // rows of a copy: 32, or a page of 16
  unsigned* done;          // [n_req * n_kv] pieces that are done; zero between launches
  float* part;             // [2 * pieces][rows][HD], then [2 * pieces][rows][2]: a piece's first and last (request, head)
};

DT_DEVINL void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

DT_DEVINL void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit values held as mma fragments.
DT_DEVINL uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

DT_DEVINL uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Tiles of a request: at least one, so that a request without cached tokens has a place in the work too.
DT_DEVINL int tiles_of(int len, int max_len, int tile) {
  len = min(max(len, 0), max_len);
  return max(1, (len + tile - 1) / tile);
}
struct DecodeTiles {
  int max_len;
  DT_DEVINL int operator()(int len) const { return tiles_of(len, max_len, kDecodeTile); }
};

// Where each request's tiles start in the row of all requests' tiles: starts of
// THREADS bins of requests in shared memory, the rest is summed when asked for.
// (The host refuses calls whose tiles over all heads could pass 2^30.)
template <int THREADS, class Tiles>
struct TileRow {
  const int32_t* length;
  int n_req;
  Tiles tiles;  // of a request of that length
  int per;      // requests of a bin
  int* start;   // [THREADS + 1] shared
  // All threads of the block (THREADS of them at least, and that many bins); ends with a barrier.
  DT_DEVINL void sum(int* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    per = (n_req + THREADS - 1) / THREADS;
    int own = 0;
    if (tid < THREADS)
      for (int q = tid * per; q < min(n_req, (tid + 1) * per); ++q) own += tiles(length[q]);
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31 && tid < THREADS) scratch[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) incl += w < warp ? scratch[w] : 0;
    if (tid < THREADS) start[tid + 1] = incl;
    if (tid == 0) start[0] = 0;
    __syncthreads();
  }
  DT_DEVINL int total() const { return start[THREADS]; }
  // The request in which tile `index` lies, and that request's first tile.
  DT_DEVINL void find(int index, int& req, int& first) const {
    int lo = 0, hi = THREADS;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= index) lo = mid; else hi = mid;
    }
    req = lo * per;
    first = start[lo];
    if (per == 1) return;
    for (;; ++req) {
      const int n = tiles(length[req]);
      if (index < first + n) break;
      first += n;
    }
  }
};

// [0, work) cut into n pieces that differ by one at most (n <= work).
struct Cut {
  int each, more;  // the first `more` pieces have each + 1
  DT_DEVINL Cut(int work, int n) : each(work / n), more(work % n) {}
  DT_DEVINL int begin(int i) const { return i * each + min(i, more); }
  DT_DEVINL int of(int u) const {
    const int edge = more * (each + 1);
    return u < edge ? u / (each + 1) : more + (u - edge) / each;
  }
};

// p.box key rows from row `row` of the cache, all of a row's bytes.
DT_DEVINL void tma_rows(void* dst, const void* tmap, uint64_t* bar, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(0), "r"(row)
      : "memory");
}

template <int HD, int RH>
struct DecodeSmem {
  // ring: [stage][warp][K, V][32 keys][HD], rows swizzled in 16-byte pieces; then the join (whose place the sums
  // of lengths take at first), the ring's barriers
  static constexpr int kStages = RH == 1 ? 3 : 2;  // (two CTAs' rings and joins fill an SM's shared memory)
  static constexpr int kStep = 2 * 32 * HD;        // a warp's step
  static constexpr int kRing = kStages * kDecodeWarps * kStep;
  static constexpr int kRows = 8 * RH;
  static constexpr int kJoin = kDecodeWarps * kRows * (HD + 2) * 4;
  static constexpr int kBytes = kRing + kJoin + kStages * kDecodeWarps * 8 + 16;
};

// A stretch of one (request, head) inside a piece.
struct DecodeSegment {
  int req, kvh, first, tiles;  // first: the (request, head)'s first tile in the work
  int begin, end;              // tokens
  int stop;                    // the tile behind it
};

template <int HD, int RH>  // RH: halves of 8 rows in use, 1 or 2
__global__ void __launch_bounds__(kDecodeThreads, kDecodeCtas)
    k_decode(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeParams p) {
  using Smem = DecodeSmem<HD, RH>;
  constexpr int kStages = Smem::kStages;
  constexpr int kKSteps = HD / 16;  // products of 16 channels; also tiles of 16 output channels
  constexpr int kVec = HD / 64;     // 16-byte pieces of a key per thread
  constexpr int kRows = Smem::kRows;
  constexpr int kQuads = HD / 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* s_o = reinterpret_cast<float*>(smem + Smem::kRing);  // [warps][kRows][HD]
  float* s_m = s_o + kDecodeWarps * kRows * HD;               // [warps][kRows]
  float* s_l = s_m + kDecodeWarps * kRows;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::kRing + Smem::kJoin);  // [warps][stages]
  int& s_last = *reinterpret_cast<int*>(bars + kDecodeWarps * kStages);
  int* s_start = reinterpret_cast<int*>(s_o);  // [threads + 1], then [warps]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const dt_cache_attention_args& a = p.a;
  const int n_kv = p.c.n_kv, max_len = a.max_blocks << p.shift;
  const __nv_bfloat16* q_base = static_cast<const __nv_bfloat16*>(a.q);
  const int page_mask = (1 << p.shift) - 1;
  uint8_t* ring = smem + warp * Smem::kStep;

  if (tid < kDecodeWarps * kStages) mbar_init(&bars[tid], 1);
  fence_mbar_init();
  bars += warp * kStages;
  int issued = 0, used = 0;  // of this warp's steps
  // a bounded wait did (the same for a warp's lanes): from then on there are neither waits nor copies, the joins go on as ever,
  // and the copies from `lost` on are waited for at the end
  bool gave_up = false;
  int lost = 0;
  TileRow<kDecodeThreads, DecodeTiles> row_of = {a.length, a.n_req, {max_len}, 0, s_start};
  row_of.sum(s_start + kDecodeThreads + 1);
  const int work = row_of.total() * n_kv;
  const int pieces = min(work, static_cast<int>(gridDim.x));
  // (where this kernel was started beside the one before it in the stream, it ends after that one)
  if (static_cast<int>(blockIdx.x) >= pieces) {
    dt_grid_wait();
    return;
  }
  const Cut cut(work, pieces);
  float* stats = p.part + static_cast<size_t>(2 * pieces) * p.rows * HD;
  const int piece = blockIdx.x;
  const int u_end = cut.begin(piece + 1);

  // where this thread's bytes of a key row stand: K: channels t * HD / 4 .. of key g; V: channels g * HD / 8 .. of
  // keys 2t and 2t + 1 (16-byte piece x of row r is at x ^ r % 8, of 64-byte rows at x ^ r / 2 % 4)
  int k_at[kVec], v_at[2];
#pragma unroll
  for (int y = 0; y < kVec; ++y)
    k_at[y] = g * HD + (HD == 128 ? ((2 * t + y) ^ g) << 4 : (t ^ (g >> 1)) << 4);
#pragma unroll
  for (int r = 0; r < 2; ++r)
    v_at[r] = (2 * t + r) * HD + (HD == 128 ? (g ^ (2 * t + r)) << 4 : ((g >> 1) ^ t) << 4 | (g & 1) << 3);

  // --- a segment's start: page numbers, the first steps and Q on their way
  DecodeSegment sg = {};
  int tok0 = 0, steps = 0;
  // lane 2 i + x keeps page and scales of half x of step 16 b + i, for the blocks b being copied and used
  int pg = -1;
  float ks[2] = {0, 0}, vs[2] = {0, 0};
  uint2 qw[RH][kKSteps];

  auto place = [&](int u) {  // sg.req, kvh, first are known: the segment that starts at tile u
    const int len = min(max(a.length[sg.req], 0), max_len);
    sg.tiles = tiles_of(len, max_len, kDecodeTile);
    sg.stop = min(u_end, sg.first + sg.tiles);
    sg.begin = (u - sg.first) * kDecodeTile;
    sg.end = min(len, (sg.stop - sg.first) * kDecodeTile);
    tok0 = sg.begin + warp * 32;
    steps = tok0 < sg.end ? (sg.end - tok0 + kDecodeTile - 1) / kDecodeTile : 0;
  };
  auto issue = [&](int i) {
    if (i < steps && !gave_up) {
      if ((i & 15) == 0) {
        const int tok = tok0 + (i + (lane >> 1)) * kDecodeTile + (lane & 1) * 16;
        float k1 = 0.0f, v1 = -1.0f;  // (a page out of range: as if it were not there)
        pg = -1;
        if (tok < sg.end) {
          pg = __ldg(a.block_table + static_cast<size_t>(sg.req) * a.max_blocks + (tok >> p.shift));
          if (pg < 0 || pg >= p.c.n_pages) {
            if (a.status) atomicOr(a.status, DT_KV_BAD_INDEX);
            pg = -1;
          } else {
            const size_t tile = static_cast<size_t>(pg) * n_kv + sg.kvh;
            k1 = __ldg(p.c.k_scale + tile);
            v1 = __ldg(p.c.v_scale + tile);
          }
        }
        if ((i >> 4) & 1) ks[1] = k1, vs[1] = v1;
        else ks[0] = k1, vs[0] = v1;
      }
      const int p0 = __shfl_sync(0xFFFFFFFFu, pg, (i & 15) * 2), p1 = __shfl_sync(0xFFFFFFFFu, pg, (i & 15) * 2 + 1);
      if (lane == 0) {
        uint8_t* st = ring + (issued % kStages) * kDecodeWarps * Smem::kStep;
        uint64_t* bar = &bars[issued % kStages];
        const int off = (tok0 + i * kDecodeTile) & page_mask;
        const bool second = p.box == 16 && p1 >= 0;  // (pages of 16: a copy for each half)
        mbar_arrive_expect_tx(bar, ((p0 >= 0) + second) * p.box * 2 * HD);
        if (p0 >= 0) {
          const int row = ((p0 * n_kv + sg.kvh) << p.shift) + off;
          tma_rows(st, &tm_k, bar, row);
          tma_rows(st + 32 * HD, &tm_v, bar, row);
        }
        if (second) {
          const int row = (p1 * n_kv + sg.kvh) << p.shift;
          tma_rows(st + 16 * HD, &tm_k, bar, row);
          tma_rows(st + 48 * HD, &tm_v, bar, row);
        }
      }
      ++issued;
    }
  };
  auto start = [&]() {
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      const int r = g + 8 * h;
      const __nv_bfloat16* row = q_base + (static_cast<int64_t>(sg.req) * a.slots + p.slot0 + r / p.group) * a.q_row_stride +
                                 (sg.kvh * p.group + r % p.group) * a.q_head_stride + t * (HD / 4);
#pragma unroll
      for (int s = 0; s < kKSteps; ++s)  // channels in the order that K's pieces give
        qw[h][s] = r < p.rows ? __ldg(reinterpret_cast<const uint2*>(row + (s >> 2) * 16 + (s & 3) * 4)) : make_uint2(0, 0);
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
  };
  {
    const int u = cut.begin(piece), total = row_of.total();
    sg.kvh = u / total;
    row_of.find(u - sg.kvh * total, sg.req, sg.first);
    sg.first += sg.kvh * total;
    place(u);
    __syncthreads();  // (the sums of lengths have been read)
    start();
  }

  for (;;) {
    // --- the new tokens' own keys, with the (request, head)'s first tile: 16 of them a step, the warps in turn.
    // The same products in bf16, as Q and they come; P as the sum of two bf16 (16 bits).  Part of the warp's share:
    // m, l and O wait in the join's place.
    const bool with_fresh = sg.begin == 0 && a.k_new;
    if (with_fresh) {
      float fo[RH][kKSteps][4], fm[RH][2], fl[RH][2];
      const int64_t row0 = static_cast<int64_t>(sg.req) * a.slots;
      const uint8_t* mask[RH][2];
      int slot[RH][2];  // of rows 8 h + 2t and 2t + 1; -1: no such row
#pragma unroll
      for (int h = 0; h < RH; ++h) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 8 * h + 2 * t + k;
          slot[h][k] = r < p.rows ? p.slot0 + r / p.group : -1;
          mask[h][k] = a.mask + (row0 + slot[h][k]) * a.slots;
          fm[h][k] = -INFINITY;
          fl[h][k] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kKSteps; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) fo[h][j][k] = 0.0f;
      }
      for (int k0 = 16 * warp; k0 < a.slots; k0 += 16 * kDecodeWarps) {
        uint4 kw[2][HD / 32], vw[4][HD / 64];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int b = k0 + g + 8 * x;
          const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k_new) + (row0 + b) * a.k_row_stride + sg.kvh * a.k_head_stride + t * (HD / 4);
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) kw[x][c] = b < a.slots ? __ldg(reinterpret_cast<const uint4*>(kp) + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int b = k0 + 2 * t + (x & 1) + 8 * (x >> 1);
          const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v_new) + (row0 + b) * a.v_row_stride + sg.kvh * a.v_head_stride + g * (HD / 8);
#pragma unroll
          for (int c = 0; c < HD / 64; ++c) vw[x][c] = b < a.slots ? __ldg(reinterpret_cast<const uint4*>(vp) + c) : make_uint4(0, 0, 0, 0);
        }
        uint32_t see = 0;  // bit 4 h + 2 x + k: row 8 h + 2t + k sees key k0 + g + 8 x
#pragma unroll
        for (int h = 0; h < RH; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int b = k0 + g + 8 * x;
              if (slot[h][k] >= 0 && b < a.slots && (a.mask ? __ldg(mask[h][k] + b) != 0 : b <= slot[h][k])) see |= 1u << (4 * h + 2 * x + k);
            }
        // values that are not finite: they take no part in the product, and O becomes NaN in the rows that see them
        uint32_t bad = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          bool odd = false;
#pragma unroll
          for (int c = 0; c < HD / 64; ++c) {
            const uint32_t y[4] = {vw[x][c].x, vw[x][c].y, vw[x][c].z, vw[x][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= (y[i] & 0x7F80u) == 0x7F80u || (y[i] & 0x7F800000u) == 0x7F800000u;
          }
          if (odd) bad |= 1u << (2 * t + (x & 1) + 8 * (x >> 1));
        }
        bad = __reduce_or_sync(0xFFFFFFFFu, bad);
        if (bad) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (bad >> (2 * t + (x & 1) + 8 * (x >> 1)) & 1u) {
#pragma unroll
              for (int c = 0; c < HD / 64; ++c) vw[x][c] = make_uint4(0, 0, 0, 0);
            }
        }
        uint32_t ph[RH][2], pl[RH][2];
#pragma unroll
        for (int h = 0; h < RH; ++h) {
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            mma_bf16(s, kw[0][c].x, kw[1][c].x, kw[0][c].y, kw[1][c].y, qw[h][2 * c].x, qw[h][2 * c].y);
            mma_bf16(s, kw[0][c].z, kw[1][c].z, kw[0][c].w, kw[1][c].w, qw[h][2 * c + 1].x, qw[h][2 * c + 1].y);
          }
          float e[4], f[2];
          bool odd[2];  // the row sees a value that is not finite
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool s0 = see >> (4 * h + k) & 1u, s1 = see >> (4 * h + 2 + k) & 1u;
            const float z0 = s0 ? s[k] * (a.scale * 1.4426950408889634f) : -INFINITY;
            const float z1 = s1 ? s[k + 2] * (a.scale * 1.4426950408889634f) : -INFINITY;
            float top = fmaxf(fm[h][k], fmaxf(z0, z1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            const float base = top == -INFINITY ? 0.0f : top;
            f[k] = ex2(fm[h][k] - base);
            fm[h][k] = top;
            e[k] = s0 ? ex2(z0 - base) : 0.0f;
            e[k + 2] = s1 ? ex2(z1 - base) : 0.0f;
            fl[h][k] = fl[h][k] * f[k] + (e[k] + e[k + 2]);
            // (a row's keys are in the lanes of its t)
            odd[k] = (__ballot_sync(0xFFFFFFFFu, (s0 && bad >> g & 1u) || (s1 && bad >> (g + 8) & 1u)) & 0x11111111u << t) != 0;
          }
#pragma unroll
          for (int j = 0; j < kKSteps; ++j) {
            fo[h][j][0] *= f[0], fo[h][j][1] *= f[1];
            fo[h][j][2] *= f[0], fo[h][j][3] *= f[1];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (odd[k & 1]) fo[h][j][k] = NAN;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const __nv_bfloat162 hi = __floats2bfloat162_rn(e[2 * x], e[2 * x + 1]);
            const __nv_bfloat162 lo = __floats2bfloat162_rn(e[2 * x] - __low2float(hi), e[2 * x + 1] - __high2float(hi));
            ph[h][x] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
            pl[h][x] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
          }
        }
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = i == 0 ? vw[x][c].x : i == 1 ? vw[x][c].y : i == 2 ? vw[x][c].z : vw[x][c].w;
            const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
            const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
            for (int h = 0; h < RH; ++h) {
              mma_bf16(fo[h][4 * c + i], a0, a1, a2, a3, ph[h][0], ph[h][1]);
              mma_bf16(fo[h][4 * c + i], a0, a1, a2, a3, pl[h][0], pl[h][1]);
            }
          }
      }
#pragma unroll
      for (int h = 0; h < RH; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = warp * kRows + 8 * h + 2 * t + k;
          float sum = fl[h][k];
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
          if (g == 0) s_m[r] = fm[h][k], s_l[r] = sum;
#pragma unroll
          for (int j = 0; j < kKSteps; ++j)
            *reinterpret_cast<float2*>(s_o + r * HD + g * (HD / 8) + 2 * j) = make_float2(fo[h][j][k], fo[h][j][k + 2]);
        }
      __syncwarp();
    }

    // --- Q fragments: rows g and g + 8
    uint32_t qf[RH][kKSteps][2];
    float c_row[RH][2];  // scale * log2(e) * the row's power of two, of rows 8 h + 2t and 2t + 1
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      float amax = 0.0f;
#pragma unroll
      for (int s = 0; s < kKSteps; ++s) {
        const uint32_t x[2] = {qw[h][s].x, qw[h][s].y};
#pragma unroll
        for (int k = 0; k < 2; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xFFFF0000u))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // q * 2^(14 - k) with 2^k <= amax < 2^(k+1): at most 2^15
      int k = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      k = min(max(k, -100), 127);
      const float up = __uint_as_float(static_cast<uint32_t>(14 - k + 127) << 23);
      const float c_own = a.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(k - 14 + 127) << 23);
      c_row[h][0] = __shfl_sync(0xFFFFFFFFu, c_own, 8 * t);
      c_row[h][1] = __shfl_sync(0xFFFFFFFFu, c_own, 8 * t + 4);
#pragma unroll
      for (int s = 0; s < kKSteps; ++s) {
        qf[h][s][0] = pack_f16(__uint_as_float(qw[h][s].x << 16) * up, __uint_as_float(qw[h][s].x & 0xFFFF0000u) * up);
        qf[h][s][1] = pack_f16(__uint_as_float(qw[h][s].y << 16) * up, __uint_as_float(qw[h][s].y & 0xFFFF0000u) * up);
      }
    }

    float o[RH][kKSteps][4];
    float m[RH][2], l[RH][2];  // of rows 8 h + 2t and 2t + 1; l: over this thread's keys
    float u[RH][2], u_high[RH][2];  // O is in units of 2^u; the largest u so far
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      m[h][0] = m[h][1] = -INFINITY;
      l[h][0] = l[h][1] = 0.0f;
      u[h][0] = u[h][1] = u_high[h][0] = u_high[h][1] = -INFINITY;
#pragma unroll
      for (int j = 0; j < kKSteps; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[h][j][k] = 0.0f;
    }

    for (int i = 0; i < steps; ++i) {
      if (!gave_up && !__all_sync(0xFFFFFFFFu, mbar_wait(&bars[used % kStages], (used / kStages) & 1, nullptr))) {
        gave_up = true;
        lost = used;
      }
      const uint8_t* st = ring + (used++ % kStages) * kDecodeWarps * Smem::kStep;
      __syncwarp();  // (every lane has read the step before this one: its place is free)
      issue(i + kStages - 1);
      const int set = (i >> 4) & 1;
      float s[2][RH][4], k_scale[2], v_scale[2];
      int valid[2];  // keys of this half that exist, if below 16
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        k_scale[x] = __shfl_sync(0xFFFFFFFFu, set ? ks[1] : ks[0], (i & 15) * 2 + x);
        v_scale[x] = __shfl_sync(0xFFFFFFFFu, set ? vs[1] : vs[0], (i & 15) * 2 + x);
        valid[x] = v_scale[x] < 0.0f ? 0 : sg.end - (tok0 + i * kDecodeTile + x * 16);
#pragma unroll
        for (int h = 0; h < RH; ++h) {
#pragma unroll
          for (int k = 0; k < 4; ++k) s[x][h][k] = 0.0f;
        }
      }
#pragma unroll
      for (int y = 0; y < kVec; ++y) {
        uint4 kf[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            kf[x][n] = *reinterpret_cast<const uint4*>(st + (16 * x + 8 * n) * HD + k_at[y]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4 k0 = kf[x][0], k1 = kf[x][1];
            uint32_t f[4];
            e4m3x4_to_f16x2x2(j == 0 ? k0.x : j == 1 ? k0.y : j == 2 ? k0.z : k0.w, f[0], f[2]);
            e4m3x4_to_f16x2x2(j == 0 ? k1.x : j == 1 ? k1.y : j == 2 ? k1.z : k1.w, f[1], f[3]);
#pragma unroll
            for (int h = 0; h < RH; ++h)
              mma_f16(s[x][h], f[0], f[1], f[2], f[3], qf[h][4 * y + j][0], qf[h][4 * y + j][1]);
          }
        }
      }
      // logits in powers of two: [half][key g, key g + 8] of rows 2t and 2t + 1; and the largest, without and with the
      // value scale's logarithm
      float z[RH][2][4], high[RH][2], high_weight[RH][2];
      const float v_log[2] = {lg2(v_scale[0]), lg2(v_scale[1])};
      bool moves = false;
#pragma unroll
      for (int h = 0; h < RH; ++h) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float c0 = c_row[h][0] * k_scale[x], c1 = c_row[h][1] * k_scale[x];
          z[h][x][0] = s[x][h][0] * c0, z[h][x][1] = s[x][h][1] * c1;
          z[h][x][2] = s[x][h][2] * c0, z[h][x][3] = s[x][h][3] * c1;
          if (valid[x] < 16) {
            if (g >= valid[x]) z[h][x][0] = z[h][x][1] = -INFINITY;
            if (g + 8 >= valid[x]) z[h][x][2] = z[h][x][3] = -INFINITY;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float high0 = fmaxf(z[h][0][k], z[h][0][k + 2]), high1 = fmaxf(z[h][1][k], z[h][1][k + 2]);
          high[h][k] = fmaxf(high0, high1);
          high_weight[h][k] = fmaxf(high0 + v_log[0], high1 + v_log[1]);  // (a NaN where a page is not there)
          // (a row's logits are in the lanes of its t)
          const bool small = (__ballot_sync(0xFFFFFFFFu, high_weight[h][k] >= u[h][k]) & 0x11111111u << t) == 0;
          moves |= high[h][k] > m[h][k] + 8.0f || high_weight[h][k] > u[h][k] + kUnitTop || (small && u[h][k] > u_high[h][k] - kUnitFall);
        }
      }
      // The maximum in use may lag behind the true one by 2^8, and O's unit moves only where a step's largest weight
      // leaves its range, so that O is rescaled a few times in a stretch and not at every step.
      if (__any_sync(0xFFFFFFFFu, moves)) {
#pragma unroll
        for (int h = 0; h < RH; ++h) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = fmaxf(high[h][k], m[h][k]), weight = high_weight[h][k];
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, y));
              weight = fmaxf(weight, __shfl_xor_sync(0xFFFFFFFFu, weight, y));
            }
            l[h][k] *= top == -INFINITY ? 1.0f : ex2(m[h][k] - top);
            m[h][k] = top;
            f[k] = move_unit(weight, top, u[h][k], u_high[h][k]);
          }
#pragma unroll
          for (int j = 0; j < kKSteps; ++j) {
            o[h][j][0] *= f[0], o[h][j][1] *= f[1];
            o[h][j][2] *= f[0], o[h][j][3] *= f[1];
          }
        }
      }
      uint32_t pb[RH][2][2];
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        const float b0 = m[h][0] == -INFINITY ? 0.0f : m[h][0], b1 = m[h][1] == -INFINITY ? 0.0f : m[h][1];
        const float unit0 = u[h][0] == -INFINITY ? 1.0f : ex2(m[h][0] - u[h][0]), unit1 = u[h][1] == -INFINITY ? 1.0f : ex2(m[h][1] - u[h][1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float f0 = v_scale[x] * unit0, f1 = v_scale[x] * unit1;
          const float e0 = ex2(z[h][x][0] - b0), e1 = ex2(z[h][x][1] - b1);
          const float e2 = ex2(z[h][x][2] - b0), e3 = ex2(z[h][x][3] - b1);
          l[h][0] += e0 + e2;
          l[h][1] += e1 + e3;
          pb[h][x][0] = transpose8x8(pack_f16(e0 * f0, e1 * f1));
          pb[h][x][1] = transpose8x8(pack_f16(e2 * f0, e3 * f1));
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t vf[4][HD / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* v = st + (32 + 16 * x + (r >> 1) * 8) * HD + v_at[r & 1];
          if (HD == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(v);
            vf[r][0] = y.x, vf[r][1] = y.y, vf[r][HD / 32 - 2] = y.z, vf[r][HD / 32 - 1] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(v);
            vf[r][0] = y.x, vf[r][1] = y.y;
          }
        }
        if (valid[x] < 16) {  // values behind the length may be NaN, and 0 * NaN is NaN
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (2 * t + (r & 1) + (r >> 1) * 8 >= valid[x]) {
#pragma unroll
              for (int w = 0; w < HD / 32; ++w) vf[r][w] = 0u;
            }
        }
#pragma unroll
        for (int w = 0; w < HD / 32; ++w) {
          const uint32_t x01 = __byte_perm(vf[0][w], vf[1][w], 0x5140), x23 = __byte_perm(vf[0][w], vf[1][w], 0x7362);
          const uint32_t y01 = __byte_perm(vf[2][w], vf[3][w], 0x5140), y23 = __byte_perm(vf[2][w], vf[3][w], 0x7362);
          uint32_t f[8];
          e4m3x4_to_f16x2x2(x01, f[0], f[1]);
          e4m3x4_to_f16x2x2(y01, f[2], f[3]);
          e4m3x4_to_f16x2x2(x23, f[4], f[5]);
          e4m3x4_to_f16x2x2(y23, f[6], f[7]);
#pragma unroll
          for (int h = 0; h < RH; ++h) {
            mma_f16(o[h][2 * w], f[0], f[1], f[2], f[3], pb[h][x][0], pb[h][x][1]);
            mma_f16(o[h][2 * w + 1], f[4], f[5], f[6], f[7], pb[h][x][0], pb[h][x][1]);
          }
        }
      }
    }
    // --- this warp's part, with that of the new tokens: sums over its keys, O in true units
    {
      float f_old[RH][2], f_fresh[RH][2];  // of O
#pragma unroll
      for (int h = 0; h < RH; ++h) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 8 * h + 2 * t + k, at = warp * kRows + r;
          float sum = l[h][k];
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
          const float fm = with_fresh ? s_m[at] : -INFINITY, fl = with_fresh ? s_l[at] : 0.0f;
          const float top = fmaxf(m[h][k], fm), base = top == -INFINITY ? 0.0f : top;
          f_old[h][k] = ex2(u[h][k] - base);
          f_fresh[h][k] = with_fresh ? ex2(fm - base) : 0.0f;
          l[h][k] = sum * ex2(m[h][k] - base) + fl * f_fresh[h][k];
          m[h][k] = top;
        }
#pragma unroll
        for (int j = 0; j < kKSteps; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = 8 * h + 2 * t + k;
            float2* x = reinterpret_cast<float2*>(s_o + (warp * kRows + r) * HD + g * (HD / 8) + 2 * j);
            float2 y = make_float2(o[h][j][k] * f_old[h][k], o[h][j][k + 2] * f_old[h][k]);
            if (with_fresh) {
              y.x += x->x * f_fresh[h][k];
              y.y += x->y * f_fresh[h][k];
            }
            *x = y;
          }
      }
      __syncwarp();  // (the new tokens' m and l have been read)
#pragma unroll
      for (int h = 0; h < RH; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (g == 0) {
            s_m[warp * kRows + 8 * h + 2 * t + k] = m[h][k];
            s_l[warp * kRows + 8 * h + 2 * t + k] = l[h][k];
          }
    }

    // --- the next segment's first loads, before this one is joined
    const DecodeSegment was = sg;
    const bool more = sg.stop < u_end;
    if (more) {
      const int u = sg.stop;
      sg.first += sg.tiles;
      if (++sg.req == a.n_req) sg.req = 0, ++sg.kvh;
      place(u);
      start();
    }
    __syncthreads();

    // --- join the warps' parts; four channels a thread
    const int c_first = cut.of(was.first), c_last = cut.of(was.first + was.tiles - 1);  // the pieces that share it
    const bool alone = c_first == c_last;
    auto finish = [&](int r, int c, float top, float sum, const float4& acc) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int64_t row = static_cast<int64_t>(was.req) * a.slots + p.slot0 + r / p.group;
      const int head = was.kvh * p.group + r % p.group;
      __nv_bfloat162 w[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv), __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * a.out_row_stride + head * a.out_head_stride + c) =
          *reinterpret_cast<uint2*>(w);
      if (a.lse && c == 0)
        a.lse[row * a.n_q + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    for (int i = tid; i < p.rows * kQuads; i += kDecodeThreads) {
      const int r = i / kQuads, c = (i % kQuads) * 4;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) top = fmaxf(top, s_m[w * kRows + r]);
      const float base = top == -INFINITY ? 0.0f : top;
      float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) {
        const float f = ex2(s_m[w * kRows + r] - base);
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kRows + r) * HD + c);
        sum += s_l[w * kRows + r] * f;
        acc.x += x.x * f, acc.y += x.y * f, acc.z += x.z * f, acc.w += x.w * f;
      }
      if (alone) {
        finish(r, c, top, sum, acc);
      } else {
        const size_t own = static_cast<size_t>(2 * piece + (piece == c_first)) * p.rows + r;
        __stcg(reinterpret_cast<float4*>(p.part + own * HD + c), acc);
        if (c == 0) __stcg(reinterpret_cast<float2*>(stats + own * 2), make_float2(top, sum));
      }
    }
    if (!alone) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        unsigned* done = p.done + static_cast<size_t>(was.req) * n_kv + was.kvh;
        s_last = atomicAdd(done, 1u) == static_cast<unsigned>(c_last - c_first);
        if (s_last) *done = 0u;  // ready for the next call
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        // parts in the order of tiles: the first piece's last one, then the first one of each that follows;
        // read in batches whose loads are in flight together
        constexpr int kBatch = 8;
        for (int i = tid; i < p.rows * kQuads; i += kDecodeThreads) {
          const int r = i / kQuads, c = (i % kQuads) * 4;
          float top = -INFINITY, sum = 0.0f;
          float4 acc = make_float4(0, 0, 0, 0);
          for (int x0 = c_first; x0 <= c_last; x0 += kBatch) {
            float2 ml[kBatch];
            float4 y[kBatch];
            float high = top;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int x = min(x0 + k, c_last);
              const size_t part = static_cast<size_t>(2 * x + (x == c_first)) * p.rows + r;
              ml[k] = __ldcg(reinterpret_cast<const float2*>(stats + part * 2));
              y[k] = __ldcg(reinterpret_cast<const float4*>(p.part + part * HD + c));
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) high = fmaxf(high, ml[k].x);
            const float base = high == -INFINITY ? 0.0f : high, f0 = ex2(top - base);
            sum *= f0;
            acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const float f = ex2(ml[k].x - base);
              if (x0 + k <= c_last) {
                sum += ml[k].y * f;
                acc.x += y[k].x * f, acc.y += y[k].y * f, acc.z += y[k].z * f, acc.w += y[k].w * f;
              }
            }
            top = high;
          }
          finish(r, c, top, sum, acc);
        }
      }
    }
    if (!more) break;
    __syncthreads();  // (the join has been read)
  }
  if (gave_up) {
    if (a.status) atomicOr(a.status, DT_KV_TIMEOUT);
    for (; lost < issued; ++lost) mbar_wait(&bars[lost % kStages], (lost / kStages) & 1, nullptr);  // (no copy may outlive the CTA)
  }
  dt_grid_wait();
}

// Grid: one wave, and no more CTAs than tiles there can be (the host knows the longest possible request).
inline int decode_grid(int n_req, int n_kv, long long max_len) {
  const long long tiles = (max_len + kDecodeTile - 1) / kDecodeTile * n_req * n_kv;
  constexpr long long wave = static_cast<long long>(kSms) * kDecodeCtas;
  return static_cast<int>(tiles < wave ? (tiles < 1 ? 1 : tiles) : wave);
}
inline size_t decode_workspace(int rows, int head_dim) {
  const size_t parts = static_cast<size_t>(2 * kSms * kDecodeCtas) * rows * (head_dim + 2) * 4;
  return kCounterBytes + (parts + 255) / 256 * 256;
}

// beside: started when the kernel before it in the stream, the tree kernel of the same call, has left SMs free
// (they share neither counters nor parts).
template <int HD, int RH>
cudaError_t launch_decode(const CUtensorMap& k, const CUtensorMap& v, const DecodeParams& p, int grid, bool beside, cudaStream_t st) {
  constexpr int bytes = DecodeSmem<HD, RH>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k_decode<HD, RH>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_decode<HD, RH>, k, v, p);
}

}  // namespace dt
