// dt_cache_attention: arguments, workspace and the choice of kernel.
//
// Up to 16 rows (new tokens x heads of a group) per key/value head the cache is
// streamed through mma.m16n8k16 (kv_decode.cuh), whose time does not depend on the
// rows there; above, 128-row tiles on tcgen05 (kv_tree.cuh).  What is left over
// behind pairs of full row tiles, as with a root and 64 drafted tokens of 4 heads a
// group, would cost as much there as a pair: up to 16 such rows go to the streaming
// kernel, launched beside the other, where there are enough heads and requests.
#include "kv_decode.cuh"
#include "kv_tree.cuh"

namespace dt {

// Rows or tokens by which a kernel's counts may pass the last one: 16 steps of 128 tokens, a tile more, and room.
constexpr int kAhead = 4095;

// Row tiles of a call with more than 16 rows per key/value head: pairs, the odd one, and
// the first slot of those left to the streaming kernel (0: none).  It takes them where
// the odd tile holds 16 rows at most, there are 8 key/value heads over all requests, for its
// pieces, and 32 pairs over all of them, which the odd tiles would keep from the SMs.  us without and
// with it (8 key/value heads of 128, 4 heads a group, where nothing else is said):
//   65 slots, 32 requests of up to 4k tokens 307 and 209, of up to 512 129 and 97; 8 requests of 4k 102 and 77; 4 of 4k 61 and
//     55, of 512 36 and 38; but 2 of 4k 52 and 75, 1 of 32k 114 and 138; head_dim 64: 32 requests 228 and 134, 4 39 and 30
//   129 slots, 32 requests of 4k 454 and 346; 2 of 32k 168 and 151; but 1 of 4k 49 and 53, of 32k 126 and 127
//   257 slots, 1 request of 2k 58 and 50, of 32k 183 and 187; 513 slots, 1 of 32k 336 and 311, of 2k 72 and 74
//   34 slots of 8 heads a group, 32 requests 309 and 220, 4 63 and 62; 1 of 8k 70 and 108
//   513 slots over 2 key/value heads, 2 requests of 16k 88 and 101; 65 slots over 1, 32 requests of 4k 66 and 60
struct RowTiles {
  int pairs, odd, rest;
  RowTiles(int n_req, int slots, int group, int n_kv) {
    const int per_tile = 128 / group, tiles = (slots + per_tile - 1) / per_tile;
    pairs = tiles / 2;
    odd = tiles % 2;
    const int first = (tiles - 1) * per_tile;
    const int64_t heads = static_cast<int64_t>(n_req) * n_kv;
    rest = odd && pairs > 0 && (slots - first) * group <= kDecodeMaxRows && heads >= 8 && heads * pairs >= 32 ? first : 0;
  }
};

}  // namespace dt

extern "C" size_t dt_cache_attention_workspace(int n_req, int slots, int n_q, int n_kv, int head_dim) {
  if (n_req < 1 || slots < 1 || slots > 0x7FFFFFFF - dt::kAhead || n_kv < 1 || n_q < n_kv || n_q % n_kv != 0 || (head_dim != 64 && head_dim != 128)) return 0;
  if (static_cast<int64_t>(slots) * (n_q / n_kv) <= dt::kDecodeMaxRows) return dt::decode_workspace(slots * (n_q / n_kv), head_dim);
  if (n_q / n_kv > 128) return 0;
  const dt::RowTiles tiles(n_req, slots, n_q / n_kv, n_kv);
  return dt::tree_workspace(head_dim) + (tiles.rest ? dt::decode_workspace(dt::kDecodeMaxRows, head_dim) : 0);
}

extern "C" dt_status dt_cache_attention(const dt_kv_cache* cache, const dt_cache_attention_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_cache_attention";
  if (dt_status s = kv_check_cache(who, cache)) return s;
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  const dt_cache_attention_args& a = *args;
  if (a.n_req < 1 || a.slots < 1 || a.n_q < 1 || a.max_blocks < 1)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: need n_req, slots, n_q, max_blocks >= 1", who);
  if (a.n_q % cache->n_kv != 0 || a.n_q / cache->n_kv > 128)
    return kv_fail(DT_ERR_SHAPE, "%s: %d query heads over %d key/value heads: need a multiple, at most 128 a head", who,
                   a.n_q, cache->n_kv);
  // (positions are counted some tiles ahead, in 32 bits)
  if (static_cast<int64_t>(a.n_req) * a.slots > 0x7FFFFFFF - kAhead || static_cast<int64_t>(a.max_blocks) * cache->page > 0x7FFFFFFF - kAhead)
    return kv_fail(DT_ERR_SHAPE, "%s: more than 2^31-%d rows or tokens", who, kAhead + 1);
  if (!(a.scale - a.scale == 0.0f)) return kv_fail(DT_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (!a.block_table || !a.length || !kv_rows_ok(a.q, a.q_row_stride, a.q_head_stride) ||
      !kv_rows_ok(a.out, a.out_row_stride, a.out_head_stride))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null or misaligned q, out, block_table or length", who);
  if (!kv_rows_apart(static_cast<int64_t>(a.n_req) * a.slots, a.n_q, cache->head_dim, a.out_row_stride, a.out_head_stride))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: rows of out overlap", who);
  if ((a.k_new != nullptr) != (a.v_new != nullptr) ||
      (a.k_new && (!kv_rows_ok(a.k_new, a.k_row_stride, a.k_head_stride) || !kv_rows_ok(a.v_new, a.v_row_stride, a.v_head_stride))))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: k_new and v_new: one is null or misaligned", who);
  if (a.mask && !a.k_new) return kv_fail(DT_ERR_INVALID_ARG, "%s: a mask without new keys", who);
  const size_t need = dt_cache_attention_workspace(a.n_req, a.slots, a.n_q, cache->n_kv, cache->head_dim);
  if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u) != 0 || a.workspace_bytes < need)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: the workspace is null, misaligned or below %zu bytes", who, need);
  if (static_cast<int64_t>(a.n_req) * cache->n_kv > kMaxJoins)
    return kv_fail(DT_ERR_SHAPE, "%s: n_req * n_kv above %d", who, kMaxJoins);
  if ((static_cast<int64_t>(a.max_blocks) * cache->page / kDecodeTile + 1) * a.n_req * cache->n_kv > (1 << 30))
    return kv_fail(DT_ERR_SHAPE, "%s: more than 2^37 cached tokens over all requests and heads", who);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int group = a.n_q / cache->n_kv;
  const dt::RowTiles rows(a.n_req, a.slots, group, cache->n_kv);
  int shift = 4;
  while ((1 << shift) < cache->page) ++shift;
  unsigned* done = static_cast<unsigned*>(a.workspace);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kCounterBytes);
  // key rows of the whole cache, as the streaming kernel's copies count them: ((page * n_kv) + head) * page_size + offset
  const int64_t key_rows = static_cast<int64_t>(cache->n_pages) * cache->n_kv * cache->page;
  auto decode = [&](int slot0) -> dt_status {  // the slots from slot0 on
    DecodeParams p = {};
    p.c = *cache;
    p.a = a;
    p.group = group;
    p.slot0 = slot0;
    p.rows = (a.slots - slot0) * group;
    p.shift = shift;
    p.done = slot0 ? done + a.n_req * cache->n_kv * rows.pairs : done;  // (behind what the tree kernel uses)
    p.part = slot0 ? part + (tree_workspace(cache->head_dim) - kCounterBytes) / 4 : part;
    const int grid = decode_grid(a.n_req, cache->n_kv, static_cast<long long>(a.max_blocks) * cache->page);
    p.box = cache->page < 32 ? 16 : 32;
    CUtensorMap k, v;
    if (!kv_tmap_rows(&k, cache->k, cache->head_dim, key_rows, p.box) ||
        !kv_tmap_rows(&v, cache->v, cache->head_dim, key_rows, p.box))
      return kv_fail(DT_ERR_SHAPE, "%s: no tensor map for this cache", who);
    cudaError_t e;
    if (cache->head_dim == 64) e = p.rows <= 8 ? launch_decode<64, 1>(k, v, p, grid, slot0 > 0, st) : launch_decode<64, 2>(k, v, p, grid, slot0 > 0, st);
    else e = p.rows <= 8 ? launch_decode<128, 1>(k, v, p, grid, slot0 > 0, st) : launch_decode<128, 2>(k, v, p, grid, slot0 > 0, st);
    return kv_launched(who, e);
  };
  if (static_cast<int64_t>(a.slots) * group <= kDecodeMaxRows) {
    if (key_rows > 0x7FFFFFFF) return kv_fail(DT_ERR_SHAPE, "%s: more than 2^31-1 cached tokens and heads", who);
    return decode(0);
  }
  TreeParams p = {};
  p.c = *cache;
  p.a = a;
  p.group = group;
  p.shift = shift;
  p.per_tile = 128 / group;
  p.inverse = group_inverse(group);
  const bool stream_rest = rows.rest > 0 && key_rows <= 0x7FFFFFFF;
  p.pairs = rows.pairs;
  p.odd = stream_rest ? 0 : rows.odd;
  p.fresh_tiles = a.k_new ? (a.slots + kKeyTile - 1) / kKeyTile : 0;
  const int64_t key_tiles = (static_cast<int64_t>(a.max_blocks) * cache->page + kKeyTile - 1) / kKeyTile + p.fresh_tiles * kNewCost + 1;
  const int64_t units = key_tiles * (p.pairs + p.odd) * a.n_req * cache->n_kv;
  if (units > (1 << 30)) return kv_fail(DT_ERR_SHAPE, "%s: more than 2^30 tiles over all requests and heads", who);
  if (static_cast<int64_t>(a.n_req) * cache->n_kv * (rows.pairs + rows.odd) > kMaxJoins)
    return kv_fail(DT_ERR_SHAPE, "%s: n_req * n_kv * pairs of row tiles above %d", who, kMaxJoins);
  p.done = done;
  p.part = part;
  const int grid = tree_grid(units);
  if (dt_status s = kv_launched(who, cache->head_dim == 64 ? launch_tree<64>(p, grid, st) : launch_tree<128>(p, grid, st))) return s;
  return stream_rest ? decode(rows.rest) : DT_OK;
}
