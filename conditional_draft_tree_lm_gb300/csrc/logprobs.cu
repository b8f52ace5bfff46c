// dt_token_logprobs: log probabilities of given tokens, entropy and the best alternatives, in one pass over the logits.
//
// With c = log2(e) / T, every thread keeps m (a maximum, in use), s = sum 2^((x - m) c) and w = sum (x - m) c 2^((x - m) c)
// of the logits it has met; two such triples join by bringing the smaller maximum's to the larger's unit:
//   s' = f s,  w' = f (w + d s),  d = (m - M) c,  f = 2^d.
// At the row's end lse = M / T + ln2 log2 s, and the entropy is ln2 (log2 s - w / s); a log probability is
// (x - M) / T - ln2 log2 s.  Logits enter as differences to the maximum, taken before they are scaled: near 10^4 they
// lose nothing, and where a mask has put fp32's lowest value nothing overflows.  The maximum in use lags behind the
// true one by up to 2^8, so that sums are seldom rescaled.
//
// The best n_top: while the logits stream, a thread only notes the largest of each of up to 16 stretches of its own.  In
// every warp the q-th largest of its threads' largest, q = ceil(n_top / warps), and the smallest of that over the warps,
// is a bound that n_top logits reach, and few more do, since the best mostly lie with different threads; the stretches
// that reach it are read again.  Each warp collects the keys of its own in a list, which is cut to its best where it
// runs full, and raises the bound.  Keys are (value, lower token), all different, so that neither the order of arrival nor
// the bounds' timing changes the result.
//
// A row is read by a cluster of 1 to 16 CTAs, which join over distributed shared memory: no workspace, one launch.  Every
// thread copies its logits to shared memory ahead of their use (cp.async), and reads no other thread's, so that the stream
// has no barrier.
#include "cluster.cuh"
#include "kv_flash.cuh"
#include "select.cuh"

namespace dt {
namespace {

constexpr int kVecs = 4;  // pieces of 16 bytes of a thread's round
constexpr int kStretches = 16;
constexpr int kMaxTop = 64, kMaxSplit = 16;
// Rounds in shared memory, and its bytes: with the stretches' largest in it, two rounds leave room for four CTAs an SM.
constexpr int rounds_ahead(bool best) { return best ? 2 : 3; }
constexpr int logp_smem(bool best, int threads) { return rounds_ahead(best) * kVecs * threads * 16 + (best ? kStretches * threads * 4 : 0); }
constexpr float kLag = 8.0f;

struct LogpParams {
  dt_token_logprobs_args a;
  int split, chunk;  // CTAs of a row, logits of each
  float c;
};

struct Sums {
  float m, s, w;
};
// (m is a raw logit, -inf for none)
// The sums of `width` lanes (a power of two), all of them in every lane.
DT_DEVINL Sums join_lanes(const Sums& x, int width, float c) {
  Sums all = x;
  for (int o = width / 2; o > 0; o >>= 1) all.m = fmaxf(all.m, __shfl_xor_sync(0xFFFFFFFFu, all.m, o));
  const float d = x.m == -INFINITY ? 0.0f : (x.m - all.m) * c, f = ex2(d);
  // (far below the maximum: a part of nothing, where d s would be infinite)
  all.s = x.s * f;
  all.w = f * fmaf(fmaxf(d, -1e4f), x.s, x.w);
  for (int o = width / 2; o > 0; o >>= 1) {
    all.s += __shfl_xor_sync(0xFFFFFFFFu, all.s, o);
    all.w += __shfl_xor_sync(0xFFFFFFFFu, all.w, o);
  }
  return all;
}

// The `top` largest of keys[0, n) (different keys, in shared memory), in order to out.  All threads call, with a barrier
// before; out must not overlap the keys.
DT_DEVINL void rank_keys(const uint64_t* keys, int n, int top, uint64_t* out) {
  block_rank_all(keys, n, [&](int, uint64_t key, int rank) {
    if (rank < top) out[rank] = key;
  });
}

DT_DEVINL void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// PER: keys of a lane when a warp's list is full, 32 PER in all (0: no best tokens are asked for).  Rows that a CTA reads
// alone may take 64 threads (see the choice below).
template <bool BF16, int PER, int kLogpThreads>
__global__ void __launch_bounds__(kLogpThreads, 1024 / kLogpThreads) k_logp(const LogpParams p) {
  constexpr int kLogpWarps = kLogpThreads / 32, kMostSplit = kLogpThreads == 64 ? 1 : kMaxSplit;
  constexpr int kElems = BF16 ? 8 : 4, kBytes = BF16 ? 2 : 4, kCap = 32 * (PER ? PER : 1);
  constexpr int kKeys = kLogpWarps * kCap > kMostSplit * kMaxTop ? kLogpWarps * kCap : kMostSplit * kMaxTop;
  constexpr int kAhead = rounds_ahead(PER > 0), kRingBytes = kAhead * kVecs * kLogpThreads * 16;
  // the ring of rounds; behind the stream, the warps' lists, what is ranked of them and of the CTAs, and the stretches to read
  // again; then 64 bytes of each thread, its stretches' largest
  extern __shared__ __align__(16) uint8_t ring[];
  static_assert((kLogpWarps * kCap + kKeys) * 8 + kLogpThreads * kStretches * 2 <= kRingBytes, "");
  uint64_t* lists = reinterpret_cast<uint64_t*>(ring);
  uint64_t* keys = lists + kLogpWarps * kCap;
  uint16_t* again = reinterpret_cast<uint16_t*>(keys + kKeys) + (threadIdx.x >> 5) * 32 * kStretches;
  uint4* own = reinterpret_cast<uint4*>(ring + kRingBytes) + (threadIdx.x >> 5) * 128 + (threadIdx.x & 31);  // [4][lane] of a warp
  auto stretch_max = [&](int i) -> float& { return reinterpret_cast<float*>(own + (i >> 2) * 32)[i & 3]; };
  __shared__ uint64_t s_best[PER ? kMaxTop : 1], s_out[PER ? kMaxTop : 1];
  __shared__ uint32_t s_bound[kLogpWarps];
  __shared__ int s_n[2];
  __shared__ Sums s_warp[kLogpWarps], s_sums;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / p.split;
  const int part = static_cast<int>(blockIdx.x - row * p.split);
  const int vocab = p.a.vocab, top = p.a.n_top;
  const int lo = min(vocab, part * p.chunk), hi = min(vocab, lo + p.chunk);
  const char* x = static_cast<const char*>(p.a.logits) + row * p.a.logits_row_stride * kBytes;
  auto load = [&](int i) -> float {
    return BF16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(x)[i]) : reinterpret_cast<const float*>(x)[i];
  };
  // the part's logits: `head` up to a 16-byte boundary, `vecs` pieces of 16 bytes, the rest
  const int to_edge = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(x) + static_cast<int64_t>(lo) * kBytes) % 16u) % 16u) / kBytes;
  const int head = min(hi - lo, to_edge), vecs = (hi - lo - head) / kElems;
  const int first = lo + head, behind = first + vecs * kElems, tail = hi - behind;
  const uint4* vec = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(first) * kBytes);
  auto unpack = [](const uint4& piece, float* v) {
    const uint32_t r[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
      } else {
        v[i] = __uint_as_float(r[i]);
      }
    }
  };

  // round k of a thread: pieces tid + 256 (4 k + u), u < 4
  constexpr int kRound = kVecs * kLogpThreads;
  uint4* mine = reinterpret_cast<uint4*>(ring) + tid;
  auto fetch = [&](int at, int slot) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      if (at + u * kLogpThreads < vecs) copy16(mine + slot * kRound + u * kLogpThreads, vec + at + u * kLogpThreads);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  dt_grid_wait();
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(tid + k * kRound, k);
  // the first given token of a thread, while the logits are on their way
  const int token = part == 0 && tid < p.a.n_tokens ? p.a.tokens[row * p.a.n_tokens + tid] : -1;
  const float asked = token >= 0 && token < vocab ? load(token) : NAN;

  const float c = p.c;
  Sums sum = {-INFINITY, 0.0f, 0.0f};
  float m = 0.0f;  // sum.m, 0 while there is no maximum
  // the sums over `count` logits of a thread, the largest of which is `most`
  auto add = [&](const float* v, int count, float most) {
    if ((most - m) * c > kLag || (sum.m == -INFINITY && most > -INFINITY)) {
      const float d = sum.m == -INFINITY ? 0.0f : (m - most) * c, f = ex2(d);
      sum.w = f * fmaf(fmaxf(d, -1e4f), sum.s, sum.w);
      sum.s *= f;
      sum.m = m = most;
    }
    const uint64_t m2 = f32x2(-m, -m), c2 = f32x2(c, c);
    uint64_t e2 = 0, w2 = 0;
#pragma unroll
    for (int i = 0; i < count; i += 2) {
      float d0, d1;
      f32x2_parts(mul2(add2(f32x2(v[i], v[i + 1]), m2), c2), d0, d1);
      const uint64_t e = f32x2(ex2(d0), ex2(d1));
      e2 = add2(e2, e);
      w2 = fma2(f32x2(fmaxf(d0, -1e4f), fmaxf(d1, -1e4f)), e, w2);  // (a logit of -inf: 0, not -inf * 0)
    }
    float lo2, hi2;
    f32x2_parts(e2, lo2, hi2);
    sum.s += lo2 + hi2;
    f32x2_parts(w2, lo2, hi2);
    sum.w += lo2 + hi2;
  };

  // rounds of a stretch; the largest logit of the present one
  const int stretch = (vecs + kStretches * kRound - 1) / (kStretches * kRound);
  float largest = -INFINITY;
  int slot = 0, left = stretch, stretches = 0;
  for (int at = tid; at < vecs; at += kRound) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t none = BF16 ? 0xFF80FF80u : 0xFF800000u;
      const uint4 piece = at + u * kLogpThreads < vecs ? mine[slot * kRound + u * kLogpThreads] : make_uint4(none, none, none, none);
      float v[kElems];
      unpack(piece, v);
      float most = v[0];
#pragma unroll
      for (int i = 1; i < kElems; ++i) most = fmaxf(most, v[i]);
      add(v, kElems, most);
      if (PER) largest = fmaxf(largest, most);
    }
    fetch(at + kAhead * kRound, slot);
    slot = slot + 1 == kAhead ? 0 : slot + 1;
    if (PER && (--left == 0 || at + kRound >= vecs)) {
      stretch_max(stretches++) = largest;
      largest = -INFINITY;
      left = stretch;
    }
  }
  for (int i = stretches; PER && i < kStretches; ++i) stretch_max(i) = -INFINITY;
  float edge[2] = {-INFINITY, -INFINITY};  // what stands around the pieces of 16 bytes, with warp 0
  if (warp == 0) {
    if (lane < head) edge[0] = load(lo + lane);
    if (lane < tail) edge[1] = load(behind + lane);
    add(edge, 2, fmaxf(edge[0], edge[1]));
  }

  sum = join_lanes(sum, 32, c);
  if (lane == 0) s_warp[warp] = sum;
  if (PER) {
#pragma unroll
    for (int i = 0; i < kStretches; ++i) largest = fmaxf(largest, stretch_max(i));
    const int quota = (top + kLogpWarps - 1) / kLogpWarps;
    uint32_t rest = f32_key(largest), q = 0;
    for (int i = 0; i < quota; ++i) {
      q = __reduce_max_sync(0xFFFFFFFFu, rest);
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, rest == q);
      if (lane == __ffs(who) - 1) rest = 0;
    }
    if (lane == 0) s_bound[warp] = q;
    if (tid == 0) s_n[0] = s_n[1] = 0;
    if (tid < kMaxTop) s_best[tid] = 0;
    static_assert(kMaxTop <= 64, "");
  }
  __syncthreads();  // (and the ring has been read)
  if (warp == 0) {
    sum = join_lanes(s_warp[lane % kLogpWarps], kLogpWarps, c);
    if (lane == 0) s_sums = sum;
  }
  if (PER) {
    uint32_t q = s_bound[0];
#pragma unroll
    for (int i = 1; i < kLogpWarps; ++i) q = min(q, s_bound[i]);
    // below every key of that value (-inf, which threads without logits have too, bounds nothing)
    uint64_t tau = q > f32_key(-INFINITY) ? static_cast<uint64_t>(q) << 32 : 0;
    const float least = tau ? key_f32(q) : -INFINITY;
    uint64_t* list = lists + warp * kCap;
    int n = 0;  // keys in the warp's list
    // the list down to its best, in order
    auto cut = [&]() {
      uint64_t key[PER ? PER : 1];
      int rank[PER ? PER : 1];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        key[i] = lane + 32 * i < n ? list[lane + 32 * i] : 0;
        rank[i] = 0;
      }
#pragma unroll 4
      for (int e = 0; e < n; ++e) {
        const uint64_t k = list[e];
#pragma unroll
        for (int i = 0; i < PER; ++i) rank[i] += k > key[i] ? 1 : 0;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane + 32 * i < n && rank[i] < top) list[rank[i]] = key[i];
      __syncwarp();
      n = min(n, top);
      if (n == top) tau = max(tau, list[top - 1]);
    };
    auto take = [&](const float* v, uint32_t mask, int index) {  // the logits of `mask` of every lane, from token `index` on
      while (__any_sync(0xFFFFFFFFu, mask != 0)) {
        const int bit = __ffs(mask) - 1;
        float y = v[0];
#pragma unroll
        for (int i = 1; i < kElems; ++i) y = bit == i ? v[i] : y;
        const uint64_t key = mask ? rank_key(y + 0.0f, static_cast<uint32_t>(index + bit)) : 0;  // (-0 counts as 0)
        mask &= mask - 1;
        const bool in = key > tau;
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
        if (in) list[n + __popc(who & ((1u << lane) - 1u))] = key;
        n += __popc(who);
        if (n > kCap - 32) cut();
      }
    };
    // the stretches that reach the bound, four at a time, a piece to a lane
    int n_again = 0;
    uint32_t reach = 0;
#pragma unroll
    for (int i = 0; i < kStretches; ++i) reach |= (stretch_max(i) >= least && stretch_max(i) > -INFINITY ? 1u : 0u) << i;
    reach &= (1u << stretches) - 1u;
    while (__any_sync(0xFFFFFFFFu, reach != 0)) {
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, reach != 0);
      if (reach) again[n_again + __popc(who & ((1u << lane) - 1u))] = static_cast<uint16_t>((__ffs(reach) - 1) * 32 + lane);
      reach &= reach - 1;
      n_again += __popc(who);
    }
    __syncwarp();
    // (a list that has been cut has raised the bound: of equal logits later stretches have nothing then)
    const float* largest_of = reinterpret_cast<const float*>(ring + kRingBytes) + warp * 512;
    auto value_of = [](uint64_t key) { return key ? key_f32(static_cast<uint32_t>(key >> 32)) : -INFINITY; };
    for (int s = 0; s < n_again; s += 4) {
      int begin[4];  // the stretch's first piece, -1 where it cannot reach the bound
      bool any = false;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int which = s + u < n_again ? again[s + u] : -1, i = which >> 5, owner = which & 31;
        begin[u] = -1;
        if (which < 0) continue;
        const int at = warp * 32 + owner + i * stretch * kRound;
        if (rank_key(largest_of[(i >> 2) * 128 + owner * 4 + (i & 3)] + 0.0f, static_cast<uint32_t>(first + at * kElems)) > tau) begin[u] = at, any = true;
      }
      if (!any) continue;
      for (int from = lane; from - lane < stretch * kVecs; from += 32) {
        int here[4];
        uint4 piece[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          here[u] = begin[u] + from * kLogpThreads;
          if (begin[u] < 0 || from >= stretch * kVecs || here[u] >= vecs) here[u] = -1;
          piece[u] = here[u] < 0 ? make_uint4(0, 0, 0, 0) : vec[here[u]];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (begin[u] < 0) continue;
          const float now = value_of(tau);
          float v[kElems];
          unpack(piece[u], v);
          uint32_t mask = 0;
#pragma unroll
          for (int i = 0; i < kElems; ++i) mask |= (v[i] >= now && v[i] > -INFINITY ? 1u : 0u) << i;
          take(v, here[u] < 0 ? 0u : mask, first + here[u] * kElems);
        }
      }
    }
    // where a mask leaves fewer logits than are asked for: the first of -inf, piece after piece
    for (int at = warp * 32; n < top && tau == 0 && at < vecs; at += kLogpThreads) {
      const bool there = at + lane < vecs;
      float v[kElems];
      unpack(there ? vec[at + lane] : make_uint4(0, 0, 0, 0), v);
      uint32_t mask = 0;
#pragma unroll
      for (int i = 0; i < kElems; ++i) mask |= (v[i] == -INFINITY ? 1u : 0u) << i;
      take(v, there ? mask : 0u, first + (at + lane) * kElems);
    }
    if (warp == 0) {
      float v[kElems] = {edge[0]};
      take(v, lane < head && edge[0] >= least ? 1u : 0u, lo + lane);
      v[0] = edge[1];
      take(v, lane < tail && edge[1] >= least ? 1u : 0u, behind + lane);
    }
    __syncwarp();
    int base = 0;
    if (lane == 0) base = atomicAdd(&s_n[0], n);
    base = __shfl_sync(0xFFFFFFFFu, base, 0);
    for (int e = lane; e < n; e += 32) keys[base + e] = list[e];
    __syncthreads();
    rank_keys(keys, s_n[0], top, s_best);
  }
  __syncthreads();
  const uint64_t* best = s_best;
  Sums all = s_sums;
  if (kMostSplit > 1 && p.split > 1) {
    cluster_barrier();
    if (part == 0) {
      if (warp == 0) {
        const uint32_t at = peer_addr(&s_sums, lane % p.split);
        sum = join_lanes({peer_ld(at), peer_ld(at + 4), peer_ld(at + 8)}, p.split, c);
        if (lane == 0) s_warp[0] = sum;
      }
      if (PER) {
        // likewise of the row
        constexpr int kMine = kMaxSplit * kMaxTop / kLogpThreads;
        uint64_t key[kMine];
        uint32_t rest = 0, q = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int e = tid + i * kLogpThreads, r = e / top;
          key[i] = r < p.split ? peer_ld_u64(peer_addr(&s_best[e - r * top], r)) : 0;
          rest = max(rest, static_cast<uint32_t>(key[i] >> 32));
        }
        // (of the warps whose lanes all have a key)
        const int warps = max(1, min(kLogpWarps, p.split * top / 32)), quota = (top + warps - 1) / warps;
        for (int i = 0; i < quota; ++i) {
          q = __reduce_max_sync(0xFFFFFFFFu, rest);
          const uint32_t who = __ballot_sync(0xFFFFFFFFu, rest == q);
          if (lane == __ffs(who) - 1) rest = 0;
        }
        if (lane == 0) s_bound[warp] = q;
        __syncthreads();
        q = s_bound[0];
        for (int i = 1; i < warps; ++i) q = min(q, s_bound[i]);
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (key[i] && key[i] >> 32 >= q) keys[atomicAdd(&s_n[1], 1)] = key[i];
      }
    }
    cluster_barrier();  // (no CTA leaves while its memory is read)
    if (part != 0) return;
    all = s_warp[0];
    if (PER) {
      if (tid < kMaxTop) s_out[tid] = 0;
      __syncthreads();
      rank_keys(keys, s_n[1], top, s_out);
      best = s_out;
      __syncthreads();
    }
  }

  const float top_logit = all.m == -INFINITY ? 0.0f : all.m;
  const bool broken = all.s != all.s, nothing = all.s == 0.0f;
  const float log2s = broken ? NAN : log2f(all.s);
  auto logp = [&](float v) { return nothing ? -INFINITY : (v - top_logit) / p.a.temperature - log2s * 0.693147180559945f; };
  if (tid == 0) {
    if (p.a.lse) p.a.lse[row] = nothing ? -INFINITY : top_logit / p.a.temperature + log2s * 0.693147180559945f;
    if (p.a.entropy) p.a.entropy[row] = nothing ? 0.0f : broken ? NAN : fmaxf((log2s - all.w / all.s) * 0.693147180559945f, 0.0f);
  }
  for (int j = tid; j < p.a.n_tokens; j += kLogpThreads) {
    const int t = j == tid ? token : p.a.tokens[row * p.a.n_tokens + j];
    if (t >= vocab && p.a.status) atomicOr(p.a.status, DT_KV_BAD_INDEX);
    p.a.logp[row * p.a.n_tokens + j] = t < 0 ? 0.0f : t >= vocab ? NAN : logp(j == tid ? asked : load(t));
  }
  if (PER)
    for (int j = tid; j < top; j += kLogpThreads) {
      const uint64_t k = broken ? 0 : best[j];
      p.a.top_tok[row * top + j] = k ? static_cast<int>(rank_key_id(k)) : -1;
      p.a.top_logp[row * top + j] = k ? logp(key_f32(static_cast<uint32_t>(k >> 32))) : NAN;
    }
}

template <bool BF16, int PER, int THREADS>
cudaError_t launch(const LogpParams& p, cudaStream_t st) {
  const auto kernel = k_logp<BF16, PER, THREADS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_a_device(done, [&] {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, logp_smem(PER > 0, THREADS));
    return e == cudaSuccess && THREADS > 64 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : e;
  });
  if (e != cudaSuccess) return e;
  return launch_behind(kernel, static_cast<unsigned>(p.a.rows * p.split), THREADS, logp_smem(PER > 0, THREADS), st, p.split, p);
}
template <bool BF16, int PER>
cudaError_t launch(const LogpParams& p, cudaStream_t st) {
  // 64 threads: short rows, and where rows fill all places and their ends, of which there are more side by side then, count.
  // us by 256 and 64 threads: 4000 rows of 8192, 5 best 70 and 39, of 32768 111 and 100; 2000 of 65536 102 and 98; 8192 of 151936 in
  // bf16 468 and 414, without best 380 and 396; but 2080 of 151936 212 and 223; 320 of 32768 17 and 22.
  const int64_t bytes = static_cast<int64_t>(p.a.vocab) * (BF16 ? 2 : 4);
  const bool small = p.split == 1 && (bytes <= 8192 || (p.a.rows >= 12 * kSms && bytes <= (PER ? 320 : 32) * 1024));
  return small ? launch<BF16, PER, 64>(p, st) : launch<BF16, PER, 256>(p, st);
}

}  // namespace
}  // namespace dt

extern "C" dt_status dt_token_logprobs(const dt_token_logprobs_args* args, void* stream) {
  using namespace dt;
  const char* who = "dt_token_logprobs";
  if (!args) return kv_fail(DT_ERR_INVALID_ARG, "%s: null arguments", who);
  const dt_token_logprobs_args& a = *args;
  if (a.rows < 0 || a.rows > (1 << 26)) return kv_fail(DT_ERR_SHAPE, "%s: rows outside 0..2^26", who);
  if (a.vocab < 1 || a.vocab > (1 << 30)) return kv_fail(DT_ERR_SHAPE, "%s: vocab outside 1..2^30", who);
  if (a.n_tokens < 0 || a.n_tokens > 65536) return kv_fail(DT_ERR_SHAPE, "%s: n_tokens outside 0..65536", who);
  if (a.n_top < 0 || a.n_top > kMaxTop || a.n_top > a.vocab)
    return kv_fail(DT_ERR_SHAPE, "%s: n_top %d outside 0..%d or above vocab", who, a.n_top, kMaxTop);
  if (!(a.temperature >= 0x1p-100f) || a.temperature - a.temperature != 0.0f)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: temperature is not finite or below 2^-100", who);
  if (a.rows == 0) return DT_OK;
  if (!a.logits || (reinterpret_cast<uintptr_t>(a.logits) & (a.logits_bf16 ? 1u : 3u)) != 0)
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null or misaligned logits", who);
  if ((a.n_tokens && (!a.tokens || !a.logp)) || (a.n_top && (!a.top_tok || !a.top_logp)))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: null tokens, logp, top_tok or top_logp", who);
  if (!kv_aligned(4, a.tokens, a.logp, a.lse, a.entropy, a.top_tok, a.top_logp, a.status))
    return kv_fail(DT_ERR_INVALID_ARG, "%s: misaligned tokens, logp, lse, entropy, top_tok, top_logp or status", who);
  const int64_t item = a.logits_bf16 ? 2 : 4;
  auto flat = [](const void* d, int64_t count) { return MemoryRows{reinterpret_cast<uintptr_t>(d), 1, 0, 4 * count}; };
  const MemoryRows read[2] = {{reinterpret_cast<uintptr_t>(a.logits), a.rows, a.logits_row_stride * item, a.vocab * item}, flat(a.tokens, a.rows * a.n_tokens)};
  const MemoryRows written[6] = {flat(a.logp, a.rows * a.n_tokens), flat(a.lse, a.rows), flat(a.entropy, a.rows), flat(a.top_tok, a.rows * a.n_top),
                                 flat(a.top_logp, a.rows * a.n_top), flat(a.status, 1)};
  for (int i = 0; i < 6; ++i) {
    if (!written[i].at || !written[i].width) continue;
    bool meets = rows_meet(written[i], read[0]) || (a.n_tokens && rows_meet(written[i], read[1]));
    for (int j = 0; j < i; ++j) meets = meets || (written[j].at && written[j].width && rows_meet(written[i], written[j]));
    if (meets) return kv_fail(DT_ERR_INVALID_ARG, "%s: an output overlaps logits, tokens or another output", who);
  }
  LogpParams p = {};
  p.a = a;
  p.c = static_cast<float>(1.4426950408889634 / a.temperature);
  // Few rows are split: over two CTAs an SM at most, each with 2048 logits or more; clusters of 16 only while all of them
  // stand beside each other (16 rows of 151936, 20 best: 15.6 us, 14.0 by 8; one row 11.1 and 11.2; 65 rows by 4 17.8, 8 19.0,
  // 2 19.7; 130 rows by 2 23.7, 1 26.4, 4 26.7).
  p.split = 1;
  const int widest = a.rows <= 6 ? kMaxSplit : 8;
  while (p.split < widest && a.rows * p.split * 2 <= 2 * kSms && a.vocab / (2 * p.split) >= 2048) p.split *= 2;
  p.chunk = ((a.vocab + p.split - 1) / p.split + 63) & ~63;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.logits_bf16) e = a.n_top == 0 ? launch<true, 0>(p, st) : a.n_top <= 32 ? launch<true, 2>(p, st) : launch<true, 4>(p, st);
  else e = a.n_top == 0 ? launch<false, 0>(p, st) : a.n_top <= 32 ? launch<false, 2>(p, st) : launch<false, 4>(p, st);
  return kv_launched(who, e);
}
