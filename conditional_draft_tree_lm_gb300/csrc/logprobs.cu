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
// The best n_top: every warp has a list of its own and takes in what passes the best bound known in the CTA, so that the
// stream needs no barrier between warps.  The first bound comes from the first logits: the q-th largest of a warp's lane
// maxima, q = ceil(n_top / warps), smallest over the warps, is reached by n_top logits or more.  Full lists are cut to
// their n_top best by ranks, and raise the bound.  Keys are (value, lower token), all different, so that neither the
// order of arrival nor the bounds' timing changes the result.
//
// A row is read by a cluster of 1 to 16 CTAs, which join over distributed shared memory: no workspace, one launch.
#include "cluster.cuh"
#include "kv.cuh"

namespace dt {
namespace {

constexpr int kLogpThreads = 256, kLogpWarps = kLogpThreads / 32;
constexpr int kVecs = 4;             // 16-byte loads of a thread in flight
constexpr int kMaxTop = 64, kMaxSplit = 16;
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
DT_DEVINL Sums join(const Sums& x, const Sums& y, float c) {
  const float m = fmaxf(x.m, y.m);
  const float dx = x.m == -INFINITY ? 0.0f : (x.m - m) * c, dy = y.m == -INFINITY ? 0.0f : (y.m - m) * c;
  const float fx = ex2(dx), fy = ex2(dy);
  // (far below the other: a part of nothing, where d s would be infinite)
  return {m, x.s * fx + y.s * fy, fx * fmaf(fmaxf(dx, -1e4f), x.s, x.w) + fy * fmaf(fmaxf(dy, -1e4f), y.s, y.w)};
}

// Of `lists` lists in descending order, list l's n[l] keys at at(l, i): the `top` largest keys to out, in order.  All
// threads call; out must not overlap the lists.  Returns their number.
template <class At>
DT_DEVINL int merge_lists(int lists, const int* n, int top, At at, uint64_t* out) {
  int total = 0;
  for (int l = 0; l < lists; ++l) total += n[l];
  for (int e = threadIdx.x; e < lists * top; e += kLogpThreads) {
    const int l = e / top, i = e - l * top;
    if (i >= n[l]) continue;
    const uint64_t key = at(l, i);
    int rank = i;
    for (int o = 0; o < lists; ++o) {
      if (o == l) continue;
      int lo = 0, hi = n[o];  // the first of list o that is below key
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (at(o, mid) > key) lo = mid + 1;
        else hi = mid;
      }
      rank += lo;
    }
    if (rank < top) out[rank] = key;
  }
  return min(total, top);
}

// PER: keys of a lane when a warp's list is full, 32 PER in all (0: no best tokens are asked for).
template <bool BF16, int PER>
__global__ void __launch_bounds__(kLogpThreads, 4) k_logp(const LogpParams p) {
  constexpr int kElems = BF16 ? 8 : 4, kCap = 32 * (PER ? PER : 1);
  __shared__ uint64_t s_list[PER ? kLogpWarps : 1][kCap];
  __shared__ uint64_t s_best[PER ? kMaxTop : 1], s_all[PER ? kMaxSplit * kMaxTop : 1], s_out[PER ? kMaxTop : 1];
  __shared__ unsigned long long s_tau;
  __shared__ uint32_t s_bound[kLogpWarps];
  __shared__ int s_n[kLogpWarps], s_nbest, s_nall[kMaxSplit];
  __shared__ float s_sums[4];
  __shared__ Sums s_warp[kLogpWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / p.split;
  const int part = static_cast<int>(blockIdx.x - row * p.split);
  const int vocab = p.a.vocab, top = p.a.n_top;
  const int lo = min(vocab, part * p.chunk), hi = min(vocab, lo + p.chunk);
  const char* x = static_cast<const char*>(p.a.logits) + row * p.a.logits_row_stride * (BF16 ? 2 : 4);
  auto load = [&](int i) -> float {
    return BF16 ? bf16_to_f32(__ldg(reinterpret_cast<const uint16_t*>(x) + i)) : __ldg(reinterpret_cast<const float*>(x) + i);
  };
  // the part's logits: `head` up to a 16-byte boundary, `vecs` pieces of 16 bytes, the rest
  const int to_edge = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(x) + static_cast<int64_t>(lo) * (BF16 ? 2 : 4)) % 16u) % 16u) / (BF16 ? 2 : 4);
  const int head = min(hi - lo, to_edge), vecs = (hi - lo - head) / kElems;
  const int first = lo + head, behind = first + vecs * kElems, tail = hi - behind;
  const uint4* vec = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(first) * (BF16 ? 2 : 4));

  const float c = p.c;
  Sums sum = {-INFINITY, 0.0f, 0.0f};
  float m = 0.0f;      // sum.m, 0 while there is no maximum
  int n = 0;           // keys in the warp's list
  uint64_t tau = 0;
  if (PER && tid == 0) s_tau = 0;

  // the warp's list down to its `top` best, in order
  auto cut = [&]() {
    uint64_t* list = s_list[PER ? warp : 0];
    uint64_t key[PER ? PER : 1];
    int rank[PER ? PER : 1];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      key[i] = lane + 32 * i < n ? list[lane + 32 * i] : 0;
      rank[i] = 0;
    }
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
    if (n == top) {
      tau = max(tau, list[top - 1]);
      if (lane == 0) atomicMax(&s_tau, static_cast<unsigned long long>(tau));
    }
  };
  // takes the logits of `mask` (of this lane, whose index is index(bit)) into the list; the whole warp calls
  auto take = [&](uint32_t mask, auto index) {
    while (__any_sync(0xFFFFFFFFu, mask != 0)) {
      uint64_t key = 0;
      if (mask) {
        const int i = index(__ffs(mask) - 1);
        mask &= mask - 1;
        key = rank_key(load(i) + 0.0f, static_cast<uint32_t>(i));  // (-0 counts as 0)
      }
      const bool in = key > tau;
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
      if (in) s_list[PER ? warp : 0][n + __popc(who & ((1u << lane) - 1u))] = key;
      n += __popc(who);
      if (n > kCap - 32) cut();
    }
  };
  auto bound = [&]() {  // the value below which nothing of this row is among the best
    tau = max(tau, static_cast<uint64_t>(*reinterpret_cast<volatile unsigned long long*>(&s_tau)));
    return tau ? key_f32(static_cast<uint32_t>(tau >> 32)) : -INFINITY;
  };
  // the sums over N logits of a thread, the largest of which is `most`
  auto add = [&](const float* v, int count, float most) {
    if ((most - m) * c > kLag || (sum.m == -INFINITY && most > -INFINITY)) {
      const float d = sum.m == -INFINITY ? 0.0f : (m - most) * c, f = ex2(d);
      sum.w = f * fmaf(fmaxf(d, -1e4f), sum.s, sum.w);
      sum.s *= f;
      sum.m = m = most;
    }
#pragma unroll
    for (int i = 0; i < count; ++i) {
      const float d = (v[i] - m) * c, e = ex2(d);
      sum.s += e;
      sum.w = fmaf(fmaxf(d, -1e4f), e, sum.w);  // (a logit of -inf: 0, not -inf * 0)
    }
  };

  for (int at = tid, round = 0; round == 0 || at - tid < vecs; at += kVecs * kLogpThreads, ++round) {
    uint4 raw[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t none = BF16 ? 0xFF80FF80u : 0xFF800000u;
      raw[u] = at + u * kLogpThreads < vecs ? __ldcs(vec + at + u * kLogpThreads) : make_uint4(none, none, none, none);
    }
    float most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t r[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      float v[kElems];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (BF16) {
          v[2 * i] = __uint_as_float(r[i] << 16);
          v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        } else {
          v[i] = __uint_as_float(r[i]);
        }
      }
      float mine = v[0];
#pragma unroll
      for (int i = 1; i < kElems; ++i) mine = fmaxf(mine, v[i]);
      add(v, kElems, mine);
      most = fmaxf(most, mine);
    }
    if (PER) {
      if (round == 0) {
        const int quota = (top + kLogpWarps - 1) / kLogpWarps;
        uint32_t mine = f32_key(most), q = 0;
        for (int i = 0; i < quota; ++i) {
          q = __reduce_max_sync(0xFFFFFFFFu, mine);
          const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine == q);
          if (lane == __ffs(who) - 1) mine = 0;
        }
        if (lane == 0) s_bound[warp] = q;
        __syncthreads();
        q = s_bound[0];
#pragma unroll
        for (int i = 1; i < kLogpWarps; ++i) q = min(q, s_bound[i]);
        // (below every key of that value; -inf, which absent logits have too, bounds nothing)
        tau = q > f32_key(-INFINITY) ? static_cast<uint64_t>(q) << 32 : 0;
      }
      const float least = bound();
      if (__any_sync(0xFFFFFFFFu, most >= least)) {
#pragma unroll 1
        for (int u = 0; u < kVecs; ++u) {
          const int here = at + u * kLogpThreads;
          uint32_t mask = 0;
          if (here < vecs && most >= least) {
            for (int i = 0; i < kElems; ++i) mask |= (load(first + here * kElems + i) >= least ? 1u : 0u) << i;
          }
          take(mask, [&](int i) { return first + here * kElems + i; });
        }
      }
    }
  }
  if (warp == 0) {  // what stands around the pieces of 16 bytes
    float v[2] = {lane < head ? load(lo + lane) : -INFINITY, lane < tail ? load(behind + lane) : -INFINITY};
    add(v, 2, fmaxf(v[0], v[1]));
    if (PER) {
      const float least = bound();
      take((lane < head && v[0] >= least ? 1u : 0u) | (lane < tail && v[1] >= least ? 2u : 0u),
           [&](int i) { return i ? behind + lane : lo + lane; });
    }
  }

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums y = {__shfl_xor_sync(0xFFFFFFFFu, sum.m, o), __shfl_xor_sync(0xFFFFFFFFu, sum.s, o), __shfl_xor_sync(0xFFFFFFFFu, sum.w, o)};
    sum = lane & o ? join(y, sum, c) : join(sum, y, c);
  }
  if (lane == 0) s_warp[warp] = sum;
  if (PER) {
    cut();
    if (lane == 0) s_n[warp] = n;
  }
  __syncthreads();
  Sums all = s_warp[0];
#pragma unroll
  for (int i = 1; i < kLogpWarps; ++i) all = join(all, s_warp[i], c);
  if (tid == 0) {
    s_sums[0] = all.m;
    s_sums[1] = all.s;
    s_sums[2] = all.w;
  }
  if (PER) {
    const int k = merge_lists(kLogpWarps, s_n, top, [&](int l, int i) { return s_list[PER ? l : 0][i]; }, s_best);
    if (tid == 0) s_nbest = k;
  }
  const uint64_t* best = s_best;
  int n_best = 0;
  if (p.split > 1) {
    cluster_barrier();
    if (part == 0) {
      all = {peer_ld(peer_addr(&s_sums[0], 0)), peer_ld(peer_addr(&s_sums[1], 0)), peer_ld(peer_addr(&s_sums[2], 0))};
      for (int r = 1; r < p.split; ++r) {
        const uint32_t at = peer_addr(s_sums, r);
        all = join(all, {peer_ld(at), peer_ld(at + 4), peer_ld(at + 8)}, c);
      }
      if (PER) {
        if (tid < p.split) s_nall[tid] = __float_as_int(peer_ld(peer_addr(&s_nbest, tid)));
        for (int e = tid; e < p.split * top; e += kLogpThreads) s_all[e] = peer_ld_u64(peer_addr(s_best, e / top) + (e % top) * 8);
      }
    }
    cluster_barrier();  // (no CTA leaves while its memory is read)
    if (part != 0) return;
    if (PER) {
      n_best = merge_lists(p.split, s_nall, top, [&](int l, int i) { return s_all[l * top + i]; }, s_out);
      best = s_out;
      __syncthreads();
    }
  } else if (PER) {
    __syncthreads();
    n_best = s_nbest;
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
    const int t = p.a.tokens[row * p.a.n_tokens + j];
    if (t >= vocab && p.a.status) atomicOr(p.a.status, DT_KV_BAD_INDEX);
    p.a.logp[row * p.a.n_tokens + j] = t < 0 ? 0.0f : t >= vocab ? NAN : logp(load(t));
  }
  if (PER)
    for (int j = tid; j < top; j += kLogpThreads) {
      const bool there = !broken && j < n_best;
      const uint64_t k = there ? best[j] : 0;
      p.a.top_tok[row * top + j] = there ? static_cast<int>(rank_key_id(k)) : -1;
      p.a.top_logp[row * top + j] = there ? logp(key_f32(static_cast<uint32_t>(k >> 32))) : NAN;
    }
}

template <bool BF16, int PER>
cudaError_t launch(const LogpParams& p, cudaStream_t st) {
  if (p.split > 8) {
    cudaError_t e = cudaFuncSetAttribute(k_logp<BF16, PER>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.a.rows * p.split));
  cfg.blockDim = dim3(kLogpThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_logp<BF16, PER>, p);
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
  LogpParams p = {};
  p.a = a;
  p.c = static_cast<float>(1.4426950408889634 / a.temperature);
  // Few rows are split: as many CTAs as two a SM, each with 2048 logits or more.
  p.split = 1;
  while (p.split < kMaxSplit && a.rows * p.split < 2 * kSms && a.vocab / (2 * p.split) >= 2048) p.split *= 2;
  p.chunk = ((a.vocab + p.split - 1) / p.split + 63) & ~63;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.logits_bf16) e = a.n_top == 0 ? launch<true, 0>(p, st) : a.n_top <= 32 ? launch<true, 2>(p, st) : launch<true, 4>(p, st);
  else e = a.n_top == 0 ? launch<false, 0>(p, st) : a.n_top <= 32 ? launch<false, 2>(p, st) : launch<false, 4>(p, st);
  return kv_launched(who, e);
}
