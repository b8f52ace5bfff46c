// What the two tensor-core attention kernels share: tensor-memory accesses, the
// products' issue, and the softmax of one 128-key tile.
//
// Both keep S = Q K^T (128 rows x 128 keys, fp32) and O (128 rows x head_dim) in
// tensor memory, one lane a row.  A softmax thread owns a row: it reads its 128
// logits, writes P as 16-bit pairs over S's columns, and the next product takes P
// from there (A from tensor memory) and V from shared memory as it was stored, rows
// of channels (B, MN-major), so that V is never transposed.
// Two such tiles of rows share every key tile: while one's softmax runs on the
// ordinary cores, the tensor core does the other's products.
//
// Order of one row tile's products (one issuing thread, and the tensor core runs
// them in order): S(0); then for every key tile j, when P(j) is there: O += P(j)
// V(j), S(j + 1).  So S(j + 1) being complete tells the softmax that O is at rest
// and may be rescaled, and P(j)'s place free.
//
// The maximum in use lags behind the true one by up to 2^8: a row's sum (and with it
// the prompts' O) is rescaled only where its maximum has grown by more; sums and O
// stay exact in that unit.
#pragma once

#include "kv.cuh"

namespace dt {

constexpr int kKeyTile = 128;
// Shared memory of a CTA, and what of it a kernel's static variables may take (with their alignment).
constexpr uint32_t kSmemBytes = 227 * 1024, kStaticBytes = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 32 lanes x 32 consecutive 32-bit columns, without waiting (tmem_wait_ld).
DT_DEVINL void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// A bounded wait by a whole warp, which goes on or gives up together.
DT_DEVINL bool warp_wait(uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, nullptr)); }

DT_DEVINL void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// (after the wait: ties the registers to it, so that nothing that uses them moves before it)
DT_DEVINL void tmem_landed32(uint32_t* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7]));
}
DT_DEVINL void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
DT_DEVINL void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
DT_DEVINL void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
DT_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem], kind::f16
DT_DEVINL void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Operand descriptors in the 128-byte swizzle, to which a byte offset inside the
// operand is added as off >> 4.  Rows of 64 channels, K-major (Q, K): groups of 8
// rows 1024 bytes apart.  V as operand B, MN-major: groups of 64 channels (128
// bytes a key) kHalfBytes apart, groups of 8 keys 1024 bytes apart.
constexpr uint32_t kHalfBytes = 128 * 128;
DT_DEVINL uint64_t flash_desc(uint32_t saddr, bool mn) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (mn ? static_cast<uint64_t>(kHalfBytes >> 4) << 16 : 0ull) |
         static_cast<uint64_t>(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// One lane of a converged warp.
DT_DEVINL bool elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}

// What P is: the probabilities in bf16 (prompts); probabilities times their keys' value scales, in fp16 and the row's
// unit (cached tokens); or the same as the sum of two bf16 (new tokens), see softmax_tile.
enum { kProbs, kWeights, kWeightPairs };

// kind::f16 with fp32 D; operands in bf16 or both in fp16; b_mn: B is MN-major.
DT_HOST_DEVICE_INLINE uint32_t idesc_flash(bool bf16, uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// A row tile's (or key tile's) operand in shared memory: halves of 64 channels, 128 rows of 128 bytes, swizzled.
template <int HD>
constexpr uint32_t kOperandBytes = HD / 64 * kHalfBytes;

// S = Q K^T and O (+)= P V of one tile; issued by one lane, with operands that the
// whole warp has computed (so that they stand in uniform registers: with one lane
// walking the tiles by itself the issue, not the tensor core, was the bound).
template <int HD>
DT_DEVINL void issue_qk(bool bf16, uint32_t s_tmem, uint64_t q, uint64_t k) {
  const uint32_t idesc = idesc_flash(bf16, 128, kKeyTile, false);
#pragma unroll
  for (int i = 0; i < HD / 16; ++i) {
    const uint32_t off = ((i >> 2) * kHalfBytes + (i & 3) * 32) >> 4;
    tc_mma_bf16(s_tmem, q + off, k + off, idesc, i != 0);
  }
}
template <int HD>  // half 0 or 1 of the keys; p: what P is
DT_DEVINL void issue_pv(int p, uint32_t o_tmem, uint32_t p_tmem, uint64_t v, bool first, int half) {
  const uint32_t idesc = idesc_flash(p != kWeights, 128, HD, true);
#pragma unroll
  for (int k = 0; k < kKeyTile / 32; ++k) {
    const int i = half * (kKeyTile / 32) + k;
    const uint32_t at = p_tmem + (p == kWeightPairs ? (i >> 1) * 32 + (i & 1) * 8 : i * 8);
    tc_mma_ts(o_tmem, at, v + (i * 2048 >> 4), idesc, !(first && i == 0));
    if (p == kWeightPairs) tc_mma_ts(o_tmem, at + 16, v + (i * 2048 >> 4), idesc, 1u);
  }
}

// Two numbers to a pair of bf16, the first in the low half.
DT_DEVINL uint32_t pack_p(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// O *= f for this warp's 32 lanes.
template <int HD>
DT_DEVINL void rescale_o(uint32_t o_tmem, float f) {
#pragma unroll
  for (int c = 0; c < HD; c += 32) {
    uint32_t v[32];
    tmem_ld32(o_tmem + c, v);
    tmem_wait_ld();
    tmem_landed32(v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
    tmem_st32(o_tmem + c, v);
  }
  tmem_wait_st();
}

// The first `n` of 128 keys, as four words of 32 bits.
DT_DEVINL uint32_t first_bits(int n, int word) {
  n -= word * 32;
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Two fp32 at a time (one issue slot for a pair).
DT_DEVINL uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
DT_DEVINL void f32x2_parts(uint64_t x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
DT_DEVINL uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
DT_DEVINL uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
DT_DEVINL uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A warp's 32 rows x 64 channels of bf16, one row a lane (w: 8 pieces of 16 bytes),
// to global memory through 4 KB of the warp's own shared memory: eight lanes write
// a row's 128 bytes together, where a lane writing its own row would touch 32 lines
// an instruction.  row_of(r): where the lane r's row goes, null for nowhere.
template <class RowOf>
DT_DEVINL void store_rows(uint8_t* mine, const uint4 (&w)[8], RowOf row_of) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // (the last rows have been read)
#pragma unroll
  for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(mine + lane * 128 + ((k ^ (lane & 7)) << 4)) = w[k];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3), k = lane & 7;
    __nv_bfloat16* to = row_of(r);
    if (to) *reinterpret_cast<uint4*>(to + 8 * k) = *reinterpret_cast<const uint4*>(mine + r * 128 + ((k ^ (r & 7)) << 4));
  }
}

// y / group for y < 128, group <= 128: y * inverse >> 16 with inverse = ceil(2^16 / group).
inline uint32_t group_inverse(int group) { return (65536u + group - 1) / group; }
DT_DEVINL int over_group(int y, uint32_t inverse) { return static_cast<int>(static_cast<uint32_t>(y) * inverse >> 16); }

// The running softmax of one row.
struct SoftmaxRow {
  float m = -INFINITY, l = 0.0f;  // the maximum in use, in powers of two, and the sum in its unit
  // kWeights, kWeightPairs: O is in units of 2^u, whatever m is; the largest u so far
  float u = -INFINITY, u_high = -INFINITY;
};
// New tokens come in where u >= m + kUnitNew: the largest of their values stay finite in O.
constexpr float kUnitNew = 16.0f;

// One 128-key tile of a row: S at s_at becomes P there, and the row's state (and O, where its unit changes: for
// kProbs with m) is brought up to date.  scale(g): what turns a raw logit of keys 16 g .. 16 g + 15 into
// powers of two; value(g), value_log(g): those keys' value scale and its logarithm (kWeights).  All three are asked for
// two g at a time, by g / 2.  NEGATIVE: the scale is (as code of its own: beside the other's it cost 65 of 440 us in the
// tree kernel, whose queries take the sign instead, and 11 of 278 for 48 prompts').  see: the row's visible keys, all of them unless MASKED.  ready(i):
// called when half i of P is stored.
// kWeightPairs: a weight goes to the product as the sum of two bf16 (its first 8 bits, cut off, and the rest
// rounded: 2^-16 relative), since a new token's values come in bf16, which fp16 cannot hold beside each other.  The
// pair stands in the 32 columns that its keys' logits leave, first parts before rests.
// S is read twice, 32 columns ahead of their use, and both loops are rolled up: with
// several roles' code running at once, instruction fetches count (S in 128 registers
// between the maximum and the exponentials, loops unrolled: 48 prompts of up to 1k
// tokens 300 us instead of 272, 16k tokens 1380 instead of 1367).  One body for
// masked tiles and others costs more than it saves there: 288 and 1650 us.
template <int HD, int P, bool MASKED, bool NEGATIVE, class Scale, class Value, class ValueLog, class Ready>
DT_DEVINL void softmax_tile(uint32_t s_at, uint32_t o_at, bool first, Scale scale, Value value, ValueLog value_log,
                            const uint32_t (&see)[4], SoftmaxRow& row, Ready ready) {
  constexpr bool SPLIT = P == kWeightPairs;
  uint32_t s[64];
  tmem_ld32(s_at, s);
  float top = -INFINITY, top_weight = -INFINITY;
#pragma unroll 1
  for (int w2 = 0; w2 < 4; w2 += 2)
#pragma unroll
  for (int w1 = 0; w1 < 2; ++w1) {
    const int w = w2 + w1;
    uint32_t* v = s + 32 * w1;
    tmem_wait_ld();
    tmem_landed32(v);
    tmem_ld32(s_at + 32 * ((w + 1) & 3), s + 32 * (w1 ^ 1));  // (the last one: the first, for the second reading)
    const float2 scale2 = scale(w), log2v = P == kWeights ? value_log(w) : make_float2(0.0f, 0.0f);
    if (MASKED) {
      const uint32_t out = NEGATIVE ? 0x7F800000u : 0xFF800000u;
      const uint32_t bits = w1 == 0 ? (w2 == 0 ? see[0] : see[2]) : (w2 == 0 ? see[1] : see[3]);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = bits >> i & 1u ? v[i] : out;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float a = __uint_as_float(v[16 * h]), b = __uint_as_float(v[16 * h + 1]);
      if (!NEGATIVE) {
#pragma unroll
        for (int i = 2; i < 16; i += 4) {
          a = fmaxf(fmaxf(a, __uint_as_float(v[16 * h + i])), __uint_as_float(v[16 * h + i + 1]));
          if (i + 2 < 16) b = fmaxf(fmaxf(b, __uint_as_float(v[16 * h + i + 2])), __uint_as_float(v[16 * h + i + 3]));
        }
        a = fmaxf(a, b);
      } else {
#pragma unroll
        for (int i = 2; i < 16; ++i) a = fminf(a, __uint_as_float(v[16 * h + i]));
        a = fminf(a, b);
      }
      // (the maximum passes over a NaN, as an unseen -inf times a scale of zero is)
      const float c = h ? scale2.y : scale2.x;
      top = fmaxf(top, a * c);
      if (P == kWeights) top_weight = fmaxf(top_weight, fmaf(a, c, h ? log2v.y : log2v.x));
    }
  }
  // (a tile of which the row sees nothing has top = -inf: no harm, P is 0)
  bool moves = top > row.m + 8.0f;
  if (P == kWeights)
    moves |= top_weight > row.u + kUnitTop ||
             (top_weight < row.u && top_weight > -INFINITY && fmaxf(top_weight - kUnitSet, row.u_high - kUnitFall) < row.u);
  if (P == kWeightPairs) moves |= row.u < row.m + kUnitNew;
  if (__any_sync(0xFFFFFFFFu, moves)) {
    const float m2 = fmaxf(row.m, top), f = m2 == -INFINITY ? 1.0f : ex2(row.m - m2);
    row.l *= f;
    row.m = m2;
    float f_o = f;
    bool o_moves = true;
    if (P != kProbs) {
      const float before = row.u;
      if (P == kWeights) {
        f_o = move_unit(top_weight, m2, row.u, row.u_high);
      } else {
        row.u = fmaxf(before, m2 + kUnitNew);
        f_o = row.u == before ? 1.0f : ex2(before - row.u);
      }
      o_moves = __any_sync(0xFFFFFFFFu, row.u != before);
    }
    tmem_wait_ld();  // (s is on its way; the rescaling waits for its own)
    if (!first && o_moves) rescale_o<HD>(o_at, f_o);
  }
  const float unit = P == kProbs || row.u == -INFINITY ? 1.0f : ex2(row.m - row.u);
  const float base = row.m == -INFINITY ? 0.0f : row.m;
  const uint64_t base2 = f32x2(-base, -base);
  uint64_t sum[2] = {0, 0};
#pragma unroll 1
  for (int w2 = 0; w2 < 4; w2 += 2)
#pragma unroll
  for (int w1 = 0; w1 < 2; ++w1) {
    const int w = w2 + w1;
    uint32_t pk[16];
    uint32_t* v = s + 32 * w1;
    const uint32_t p_at = s_at + (SPLIT ? 32 : 16) * w;
    tmem_wait_ld();
    tmem_landed32(v);
    if (w1 == 0 || w2 == 0) tmem_ld32(s_at + 32 * (w + 1), s + 32 * (w1 ^ 1));
    const uint32_t bits = w1 == 0 ? (w2 == 0 ? see[0] : see[2]) : (w2 == 0 ? see[1] : see[3]);
    // (of a masked tile, most 32-key parts are seen by all of a warp's rows or by none)
    const bool none = MASKED && __all_sync(0xFFFFFFFFu, bits == 0u);
    const bool all = !MASKED || __all_sync(0xFFFFFFFFu, bits == 0xFFFFFFFFu);
    if (none) {
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = 0u;
      if (SPLIT) tmem_st16(p_at + 16, pk);
    } else {
      const float2 scale2 = scale(w);
      float2 f2 = P == kWeights ? value(w) : make_float2(1.0f, 1.0f);
      f2.x *= unit, f2.y *= unit;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float c = i < 8 ? scale2.x : scale2.y, f = i < 8 ? f2.x : f2.y;
        float e0, e1;
        f32x2_parts(fma2(f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f32x2(c, c), base2), e0, e1);
        e0 = ex2(e0);
        e1 = ex2(e1);
        if (!all) {
          e0 = bits >> (2 * i) & 1u ? e0 : 0.0f;
          e1 = bits >> (2 * i + 1) & 1u ? e1 : 0.0f;
        }
        const uint64_t e = f32x2(e0, e1);
        sum[i & 1] = add2(sum[i & 1], e);
        if (P == kProbs) {
          pk[i] = pack_p(e0, e1);
        } else if (P == kWeights) {
          float w0, w1;
          f32x2_parts(mul2(e, f32x2(f, f)), w0, w1);
          const __half2 h = __floats2half2_rn(w0, w1);
          pk[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          float w0, w1, r0, r1;
          f32x2_parts(mul2(e, f32x2(f, f)), w0, w1);
          const uint32_t b0 = __float_as_uint(w0), b1 = __float_as_uint(w1);
          f32x2_parts(add2(f32x2(w0, w1), f32x2(__uint_as_float(b0 & 0xFFFF0000u ^ 0x80000000u), __uint_as_float(b1 & 0xFFFF0000u ^ 0x80000000u))), r0, r1);
          pk[i & 7] = __byte_perm(b0, b1, 0x7632);
          pk[8 + (i & 7)] = pack_p(r0, r1);
          if ((i & 7) == 7) {
            tmem_st8(p_at + (i & 8), pk);
            tmem_st8(p_at + 16 + (i & 8), pk + 8);
          }
        }
      }
    }
    // (P's columns end before those of S that are still to be read, 32 (w + 1) ..)
    if (!SPLIT || none) tmem_st16(p_at, pk);
    if (w1 == 1) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      ready(w2 >> 1);
    }
  }
  float lo, hi;
  f32x2_parts(add2(sum[0], sum[1]), lo, hi);
  row.l += lo + hi;
}

}  // namespace dt
