// Shared by the kernels around the target model's key/value cache: argument
// checks, the smallest power-of-two scale, e4m3 conversions.
#pragma once

#include <cstdarg>
#include <cstdio>

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace dt {

DT_DEVINL float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

DT_DEVINL float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The unit of a row's O over cached tokens.  A weight 2^z v (z: logit, v: its key's value scale) goes to the product with V
// in fp16 as 2^(z - u) v, and O is in units of 2^u.  u follows the keys, up and down: of the keys of a tile or step the
// largest weight stands at 2^0 .. 2^15 (2^8 where u has moved), so that what fp16 cannot hold, 2^-25 or less, is that small beside
// the largest of the same keys, whatever stands in other tiles and whatever scale a page without weight has.  Downwards u
// stops 60 below its highest value, behind which O, in 32 bits, might overflow and what is added is lost to it all the same;
// and it stays above m - 118 (m: the maximum in use), so that 2^(m - u) is a number.
constexpr float kUnitTop = 15.0f, kUnitSet = 8.0f, kUnitFall = 60.0f, kUnitBelow = 118.0f;
// weight: the largest z + log2 v of the row's keys.  Returns what O is to be multiplied by.
DT_DEVINL float move_unit(float weight, float m, float& u, float& high) {
  const float before = u;
  if (weight > -INFINITY && (weight > u + kUnitTop || weight < u)) u = fmaxf(weight - kUnitSet, high - kUnitFall);
  u = fmaxf(u, m - kUnitBelow);
  high = fmaxf(high, u);
  return u == before ? 1.0f : ex2(before - u);
}

constexpr int kSms = 152;  // of a GB300: grids of one wave

// Smallest power of two s in [2^-126, 2^120] with 448 s >= amax (amax finite,
// >= 0).  448 = 1.75 * 2^8, so with amax = m 2^k (1 <= m < 2) s is 2^(k-8)
// where m <= 1.75 and 2^(k-7) above: read off the bits, no logarithm.
DT_DEVINL float kv_pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : (e > 120 ? 120 : e);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four e4m3 bytes (lowest first) to two pairs of fp16, exact.
DT_DEVINL void e4m3x4_to_f16x2x2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// Asks for a CTA of this grid that has not started; the answer (16 bytes) completes on `bar`.
DT_DEVINL void take_next(void* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// The CTA that was taken over, or -1.
DT_DEVINL int taken(const void* answer) {
  const volatile uint64_t* w = reinterpret_cast<const volatile uint64_t*>(answer);
  const uint64_t lo = w[0], hi = w[1];
  int ok, id;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tmov.b128 h, {%2, %3};\n\tmov.b32 %1, 0;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.b32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(id)
      : "l"(lo), "l"(hi));
  return ok ? id : -1;
}

inline dt_status kv_fail(dt_status s, const char* fmt, ...) {
  char msg[240];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_last_error(msg);
  return s;
}

inline dt_status kv_launched(const char* who, cudaError_t e) {
  if (e == cudaSuccess) return DT_OK;
  return kv_fail(DT_ERR_CUDA, "%s: launch failed: %s (%d)", who, cudaGetErrorString(e), static_cast<int>(e));
}

inline bool kv_page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Rows of heads: 16-byte aligned base, strides that keep every head 16-byte aligned.
inline bool kv_rows_ok(const void* p, int64_t row_stride, int64_t head_stride) {
  return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && row_stride >= 0 && head_stride >= 0 &&
         row_stride % 8 == 0 && head_stride % 8 == 0;
}

// Rows of heads that are written: no two of them may share an element.
inline bool kv_rows_apart(int64_t rows, int heads, int head_dim, int64_t row_stride, int64_t head_stride) {
  return (rows == 1 || row_stride >= head_dim) && (heads == 1 || head_stride >= head_dim) &&
         (rows == 1 || heads == 1 || row_stride >= (heads - 1) * head_stride + head_dim || head_stride >= (rows - 1) * row_stride + head_dim);
}

dt_status kv_check_cache(const char* who, const dt_kv_cache* c);

// Rows of heads in bf16 (strides in elements) as a 3D tensor map: boxes of 64 channels x heads x rows, swizzled.
bool kv_tmap_heads(CUtensorMap* tm, const void* base, int head_dim, int heads, int64_t rows, int64_t head_stride,
                   int64_t row_stride, int box_heads, int box_rows);
// Contiguous rows of 64 or 128 bytes as a 2D map of bytes, swizzled by the row's length: boxes of whole rows.
bool kv_tmap_rows(CUtensorMap* tm, const void* base, int row_bytes, int64_t rows, int box_rows);

}  // namespace dt
