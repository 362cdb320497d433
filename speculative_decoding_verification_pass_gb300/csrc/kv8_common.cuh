// Helpers of the 8-bit paged KV cache: e4m3 conversions, the block scale and
// page addressing.
//
// A cached row is code x scale: the codes are e4m3, the scale a power of two
// shared by a block of kKv8Block slots of one KV head.  A power of two makes
// code x scale exact, and every change of scale for values that stay normal e4m3
// numbers, which a larger scale for a later row then leaves as they are; values
// that become subnormal (below 2^-6 of the new scale) are rounded again at each
// growth and each move.
#pragma once

#include "common.cuh"

namespace spec {
namespace {

constexpr int kKv8Block = SPEC_KV8_BLOCK;             // slots per scale
constexpr int kKv8Sub = kPageSlots / kKv8Block;       // scales per page and head
constexpr float kKv8Min = 9.094947017729282e-13f;     // 2^-40, the smallest scale
constexpr int kKv8MaxExp = 40;

// Two fp32 values to two e4m3 codes (nearest, ties to even; beyond +-448 and
// infinities to +-448, NaN to the NaN code), `a` in the low byte.
SPEC_DEVINL uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
SPEC_DEVINL uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// The two low codes of w as fp32 (exact: every e4m3 value is an fp16 value).
SPEC_DEVINL float2 e4m3x2_to_f32(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  float2 f;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The scale of a block whose largest finite magnitude is amax: the smallest
// power of two s in [2^-40, 2^40] with amax <= 448 s (448 = 1.75 * 2^8 is the
// largest e4m3 value), from amax's own exponent and fraction.
SPEC_DEVINL float kv8_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8;
  if ((u & 0x7FFFFFu) > 0x600000u) ++e;  // fraction above 1.75
  e = e < -kKv8MaxExp ? -kKv8MaxExp : (e > kKv8MaxExp ? kKv8MaxExp : e);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// 1 / s of a power-of-two scale, exactly.
SPEC_DEVINL float pow2_inv(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

// Four codes re-rounded from scale s_old to s_new, ratio = s_old / s_new.
SPEC_DEVINL uint32_t kv8_rescale4(uint32_t w, float ratio) {
  const float2 a = e4m3x2_to_f32(w), b = e4m3x2_to_f32(w >> 16);
  return e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// Slot addressing of one layer: rows [page][Hkv][64][hd], scales [page][Hkv][4].
struct Kv8Map {
  const int32_t* table;
  int max_pages, n_pages, Hkv, hd;
  // the page holding slot t of sequence b, clamped into the pool
  SPEC_DEVINL int page(int b, int t) const {
    const int pg = table[static_cast<long long>(b) * max_pages + t / kPageSlots];
    return pg < 0 ? 0 : (pg >= n_pages ? n_pages - 1 : pg);
  }
  SPEC_DEVINL long long row(int page, int h, int t) const {
    return ((static_cast<long long>(page) * Hkv + h) * kPageSlots + t % kPageSlots) * hd;
  }
  SPEC_DEVINL long long scale(int page, int h, int t) const {
    return (static_cast<long long>(page) * Hkv + h) * kKv8Sub + (t % kPageSlots) / kKv8Block;
  }
};

// 0 when slots [L, L + n) of sequence b (n <= 128) lie within the capacity and
// on pages of the pool, else the status bit.  Only those pages are looked at, a
// lane each; every lane of the warp calls it and gets the answer, and in *page
// the page of slot t (one of the slots, or of the block that slot L is in).
SPEC_DEVINL int32_t kv8_fit_warp(int L, int n, const int32_t* table, int max_pages, int n_pages, int b, int t,
                                 int* page) {
  *page = 0;
  if (L < 0 || L > max_pages * kPageSlots - n) return SPEC_DEV_KV_OVERFLOW;
  const int p0 = L / kPageSlots, np = (L + n - 1) / kPageSlots - p0 + 1, lane = threadIdx.x & 31;
  const int pg = lane < np ? table[static_cast<long long>(b) * max_pages + p0 + lane] : 0;
  if (__any_sync(0xffffffffu, pg < 0 || pg >= n_pages)) return SPEC_DEV_BAD_PAGE;
  *page = __shfl_sync(0xffffffffu, pg, t / kPageSlots - p0);
  return 0;
}

}  // namespace
}  // namespace spec
