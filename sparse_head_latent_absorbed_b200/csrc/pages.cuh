// The paged latent cache: row formats, argument checks and the exact
// conversion between bf16 values and 8-bit codes with power-of-two scales.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "host_util.h"

namespace shla {
namespace pages {

constexpr int kLatent = MLA_LATENT, kRope = MLA_ROPE, kRow = MLA_ROW;
constexpr int kRow8Bytes = MLA_PAGE_ROW8;          // 512 codes, 4 scales, 64 rotary values
constexpr int kScaleOff = kLatent;                 // byte offsets in an 8-bit row
constexpr int kRopeOff = kLatent + 16;
static_assert(kRopeOff + 2 * kRope == kRow8Bytes, "8-bit row");

inline int min_row_bytes(int kind) { return kind == MLA_PAGE_E4M3 ? kRow8Bytes : 2 * kRow; }

// Checks of a pool of pages: sizes first, then alignment.  Rows are addressed
// as page * (page_stride / row_stride) + offset, so the page stride is a
// multiple of the row stride and the last row's index fits 32 bits (with room
// for one box of rows past the end).
inline int check_pool(const void* pool, int kind, int num_pages, int page_size,
                      int64_t page_stride, int row_stride) {
  if (!pool) return MLA_ERR_NULL;
  if (kind != MLA_PAGE_BF16 && kind != MLA_PAGE_E4M3) return MLA_ERR_SHAPE;
  if (num_pages < 1 || page_size < 1 || row_stride < min_row_bytes(kind) || page_stride < 0)
    return MLA_ERR_SHAPE;
  if (!aligned16(pool) || row_stride % 16 || page_stride % 16) return MLA_ERR_ALIGN;
  if (page_stride % row_stride || page_stride / row_stride < page_size) return MLA_ERR_SHAPE;
  // (bounds the product below: 2^31 pages of at most 2^32 rows each)
  if (page_stride / row_stride > 0x7fffff00LL) return MLA_ERR_SHAPE;
  if ((int64_t)(num_pages - 1) * (page_stride / row_stride) + page_size > 0x7fffff00LL)
    return MLA_ERR_SHAPE;
  return MLA_OK;
}

// least n with top <= 448 * 2^n, kept in [-117, 119]: 448 = 1.75 * 2^8, so
// from the bits of top = m * 2^e (m in [1, 2)) it is e - 8, or e - 7 when m
// is above 1.75.  At n >= -117 the smallest code step 2^(n-9) is a normal
// bf16; at n <= 119 the largest value 448 * 2^n is finite.
DEV int scale_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127;
  const int n = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(119, max(-117, n));
}
DEV float pow2(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }  // -126 <= n <= 127

// two fp32 values to two e4m3 codes (lo in bits 0-7): nearest even, past 448
// saturated, NaN kept
DEV uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// two codes (bits 0-15) as fp32 values, exactly
DEV float2 from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Four codes times a power of two 2^n, n <= 7, as four bf16 values, exactly: a
// code's sign, exponent and mantissa bits moved into bf16's places read as
// value * 2^-120 (bf16 subnormals for e4m3 subnormals), so one exact product
// by f = 2^(120 + n) restores it.  (NaN is in the scale, never in a code.)
DEV uint2 dequant4(uint32_t w, __nv_bfloat162 f) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  uint32_t lo = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u);
  uint32_t hi = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&lo), f);
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&hi), f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// whether a scale of the warp is past dequant4's range
template <int N>
DEV bool any_big(const float (&sc)[N]) {
  float m = sc[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, sc[i]);
  return __any_sync(0xffffffffu, m > 128.f);
}

// sixteen codes times `scale` as sixteen bf16 values (big: the scale may be
// above 2^7)
DEV void dequant16(const uint4& c, float scale, bool big, uint4& o0, uint4& o1) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t r[8];
  if (big) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const uint32_t wi = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
      const float2 f = from_e4m3x2(wi), g = from_e4m3x2(wi >> 16);
      const uint32_t a = pack_bf16x2(f.x * scale, f.y * scale);
      const uint32_t b = pack_bf16x2(g.x * scale, g.y * scale);
      if (i == 0) { r[0] = a; r[1] = b; }
      if (i == 1) { r[2] = a; r[3] = b; }
      if (i == 2) { r[4] = a; r[5] = b; }
      if (i == 3) { r[6] = a; r[7] = b; }
    }
  } else {
    const __nv_bfloat162 f = __float2bfloat162_rn(scale * __uint_as_float(0x7b800000u));  // 2^120
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 v = dequant4(w[i], f);
      r[2 * i] = v.x;
      r[2 * i + 1] = v.y;
    }
  }
  o0 = make_uint4(r[0], r[1], r[2], r[3]);
  o1 = make_uint4(r[4], r[5], r[6], r[7]);
}

}  // namespace pages
}  // namespace shla
