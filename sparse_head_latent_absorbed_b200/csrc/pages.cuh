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
  // (bounds the product below: 2^31 pages of less than 2^31 rows each)
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
// by f = 2^(120 + n) restores it.  (NaN is in the scale, never in a code: one would
// read as 480 * 2^n.)
DEV uint2 dequant4(uint32_t w, __nv_bfloat162 f) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  uint32_t lo = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u);
  uint32_t hi = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&lo), f);
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&hi), f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// The same for any scale: through fp32, the product rounded to bf16.  Out of
// line, for scales above 2^7 and for those of rows from elsewhere that are no
// power of two (where the exact product above would round the scale too).
static __device__ __noinline__ uint4 dequant8_any(uint2 c, float scale) {
  const float2 a = from_e4m3x2(c.x), b = from_e4m3x2(c.x >> 16);
  const float2 d = from_e4m3x2(c.y), e = from_e4m3x2(c.y >> 16);
  return make_uint4(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale),
                    pack_bf16x2(d.x * scale, d.y * scale), pack_bf16x2(e.x * scale, e.y * scale));
}

// whether dequant4 cannot take the scale: anything but 0 and the powers of two from
// 2^-126 to 2^7
DEV bool needs_fp32(float scale) {
  const uint32_t u = __float_as_uint(scale);
  return u > 0x43000000u || (u & 0x7fffffu) != 0;
}

// a scale and what dequant4 multiplies by
struct Factor {
  float scale;
  __nv_bfloat162 f;
  DEV explicit Factor(float s)
      : scale(s), f(__float2bfloat162_rn(s * 1.329227995784916e36f)) {}  // 2^120
};

// sixteen codes times a scale as sixteen bf16 values; fp32: needs_fp32 of the scale
// (any scale may take that way)
DEV void dequant16(const uint4& c, const Factor& f, bool fp32, uint4& o0, uint4& o1) {
  if (fp32) {
    o0 = dequant8_any(make_uint2(c.x, c.y), f.scale);
    o1 = dequant8_any(make_uint2(c.z, c.w), f.scale);
    return;
  }
  const uint2 a = dequant4(c.x, f.f), b = dequant4(c.y, f.f), d = dequant4(c.z, f.f),
              e = dequant4(c.w, f.f);
  o0 = make_uint4(a.x, a.y, b.x, b.y);
  o1 = make_uint4(d.x, d.y, e.x, e.y);
}

}  // namespace pages
}  // namespace shla
