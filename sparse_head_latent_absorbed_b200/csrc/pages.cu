// Writing rows into a paged latent cache and reading them back, in 8 or 16
// bits.  Both are bound by memory: a row is read once and written once
// (1152 B on the bf16 side, 656 or 1152 B on the page side).  Measured from a cold
// L2: 16384 rows written in 10 us (8 bits; 4.5 at the copy rate) and 10 to 12 (16
// bits; 5.8), 32768 read in 16 us (9.1) and 18 (11.5); a few rows in 6, which is a
// launch.  A warp's one row (its slot, then its address, then its store) has
// nothing in flight behind it.
#include "pages.cuh"

namespace shla {
namespace pages {

// One warp per row.  A lane holds 16 latent values (two 16-byte loads), so a
// group of 128 is eight neighbouring lanes and its largest magnitude three
// shuffles; the first eight lanes also carry the rotary key.  A lane's loads
// do not depend on each other, and eight rows per block times eight blocks
// per SM keep about 70 KB in flight on each.
template <bool kE4M3>
__global__ void __launch_bounds__(256) page_write_kernel(
    const __nv_bfloat16* __restrict__ rows, long long rstride, const int32_t* __restrict__ slots,
    int N, uint8_t* __restrict__ pool, long long page_stride, int row_stride, int num_slots,
    int page_size, int32_t* status) {
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= N) return;
  const __nv_bfloat16* src = rows + (long long)r * rstride;
  const uint4 a = ld_global_nc_v4(src + lane * 16), b = ld_global_nc_v4(src + lane * 16 + 8);
  uint4 pe = make_uint4(0, 0, 0, 0);
  if (lane < 8) pe = ld_global_nc_v4(src + kLatent + lane * 8);
  const int slot = slots[r];
  if (slot < 0 || slot >= num_slots) {
    if (lane == 0 && slot != -1 && status) atomicAdd(status + 1, 1);
    return;
  }
  uint8_t* dst = pool + (long long)(slot / page_size) * page_stride +
                 (long long)(slot % page_size) * row_stride;
  if (!kE4M3) {
    *reinterpret_cast<uint4*>(dst + lane * 32) = a;
    *reinterpret_cast<uint4*>(dst + lane * 32 + 16) = b;
    if (lane < 8) *reinterpret_cast<uint4*>(dst + 2 * kLatent + lane * 16) = pe;
    return;
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16];
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = fmaxf(top, fabsf(x[i]));  // (fmaxf drops a NaN)
    finite = finite && fabsf(x[i]) <= 3.4e38f;
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // a group with a NaN or an infinity: scale NaN, codes 0
  const unsigned bad = __ballot_sync(0xffffffffu, !finite) >> (lane & 24) & 0xffu;
  const int n = scale_exponent(top);
  const float inv = pow2(-n);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
           (to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
  *reinterpret_cast<uint4*>(dst + lane * 16) =
      bad ? make_uint4(0, 0, 0, 0) : make_uint4(c[0], c[1], c[2], c[3]);
  if ((lane & 7) == 0)
    *reinterpret_cast<float*>(dst + kScaleOff + (lane >> 3) * 4) =
        bad ? __uint_as_float(0x7fc00000u) : pow2(n);
  if (lane < 8) *reinterpret_cast<uint4*>(dst + kRopeOff + lane * 16) = pe;
}

// One warp per row, the same split.  Slot -1 and slots outside the pool give
// a row of zeros.
template <bool kE4M3>
__global__ void __launch_bounds__(256) page_read_kernel(
    const uint8_t* __restrict__ pool, long long page_stride, int row_stride, int num_slots,
    int page_size, const int32_t* __restrict__ slots, int N, __nv_bfloat16* __restrict__ rows,
    long long rstride, int32_t* status) {
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= N) return;
  const int slot = ld_global_nc_s32_early(slots + r);
  const bool in = slot >= 0 && slot < num_slots;
  if (!in && slot != -1 && lane == 0 && status) atomicAdd(status + 1, 1);
  uint4 a = make_uint4(0, 0, 0, 0), b = a, pe = a;
  if (in) {
    const uint8_t* src = pool + (long long)(slot / page_size) * page_stride +
                         (long long)(slot % page_size) * row_stride;
    if (kE4M3) {
      const uint4 c = ld_global_nc_v4(src + lane * 16);
      const float s =
          __int_as_float(ld_global_nc_s32_early(reinterpret_cast<const int32_t*>(
              src + kScaleOff + (lane >> 3) * 4)));
      if (lane < 8) pe = ld_global_nc_v4(src + kRopeOff + lane * 16);
      dequant16(c, Factor(s), needs_fp32(s), a, b);
    } else {
      a = ld_global_nc_v4(src + lane * 32);
      b = ld_global_nc_v4(src + lane * 32 + 16);
      if (lane < 8) pe = ld_global_nc_v4(src + 2 * kLatent + lane * 16);
    }
  }
  __nv_bfloat16* dst = rows + (long long)r * rstride;
  *reinterpret_cast<uint4*>(dst + lane * 16) = a;
  *reinterpret_cast<uint4*>(dst + lane * 16 + 8) = b;
  if (lane < 8) *reinterpret_cast<uint4*>(dst + kLatent + lane * 8) = pe;
}

static int check_rows(const void* rows, int64_t rstride, const int32_t* slots, int N) {
  if (!rows || !slots) return MLA_ERR_NULL;
  if (N < 0 || rstride < kRow) return MLA_ERR_SHAPE;
  if (!aligned16(rows) || rstride % 8 || (reinterpret_cast<uintptr_t>(slots) & 3u))
    return MLA_ERR_ALIGN;
  return MLA_OK;
}

}  // namespace pages
}  // namespace shla

using namespace shla;

extern "C" int mla_page_write(const mla_bf16_t* rows, int64_t rstride, const int32_t* slots,
                              int N, void* pool, int kind, int num_pages, int page_size,
                              int64_t page_stride, int row_stride, int32_t* status,
                              void* stream) {
  if (int e = pages::check_rows(rows, rstride, slots, N)) return e;
  if (int e = pages::check_pool(pool, kind, num_pages, page_size, page_stride, row_stride))
    return e;
  if (N == 0) return MLA_OK;
  const int64_t ns = (int64_t)num_pages * page_size;  // <= 2^31 (check_pool)
  const dim3 grid((unsigned)(((int64_t)N + 7) / 8));
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(rows);
  if (kind == MLA_PAGE_E4M3)
    pages::page_write_kernel<true><<<grid, 256, 0, as_stream(stream)>>>(
        src, rstride, slots, N, static_cast<uint8_t*>(pool), page_stride, row_stride, (int)ns,
        page_size, status);
  else
    pages::page_write_kernel<false><<<grid, 256, 0, as_stream(stream)>>>(
        src, rstride, slots, N, static_cast<uint8_t*>(pool), page_stride, row_stride, (int)ns,
        page_size, status);
  return launch_status();
}

extern "C" int mla_page_read(const void* pool, int kind, int num_pages, int page_size,
                             int64_t page_stride, int row_stride, const int32_t* slots, int N,
                             mla_bf16_t* rows, int64_t rstride, int32_t* status, void* stream) {
  if (int e = pages::check_rows(rows, rstride, slots, N)) return e;
  if (int e = pages::check_pool(pool, kind, num_pages, page_size, page_stride, row_stride))
    return e;
  if (N == 0) return MLA_OK;
  const int64_t ns = (int64_t)num_pages * page_size;
  const dim3 grid((unsigned)(((int64_t)N + 7) / 8));
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(rows);
  if (kind == MLA_PAGE_E4M3)
    pages::page_read_kernel<true><<<grid, 256, 0, as_stream(stream)>>>(
        static_cast<const uint8_t*>(pool), page_stride, row_stride, (int)ns, page_size, slots, N,
        dst, rstride, status);
  else
    pages::page_read_kernel<false><<<grid, 256, 0, as_stream(stream)>>>(
        static_cast<const uint8_t*>(pool), page_stride, row_stride, (int)ns, page_size, slots, N,
        dst, rstride, status);
  return launch_status();
}
