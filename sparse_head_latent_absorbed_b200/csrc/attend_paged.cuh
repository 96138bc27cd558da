// What the two forms of the attention over a paged cache share: the
// description of the pages and the device-side view of a call's sequences.
#pragma once

#include "pages.cuh"

namespace shla {
namespace paged {

constexpr int kH = MLA_HEADS, kC = MLA_LATENT, kR = MLA_ROPE, kD = MLA_NOPE;
static_assert(MLA_NOPE == 128 && MLA_VDIM == 128, "key and value widths");

// The tensor cores add to an fp32 accumulator with truncation: a product of 16
// positions loses up to 2^-23 of it, always towards zero.  Measured, one latent in
// all positions: 0.6% short after 2^20 of them, 2.6% after 2^22.  So after kRun tiles
// of 128 positions (a loss of 2^-10 at most) an accumulator is added, rounded to
// nearest, to a copy in the workspace, and begins anew.
constexpr int kRun = 1024;

// Limit of a wait for the place of the next queries, which are in use for `tiles`
// key tiles: up to 131,072 of them, of 5.1 us at most (16-bit pages of one row,
// measured), so 0.67 s on a GPU that does nothing else.
DEV uint64_t queries_limit_ns(int tiles) { return kWaitLimitNs + (uint64_t)tiles * 50000u; }

template <typename T>
DEV T* align1024(T* p) {
  return reinterpret_cast<T*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// A pool of pages and the table of each sequence's pages.
struct Pool {
  const uint8_t* base;
  int kind;               // MLA_PAGE_BF16 or MLA_PAGE_E4M3
  int num_pages, page_size;
  int pitch;              // rows from one page to the next
  int row_stride;         // bytes
  int rows;               // rows from the first page's first to the last page's last
  uint32_t magic;         // pos / page_size = pos * magic >> shift, for 0 <= pos <= 2^24
  int shift;
  const int32_t* table;   // [S][max_pages]
  int max_pages;
};

// With 2^b >= page_size, shift = 24 + b and magic = ceil(2^shift / page_size), the
// product overshoots pos * 2^shift / page_size by less than pos <= 2^24 <=
// 2^shift / page_size: not as far as the next whole quotient.
inline void set_division(Pool* p) {
  int b = 0;
  while ((1ll << b) < p->page_size) ++b;
  p->shift = 24 + b;
  p->magic = (uint32_t)(((1ull << p->shift) + p->page_size - 1) / p->page_size);
}
DEV int page_of(const Pool& p, int pos) {
  return (int)((uint64_t)(uint32_t)pos * p.magic >> p.shift);
}

// The sequences of a call: sequence s has new tokens cu_q[s] .. cu_q[s+1]-1
// and kv_len[s] cached positions, the new tokens' own among them.
struct Seqs {
  const int32_t* cu_q;
  const int32_t* kv_len;
  int S, N, max_kv;

  // token range of s, whatever cu_q holds, inside [0, N]
  DEV int q0(int s) const { return min(max(cu_q[s], 0), N); }
  // positions of s, inside what the bound and the table allow
  DEV int kv(int s, const Pool& p) const {
    const long long cap = (long long)p.max_pages * p.page_size;
    return max(0, min(min(kv_len[s], max_kv), (int)(cap < max_kv ? cap : max_kv)));
  }
};

// The row of position `pos` of the sequence whose table row is `t`, or
// `p.rows` (past the end: reads as zeros) when the table holds no valid page.
DEV int row_of(const Pool& p, const int32_t* t, int pos) {
  const int pg = page_of(p, pos);
  const int page = ld_global_nc_s32_early(t + pg);
  return page >= 0 && page < p.num_pages ? page * p.pitch + (pos - pg * p.page_size) : p.rows;
}

}  // namespace paged
}  // namespace shla
