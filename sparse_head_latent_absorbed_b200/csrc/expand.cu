// Attention of new tokens over a paged latent cache, expanded form: the keys
// and values of all 128 heads are computed once for every cached position and
// the new tokens attend to those,
//   K[h,t] = [W_UK[h] c_t ; kpe_t],  V[h,t] = W_UV[h] c_t,
//   O[r,h] = softmax_t((q_nope.K + q_pe.kpe) * scale) V.
// From about 171 new tokens a sequence on this takes fewer flops than folding
// W_UK into the queries: 81,920 per token and position and head set against
// 278,528, for 33.6 Mflop a position.  Five kernels:
//
//   layout_kernel   one block: where each sequence's positions go, and the list
//                   of query blocks (up to 512 tokens), cut into equal parts
//   gather_kernel   the pages' rows, as bf16, one sequence after another
//   expand_kernel   K and V of a group of heads: a GEMM on CTA pairs
//   chunk_kernel    the attention of the group's heads, in one range of equal cost
//                   for each CTA pair
//   join_kernel     the outputs of the items that such a range's end cuts
// The last three run once per group; a group is as many heads as the workspace
// holds (all 128 up to 65,536 positions).
#include <math.h>

#include "expand.h"
#include "pair.cuh"
#include "tma_map.h"

namespace shla {
namespace expand {

using paged::kC;
using paged::kD;
using paged::kH;
using paged::kR;
using paged::kRun;
using paged::Pool;
using paged::Seqs;

constexpr int kRows = 128;     // positions of a key tile, tokens of a CTA's query tile
constexpr int kTile = 256;     // tokens of a pair's query tile
constexpr int kBlock = 512;    // tokens of a query block
constexpr size_t kGroupBytes = size_t(4) << 30;  // keys and values of a group of heads

// ===========================================================================
// layout
// ===========================================================================

// A query block: tokens [tok, tok + n) of one sequence, n <= 512; the first sees
// `lim` positions (possibly none or less), each next one more, none more than kv;
// position 0 is row `row` of the gathered rows.  A CTA pair works on two query
// tiles at a time: of up to 256 tokens, the same block for two heads; of more,
// both parts of the block for one head, and the list has the block twice, for the
// first and for the second half of the heads (`upper`).
struct Block {
  int tok, n, lim, kv, row, upper;
  DEV bool two_heads() const { return n <= kTile; }
  // tokens of a tile that each CTA takes
  DEV int width() const { return two_heads() ? (n + 1) / 2 : (n + 3) / 4; }
  DEV int first(int t) const { return two_heads() ? 0 : t * 2 * width(); }  // of tile t
  DEV int head(int t, int i, int heads) const {  // item i of heads / 2
    return two_heads() ? 2 * i + t : upper * (heads / 2) + i;
  }
  DEV int tiles(int t) const {  // key tiles of query tile t
    const int last = min(n, first(t) + 2 * width());
    return max(0, (min(kv, lim + last - 1) + kRows - 1) / kRows);
  }
};

// Where a pair's work begins: key tile j of item g (item g % (heads / 2) of block
// g / (heads / 2)).
struct Cut {
  int g, j;
};

struct Layout {
  int32_t* row;    // [S + 1] first gathered row of each sequence (multiples of 128)
  int32_t* kv;     // [S]
  Block* block;    // [N / 256 + S]
  int32_t* start;  // [N / 256 + S] cost of the blocks before it, for one item of each
  Cut* cut;        // [pairs + 1]
};

constexpr int kPairs = 74;    // at most; CTA pairs that share the work
constexpr int kItemCost = 1;  // of an item, in key tiles: its queries' load and its output
constexpr int kMinPiece = 4;  // key tiles that a cut leaves on either side

// exclusive prefix sum over the block's 1024 threads; *total: the sum
DEV int scan1024(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto up = [&](int x) {  // inclusive, over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int x = up(v);
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) part[32 + lane] = up(part[lane]);
  __syncthreads();
  *total = part[63];
  const int r = (warp ? part[31 + warp] : 0) + x - v;
  __syncthreads();
  return r;
}

// One block.  Everything follows from the sequences' order alone: where the list
// is cut decides how some outputs are rounded.
__global__ void __launch_bounds__(1024) layout_kernel(const Seqs q, const Pool pool,
                                                       const Layout ly, int items, int pairs) {
  __shared__ int part[64];
  const int tid = threadIdx.x;
  pdl_trigger();
  const int per = (q.S + 1023) / 1024;
  const int lo = min(q.S, tid * per), hi = min(q.S, lo + per);
  int rows = 0, blocks = 0;
  for (int s = lo; s < hi; ++s) {
    // a sequence without new tokens needs no keys
    const int n = q.q0(s + 1) - q.q0(s), kv = n > 0 ? q.kv(s, pool) : 0;
    ly.kv[s] = kv;
    rows += (kv + kRows - 1) / kRows * kRows;
    blocks += max(0, (n + kTile - 1) / kTile);
  }
  int total;
  int at = scan1024(rows, part, &total);
  if (tid == 0) ly.row[q.S] = total;
  // (ranges of a cu_q that decreases may overlap: no more blocks than there is room for)
  const int room = q.N / kTile + q.S;
  int i = min(scan1024(blocks, part, &total), room);
  const int first = i, n = min(total, room);
  int cost = 0;
  for (int s = lo; s < hi; ++s) {
    ly.row[s] = at;
    const int t0 = q.q0(s), len = q.q0(s + 1) - t0;
    for (int k = 0; k < len && i < room; k += kBlock) {
      Block b;
      b.tok = t0 + k;
      b.n = min(kBlock, len - k);
      b.kv = ly.kv[s];
      b.lim = b.kv - len + k + 1;
      b.row = at;
      b.upper = 0;
      const int c = b.tiles(1) + kItemCost;
      ly.block[i++] = b;
      cost += c;
      if (b.two_heads() || i >= room) continue;
      b.upper = 1;
      ly.block[i++] = b;
      cost += c;
    }
    at += (ly.kv[s] + kRows - 1) / kRows * kRows;
  }
  // the list cut into one range of equal cost for each pair
  int all;
  int run = scan1024(cost, part, &all);
  for (int k = first; k < i; ++k) {
    ly.start[k] = run;
    run += ly.block[k].tiles(1) + kItemCost;
  }
  __syncthreads();
  if (tid <= pairs) {
    Cut c = {n * items, 0};
    if (tid < pairs && n > 0) {
      const long long u = (long long)tid * all * items / pairs;
      int a = 0, e = n;  // start[a] * items <= u
      while (e - a > 1) {
        const int m = (a + e) >> 1;
        if ((long long)ly.start[m] * items <= u) a = m; else e = m;
      }
      const int tiles = ly.block[a].tiles(1), one = tiles + kItemCost;
      const long long in = u - (long long)ly.start[a] * items;
      c.g = a * items + (int)(in / one);
      c.j = (int)(in % one) - kItemCost;
      if (c.j < kMinPiece) {
        c.j = 0;
      } else if (tiles - c.j < kMinPiece) {
        c.j = 0;
        ++c.g;
      }
    }
    ly.cut[tid] = c;
  }
}

// ===========================================================================
// gather: row ly.row[s] + t = position t of sequence s as bf16, zeros from
// kv[s] to the next multiple of 128 and for entries outside the pool (counted
// once a page).  One warp per row; bound by memory (128000 8-bit rows, 231 MB, in
// 41 to 47 us; four rows a warp took the same).  `table`, if there is one:
// the rows' table as pages of 64.
// ===========================================================================
constexpr int kStagedPage = 64;

template <bool kE4M3>
__global__ void __launch_bounds__(256) gather_kernel(const Pool pool, const Layout ly, int S,
                                                      __nv_bfloat16* __restrict__ rows,
                                                      int32_t* __restrict__ table, int max_pages,
                                                      int32_t* status) {
  const int lane = threadIdx.x & 31;
  pdl_wait();  // the layout
  pdl_trigger();
  const int total = ld_global_nc_s32_early(ly.row + S);
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < total; r += gridDim.x * 8) {
    int a = 0, e = S;  // the last sequence that starts at or before row r
    while (e - a > 1) {
      const int m = (a + e) >> 1;
      if (ly.row[m] <= r) a = m; else e = m;
    }
    const int t = r - ly.row[a];
    if (table && lane == 0 && t % kStagedPage == 0)
      table[(long long)a * max_pages + t / kStagedPage] = r / kStagedPage;
    uint4 x = make_uint4(0, 0, 0, 0), y = x, pe = x;
    if (t < ly.kv[a]) {
      const int row = paged::row_of(pool, pool.table + (long long)a * pool.max_pages, t);
      if (row == pool.rows) {
        if (lane == 0 && t % pool.page_size == 0 && status) atomicAdd(status + 1, 1);
      } else {
        const uint8_t* src = pool.base + (long long)row * pool.row_stride;
        if (kE4M3) {
          const uint4 c = ld_global_nc_v4(src + lane * 16);
          const float sc = __int_as_float(ld_global_nc_s32_early(
              reinterpret_cast<const int32_t*>(src + pages::kScaleOff + (lane >> 3) * 4)));
          if (lane < 8) pe = ld_global_nc_v4(src + pages::kRopeOff + lane * 16);
          pages::dequant16(c, pages::Factor(sc), pages::needs_fp32(sc), x, y);
        } else {
          x = ld_global_nc_v4(src + lane * 32);
          y = ld_global_nc_v4(src + lane * 32 + 16);
          if (lane < 8) pe = ld_global_nc_v4(src + 2 * kC + lane * 16);
        }
      }
    }
    __nv_bfloat16* dst = rows + (long long)r * MLA_ROW;
    *reinterpret_cast<uint4*>(dst + lane * 16) = x;
    *reinterpret_cast<uint4*>(dst + lane * 16 + 8) = y;
    if (lane < 8) *reinterpret_cast<uint4*>(dst + kC + lane * 8) = pe;
  }
}

// ===========================================================================
// expand_kernel: [K | V][rows, 256] = C [rows, 512] W[h]^T for the group's heads
//
// A pair of CTAs multiplies 256 rows with one head's 256 weight rows
// (tcgen05 cta_group::2, M = 256, N = 256): CTA r holds rows [128r, +128) of C,
// all 512 columns, for as many heads as its range of the (row block, head)
// list holds, and streams its half of the weight (r = 0: W_UK, 1: W_UV),
// 16 KB for every 512 cycles of products.  (Measured: 6000 positions, 128 heads,
// 167 us, 1.2 PFLOP/s with 393 MB written.)  One CTA alone would have to take in
// 64 bytes a cycle, which is more than its share of L2.
// Warps 0-3: epilogue (TMEM -> bf16 -> swizzled shared memory -> TMA store),
// warp 4: TMA loads, warp 5: MMA (the pair's first CTA issues for both).
// Two TMEM accumulators, so the epilogue of one tile overlaps the next.
// ===========================================================================
namespace gemm {
constexpr int NB = 4;                       // weight ring depth
constexpr int CHUNK = kRows * 128;          // 64 columns of 128 rows
constexpr int OFF_B = 8 * CHUNK;
constexpr int OFF_OUT = OFF_B + NB * CHUNK; // two output boxes of 64 columns
constexpr int SMEM = OFF_OUT + 2 * CHUNK + 1024;
constexpr int THREADS = 192;
static_assert(SMEM + 512 <= 232448, "shared memory budget");

struct Bars {
  uint64_t a_full[8], a_empty[8];   // (first CTA) / (both)
  uint64_t b_full[NB], b_empty[NB];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
}  // namespace gemm

DEV void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::
                   "l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
// whether `ok` holds in all of warps 0-3 (named barrier 1)
DEV bool all_of_128(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(gemm::THREADS, 1)
    expand_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const int32_t* __restrict__ total_rows, int head0, int heads, int32_t* status) {
  using namespace gemm;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = paged::align1024(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  __shared__ Bars bars;
  volatile int* abort = &bars.abort;
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 5) tmem_alloc2(&bars.tmem_base, 512);
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&bars.a_full[i], 1);
      mbar_init(&bars.a_empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&bars.b_full[i], 1);
      mbar_init(&bars.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 8);  // four epilogue warps of each CTA
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbarrier_init_cluster();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  pdl_wait();  // the rows; of a later group, its predecessor's reads of K and V
  pdl_trigger();
  // this pair's range of the (256-row block, head) list
  const long long items =
      (long long)((ld_global_nc_s32_early(total_rows) + 2 * kRows - 1) / (2 * kRows)) * heads;
  const int pairs = gridDim.x >> 1, cid = blockIdx.x >> 1;
  const int lo = (int)(items * cid / pairs), hi = (int)(items * (cid + 1) / pairs);

  if (warp == 4) {
    // ---------------- loads: each CTA its own operands ----------------
    // The first CTA's barriers count the bytes of both; it alone arrives.
    const uint32_t a_full0 = mapa_shared(smem_u32(&bars.a_full[0]), 0);
    const uint32_t b_full0 = mapa_shared(smem_u32(&bars.b_full[0]), 0);
    int ring = 0, nblk = 0, prev = -1;
    bool ok = true;
    for (int it = lo; it < hi && ok; ++it) {
      const int rb = it / heads, h = it - rb * heads;
      const bool fresh = rb != prev;
      for (int kc = 0; kc < 8 && ok; ++kc) {
        if (fresh) {
          // the previous block's products with this chunk are done
          ok = warp_wait(&bars.a_empty[kc], (nblk & 1) ^ 1, abort, status);
          if (!ok) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&bars.a_full[kc], 2 * CHUNK);
            tma_load_2d_pair(sbase + kc * CHUNK, &map_c, kc * 64, rb * 2 * kRows + rank * kRows,
                             a_full0 + kc * 8);
          }
        }
        const int s = ring % NB;
        ok = warp_wait(&bars.b_empty[s], ((ring / NB) & 1) ^ 1, abort, status);
        if (!ok) break;
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&bars.b_full[s], 2 * CHUNK);
          tma_load_2d_pair(sbase + OFF_B + s * CHUNK, &map_w, kc * 64,
                           (head0 + h) * 256 + rank * 128, b_full0 + s * 8);
        }
        ++ring;
      }
      if (fresh) ++nblk;
      prev = rb;
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------- MMA ----------------
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256, 0, 0);
      int ring = 0, nblk = 0, prev = -1;
      bool ok = true;
      for (int it = lo; it < hi && ok; ++it) {
        const int i = it - lo, buf = i & 1, rb = it / heads;
        const bool fresh = rb != prev;
        const bool last = it + 1 == hi || (it + 1) / heads != rb;
        ok = warp_wait(&bars.acc_empty[buf], ((i >> 1) & 1) ^ 1, abort, status);
        for (int kc = 0; kc < 8 && ok; ++kc) {
          if (fresh) ok = warp_wait(&bars.a_full[kc], nblk & 1, abort, status);
          const int s = ring % NB;
          ok = ok && warp_wait(&bars.b_full[s], (ring / NB) & 1, abort, status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t al = desc_lo(sbase + kc * CHUNK, 16);
          const uint32_t bl = desc_lo(sbase + OFF_B + s * CHUNK, 16);
          if (elect_one()) {
            constexpr uint32_t hi128 = desc_hi(1024, kSwizzle128B);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma2(tmem + buf * 256, desc_join(al + ks * 2, hi128),
                      desc_join(bl + ks * 2, hi128), idesc, (kc > 0 || ks > 0) ? 1u : 0u);
            tc_commit2(&bars.b_empty[s]);
            if (last) tc_commit2(&bars.a_empty[kc]);
            if (kc == 7) tc_commit2(&bars.acc_full[buf]);
          }
          __syncwarp();
          ++ring;
        }
        if (fresh) ++nblk;
        prev = rb;
      }
      // everything issued so far has finished before TMEM is released
      if (elect_one()) tc_commit2(&bars.drain);
      __syncwarp();
      warp_wait(&bars.drain, 0, nullptr, status);
    }
  } else {
    // ---------------- epilogue: this CTA's 128 rows ----------------
    const uint32_t acc_empty0 = mapa_shared(smem_u32(&bars.acc_empty[0]), 0);
    const int row = warp * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    for (int it = lo; it < hi; ++it) {
      const int i = it - lo, buf = i & 1, rb = it / heads, h = it - rb * heads;
      // (the four warps leave together, so that none waits for another below)
      if (!all_of_128(warp_wait(&bars.acc_full[buf], (i >> 1) & 1, abort, status))) break;
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {  // keys 0-63, 64-127, values 0-63, 64-127
        uint32_t r[64];
        tmem_ld32(tmem + lanes + buf * 256 + b * 64, r);
        tmem_ld32(tmem + lanes + buf * 256 + b * 64 + 32, r + 32);
        tc_wait_ld();
        if (b == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(acc_empty0 + buf * 8);
        }
        // the store before last has read its box
        if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const uint32_t box = sbase + OFF_OUT + (b & 1) * CHUNK;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(box + sw128_off(row, c), pack_bf16x2(u2f(r[8 * c]), u2f(r[8 * c + 1])),
                       pack_bf16x2(u2f(r[8 * c + 2]), u2f(r[8 * c + 3])),
                       pack_bf16x2(u2f(r[8 * c + 4]), u2f(r[8 * c + 5])),
                       pack_bf16x2(u2f(r[8 * c + 6]), u2f(r[8 * c + 7])));
        fence_proxy_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (tid == 0) {
          tma_store_3d(b < 2 ? &map_k : &map_v, 0, rb * 2 * kRows + rank * kRows, 2 * h + (b & 1),
                       box);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // a warp that gave up may leave loads in flight, which land within
    // microseconds: a millisecond before the pair leaves
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000) {
    }
  }
  cluster_sync_all();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
  cluster_sync_all();  // neither CTA leaves before both have released
}

// ===========================================================================
// chunk_kernel: attention of two query tiles over the key tiles of 128 positions
//   S_t = Q_t K^T   K = 192, both from shared memory
//   O_t += P_t V    K = 128, P from TMEM
// A pair of CTAs (tcgen05 cta_group::2, M = 256, N = 128) holds 128 rows of each
// query tile in each CTA, and of the keys and values each CTA half: 64 positions
// of a key tile, 64 columns of a value tile.  One CTA alone (M = 128) reads 8 KB
// of operands for the 64 cycles of a score product, all that shared memory gives;
// then every wait and every load held up the products: 2060 cycles a tile instead
// of the 1290 that they take, 2590 us for 1024 tokens over 32768 positions against
// the pair's 2180 (which reads 6 KB).
// One fp32 online softmax per token, a thread each: no shuffles.  While one
// query tile's scores are in the softmax the tensor cores work for the other;
// the first half of the keys' weights is multiplied while the second half is
// still being computed.  P overlays its scores, rounded to bf16 as a tensor-core
// operand (the row sum is of the fp32 weights).
// The list of items (a block and a head or two) is cut into one range of equal
// cost for each pair; what a cut leaves is joined by the next kernel.  (Whole items
// dealt out in turn: 128 for 74 pairs take two turns, 14% of the time idle.)
// Measured (clock stamps of every pair): 512 tokens over 6000 positions, 128 heads,
// 78 to 85 steps of two tiles a pair in 316,000 cycles: 195 us at 1.62 GHz (1.24
// PFLOP/s), 222 at 1.42; 1024 over 32768, 879 steps in 3.1 million cycles, 2000 us at
// 1.56 GHz, 2250 at 1.38: the power limit holds the clock.  What bounds the cycles is a
// tile's chain: 1480 of softmax (1024 of them its 128 exponentials a thread), about
// 400 until both CTAs' weights are known to the issuer, then its own products while
// the other tile's wait; two tiles take 3480 cycles, their products 2580, and the
// first two of an item 6900.  TMEM has no room for a third tile.
// Warps 0-3 and 4-7: softmax and output of tile 0 and 1; warp 8: queries and
// keys by TMA; warp 9: MMA (of the pair's first CTA); warp 10: values by TMA.
// TMEM: scores [0,128) [128,256), outputs [256,384) [384,512).
// ===========================================================================
namespace attn {
constexpr int Q_BYTES = 3 * kRows * 128;   // a query tile, in three columns of 64
constexpr int K_BYTES = 3 * 64 * 128;      // 64 positions
constexpr int V_BYTES = kRows * 128;       // 64 columns
constexpr int NK = 3, NV = 3;              // ring depths
constexpr int OFF_K = 2 * Q_BYTES;
constexpr int OFF_V = OFF_K + NK * K_BYTES;
constexpr int SMEM = OFF_V + NV * V_BYTES + 1024;
constexpr int THREADS = 384;  // (an idle warp completes the third register group)
// register split (168 per thread at launch): 2 x 208 + 88 = 3 x 168
constexpr int REGS_SOFT = 208, REGS_REST = 88;
static_assert(2 * REGS_SOFT + REGS_REST <= 3 * 168, "register split");
constexpr float kRescaleThreshold = 8.0f;  // log2 units
static_assert(SMEM + 512 <= 232448, "shared memory budget");

struct Bars {  // "first": waited on by the first CTA; "both": committed to both
  uint64_t q_full[2], q_free[2];     // first / both
  uint64_t k_full[NK], k_empty[NK];  // first / both
  uint64_t v_full[NV], v_empty[NV];  // first / both
  uint64_t s_full[2], o_full[2];     // both
  uint64_t p_full[2][2];             // first: by tile and half of the keys
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// A pair's work: items, or parts of the key tiles of its first and last.
struct Work {
  Block b;
  int i, j0, j1;  // item, key tiles [j0, j1)
  DEV bool whole() const { return j0 == 0 && j1 == b.tiles(1); }
  DEV int count(int t) const { return max(0, min(j1, b.tiles(t)) - j0); }  // of query tile t
};
struct Range {
  int g, j, ge, je;
  DEV Range(const Cut* cut, int pair) {
    g = cut[pair].g;
    j = cut[pair].j;
    ge = cut[pair + 1].g;
    je = cut[pair + 1].j;
  }
  DEV bool next(const Layout& ly, int per, Work* w) {
    if (g > ge || (g == ge && j >= je)) return false;
    w->b = ly.block[g / per];
    w->i = g % per;
    w->j0 = j;
    w->j1 = g == ge ? je : w->b.tiles(1);
    ++g;
    j = 0;
    return true;
  }
};

// What a pair leaves of an item that others work on too: by slot (0: the pair's
// first piece, of which it does not have the beginning; 1: its last), query
// tile and CTA, 128 rows of the normalised output and the log2 of the sum of
// exponentials.
constexpr int SLOT_ROWS = 4 * kRows;
struct Parts {
  __nv_bfloat16* o;  // [pairs][2][2][2][128][128]
  float* lse;        // [pairs][2][2][2][128]
  float* acc;        // [pairs][2 CTAs][2 tiles] x ACC: accumulators taken out of TMEM
};
constexpr int ACC = 128 * 128 + 2 * 128;  // [128 / 4 columns][128 rows][4], then maximum and sum of the rows
}  // namespace attn

// D (+)= A B with A in TMEM: each CTA of the pair its own rows at the same address
template <bool kAccumulate>
DEV void tc_mma2_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(kAccumulate ? 1 : 0)
      : "memory");
}

// This softmax thread's place in the copies of the accumulators: its row's
// columns, in pieces of four 128 apart, and its maximum and sum.
DEV float4* acc_of(float* acc) {
  return reinterpret_cast<float4*>(acc + (size_t)(blockIdx.x * 2 + (threadIdx.x >> 7)) * attn::ACC) +
         (threadIdx.x & 127);
}
DEV float2* acc_sum_of(float* acc) {
  return reinterpret_cast<float2*>(
             acc + (size_t)(blockIdx.x * 2 + (threadIdx.x >> 7)) * attn::ACC + 128 * 128) +
         (threadIdx.x & 127);
}
// Adds the row's output in TMEM and its sum, both relative to the maximum m, to
// the copies (which hold earlier runs if `more`).  Out of line: inlined it costs
// the loop over the tiles registers.
static __device__ __noinline__ void end_run(uint32_t to, float* acc, float m, float l, bool more) {
  float4* const dst = acc_of(acc);
  float a = 0.f;
  if (more) {
    const float2 ml = __ldcg(acc_sum_of(acc));
    a = ml.x == m ? 1.f : fast_exp2(ml.x - m);
    l += ml.y * a;
  }
#pragma unroll 1
  for (int c = 0; c < 128; c += 16) {
    uint32_t o[16];
    tmem_ld16(to + c, o);
    tc_wait_ld();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 v = more ? __ldcg(dst + (c / 4 + k) * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
      v.x = v.x * a + u2f(o[4 * k]);
      v.y = v.y * a + u2f(o[4 * k + 1]);
      v.z = v.z * a + u2f(o[4 * k + 2]);
      v.w = v.w * a + u2f(o[4 * k + 3]);
      __stcg(dst + (c / 4 + k) * 128, v);
    }
  }
  __stcg(acc_sum_of(acc), make_float2(m, l));
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(attn::THREADS, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_qr,
                 const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_r,
                 const __grid_constant__ CUtensorMap map_v, const Layout ly,
                 const attn::Parts parts, int head0, int heads, float scale_log2,
                 __nv_bfloat16* __restrict__ O, int32_t* status) {
  using namespace attn;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = paged::align1024(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  __shared__ Bars bars;
  volatile int* abort = &bars.abort;
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = heads / 2;  // items of a block
  if (warp == 9) tmem_alloc2(&bars.tmem_base, 512);
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.q_full[t], 1);
      mbar_init(&bars.q_free[t], 1);
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t][0], 8);  // four warps of each CTA
      mbar_init(&bars.p_full[t][1], 8);
      mbar_init(&bars.o_full[t], 1);
    }
    for (int i = 0; i < NK; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 1);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbarrier_init_cluster();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  pdl_wait();  // the keys and values
  pdl_trigger();
  const int pair = blockIdx.x >> 1;
  Range range(ly.cut, pair);
  Work w;

  if (warp == 11) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));  // (idle)
  } else if (warp == 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    // ---------------- queries and keys: each CTA its own, counted by the first ----------------
    const uint32_t q_full0 = mapa_shared(smem_u32(&bars.q_full[0]), 0);
    const uint32_t k_full0 = mapa_shared(smem_u32(&bars.k_full[0]), 0);
    int u = 0, qn[2] = {0, 0}, use = 0;  // use: key tiles of the item before
    bool ok = true;
    while (ok && range.next(ly, per, &w)) {
      const Block& b = w.b;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (w.count(t) == 0) continue;
        ok = ok && warp_wait(&bars.q_free[t], (qn[t] & 1) ^ 1, abort, status,
                             paged::queries_limit_ns(use));
        if (!ok) break;
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&bars.q_full[t], 2 * Q_BYTES);
          const uint32_t dst = sbase + t * Q_BYTES, bar = q_full0 + t * 8;
          const int h = head0 + b.head(t, w.i, heads);
          const int tok = b.tok + b.first(t) + rank * b.width();
          tma_load_3d_pair(dst, &map_qn, 0, h, tok, bar);
          tma_load_3d_pair(dst + Q_BYTES / 3, &map_qn, 64, h, tok, bar);
          tma_load_3d_pair(dst + Q_BYTES / 3 * 2, &map_qr, 0, h, tok, bar);
        }
        ++qn[t];
      }
      use = w.j1 - w.j0;
      const int two = b.two_heads();
      for (int j = w.j0; j < w.j1 && ok; ++j)
        for (int t = two ? 0 : 1; t < 2; ++t) {
          const int s = u % NK;
          ok = ok && warp_wait(&bars.k_empty[s], ((u / NK) & 1) ^ 1, abort, status);
          if (!ok) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&bars.k_full[s], 2 * K_BYTES);
            const uint32_t dst = sbase + OFF_K + s * K_BYTES;
            const int r = b.row + j * kRows + rank * 64;
            tma_load_3d_pair(dst, &map_k, 0, r, 2 * b.head(t, w.i, heads), k_full0 + s * 8);
            tma_load_2d_pair(dst + K_BYTES / 3 * 2, &map_r, 0, r, k_full0 + s * 8);
          }
          ++u;
        }
    }
    __syncwarp();
  } else if (warp == 10) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    // ---------------- values ----------------
    const uint32_t v_full0 = mapa_shared(smem_u32(&bars.v_full[0]), 0);
    int u = 0;
    bool ok = true;
    while (ok && range.next(ly, per, &w)) {
      const Block& b = w.b;
      const int two = b.two_heads();
      for (int j = w.j0; j < w.j1 && ok; ++j)
        for (int t = two ? 0 : 1; t < 2; ++t) {
          const int s = u % NV;
          ok = ok && warp_wait(&bars.v_empty[s], ((u / NV) & 1) ^ 1, abort, status);
          if (!ok) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&bars.v_full[s], 2 * V_BYTES);
            tma_load_3d_pair(sbase + OFF_V + s * V_BYTES, &map_v, 0, b.row + j * kRows,
                             2 * b.head(t, w.i, heads) + rank, v_full0 + s * 8);
          }
          ++u;
        }
    }
    __syncwarp();
  } else if (warp == 9) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    // ---------------- MMA ----------------
    if (rank == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(256, 128, 0, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32(256, 128, 0, 1);
      constexpr uint32_t hi128 = desc_hi(1024, kSwizzle128B);
      int u0 = 0;  // ring position of the item's first tile
      int qn[2] = {0, 0}, pn[2] = {0, 0};
      bool ok = true;
      // scores of query tile t and the key tile at ring position u; `done`: its
      // last use; `lastq`: the query tile's last use
      auto score = [&](int t, int u, bool done, bool lastq) {
        const int s = u % NK;
        ok = ok && warp_wait(&bars.k_full[s], (u / NK) & 1, abort, status);
        if (!ok) return;
        tc_fence_after();
        const uint32_t al = desc_lo(sbase + t * Q_BYTES, 16);
        const uint32_t bl = desc_lo(sbase + OFF_K + s * K_BYTES, 16);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma2(tmem + t * 128, desc_join(al + c * (Q_BYTES / 48) + ks * 2, hi128),
                      desc_join(bl + c * (K_BYTES / 48) + ks * 2, hi128), idesc_s,
                      (c > 0 || ks > 0) ? 1u : 0u);
          tc_commit2(&bars.s_full[t]);
          if (done) tc_commit2(&bars.k_empty[s]);
          if (lastq) tc_commit2(&bars.q_free[t]);
        }
        __syncwarp();
      };
      auto value = [&](int t, int u, bool first, bool done, bool last) {
        const int s = u % NV;
        ok = ok && warp_wait(&bars.v_full[s], (u / NV) & 1, abort, status);
        const uint32_t bl = desc_lo(sbase + OFF_V + s * V_BYTES, V_BYTES);
        const uint32_t d = tmem + 256 + t * 128, a = tmem + t * 128;
        ok = ok && warp_wait(&bars.p_full[t][0], pn[t] & 1, abort, status);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          if (first) tc_mma2_tmem_a<false>(d, a, desc_join(bl, hi128), idesc_o);
          else tc_mma2_tmem_a<true>(d, a, desc_join(bl, hi128), idesc_o);
#pragma unroll
          for (int ks = 1; ks < 4; ++ks)
            tc_mma2_tmem_a<true>(d, a + ks * 8, desc_join(bl + ks * (2048 >> 4), hi128), idesc_o);
        }
        __syncwarp();
        ok = warp_wait(&bars.p_full[t][1], pn[t] & 1, abort, status);
        ++pn[t];
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 4; ks < 8; ++ks)
            tc_mma2_tmem_a<true>(d, a + ks * 8, desc_join(bl + ks * (2048 >> 4), hi128), idesc_o);
          if (done) tc_commit2(&bars.v_empty[s]);
          if (last) tc_commit2(&bars.o_full[t]);
        }
        __syncwarp();
      };
      while (ok && range.next(ly, per, &w)) {
        const int nt[2] = {w.count(0), w.count(1)};  // nt[0] <= nt[1]
        const bool two = w.b.two_heads();
        const int per_j = two ? 2 : 1;
        auto at = [&](int t, int j) { return u0 + j * per_j + (two ? t : 0); };
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (nt[t] > 0 && ok) {
            ok = warp_wait(&bars.q_full[t], qn[t] & 1, abort, status);
            ++qn[t];
            score(t, at(t, 0), two || t == 1, nt[t] == 1);
          }
        for (int j = 0; j < nt[1] && ok; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (j < nt[t] && ok)
              value(t, at(t, j), j % kRun == 0, two || t == 1, j + 1 == nt[t]);
            if (j + 1 < nt[t] && ok) score(t, at(t, j + 1), two || t == 1, j + 2 == nt[t]);
          }
        u0 += nt[1] * per_j;
      }
      // everything issued so far has finished before TMEM is released
      if (elect_one()) tc_commit2(&bars.drain);
      __syncwarp();
      warp_wait(&bars.drain, 0, nullptr, status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
    // ---------------- softmax and output of tile t, thread = token ----------------
    const int t = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const uint32_t ts = tmem + ((uint32_t)(q4 * 32) << 16) + t * 128;
    const uint32_t to = ts + 256;
    const uint32_t p_full0 = mapa_shared(smem_u32(&bars.p_full[t][0]), 0);
    int sn = 0, on = 0;
    bool ok = true;
    const uint64_t scale2 = pack2(scale_log2, scale_log2);
    while (ok && range.next(ly, per, &w)) {
      const Block& b = w.b;
      const int nt = w.count(t), width = b.width();
      const int tok0 = b.first(t) + rank * width;  // this CTA's first token of the tile, in the block
      const int mine = min(min(b.n, b.first(t) + 2 * width) - tok0, width);
      const int lim0 = b.lim + tok0;            // positions that one sees
      const int lim = min(b.kv, lim0 + row);    // ... this thread's
      float m = -INFINITY;
      uint64_t la = 0, lb = 0;  // partial row sums
#pragma unroll 1
      for (int j = w.j0; j < w.j0 + nt; ++j) {
        ok = warp_wait(&bars.s_full[t], sn & 1, abort, status);
        ++sn;
        if (!ok) break;
        tc_fence_after();
        // (the scores are read again for their weights, in a loop: unrolled over the
        // tile the code of all roles would not stay in the instruction cache)
        float mt;
        {
          uint32_t s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s + c * 32);
          tc_wait_ld();
          if (min(b.kv, lim0) < (j + 1) * kRows) {
            const int left = lim - j * kRows;
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= left) s[c] = 0xff800000u;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tmem_st32(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(s + c * 32));
            tc_wait_st();
          }
          float mx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = fmaxf(u2f(s[e]), u2f(s[8 + e]));
#pragma unroll
          for (int c = 16; c < 128; c += 16)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = max3(mx[e], u2f(s[c + e]), u2f(s[c + 8 + e]));
          mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) *
               scale_log2;
        }
        if (j > w.j0 && (j - w.j0) % kRun == 0) {
          // a run ends: the output so far and its sum, relative to the maximum before
          // this tile, move to their copies
          float x, y;
          unpack2(add2(la, lb), x, y);
          end_run(to, parts.acc, m, x + y, j - w.j0 > kRun);
          la = lb = 0;
        }
        const bool raise = mt > m + kRescaleThreshold;
        if (__any_sync(0xffffffffu, raise)) {
          // (the value products before these scores have completed with them)
          const float a = raise ? fast_exp2(m - mt) : 1.f;  // 0 at the first tile
          if (j > w.j0) {
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + c, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = f2u(u2f(o[e]) * a);
              tmem_st32(to + c, o);
            }
            const uint64_t a2 = pack2(a, a);
            la = mul2(la, a2);
            lb = mul2(lb, a2);
          }
          if (raise) m = mt;
        }
        // (a token that has seen no position yet has m = -inf: its weights are exp2(-inf) = 0)
        const float d = m == -INFINITY ? 0.f : -m;
        const uint64_t d2 = pack2(d, d);
        auto weights = [&](const uint32_t* s, int c) {
          uint32_t w2[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x, y;
            unpack2(fma2(pack2(u2f(s[2 * e]), u2f(s[2 * e + 1])), scale2, d2), x, y);
            x = fast_exp2(x);
            y = fast_exp2(y);
            if (e & 1) la = add2(la, pack2(x, y));
            else lb = add2(lb, pack2(x, y));
            w2[e] = pack_bf16x2(x, y);
          }
          tmem_st16(ts + c * 16, w2);
        };
        uint32_t s0[32], s1[32];
        tmem_ld32(ts, s0);
        tc_wait_ld();
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          tmem_ld32(ts + (c + 1) * 32, s1);
          weights(s0, c);
          tc_wait_ld();
          if (c == 0) tmem_ld32(ts + 64, s0);
          weights(s1, c + 1);
          tc_wait_ld();
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(p_full0 + (c >> 1) * 8);
        }
      }
      if (!ok) break;
      const bool moved = nt > kRun;  // earlier runs' part is in the copy
      float inv = 0.f, l = 0.f, a = 0.f;
      if (nt > 0) {
        float x, y;
        unpack2(add2(la, lb), x, y);
        l = x + y;
        if (moved) {
          const float2 ml = __ldcg(acc_sum_of(parts.acc));
          a = ml.x == m ? 1.f : fast_exp2(ml.x - m);
          l += ml.y * a;
        }
        inv = l == 0.f ? 0.f : 1.f / l;
        ok = warp_wait(&bars.o_full[t], on & 1, abort, status);
        ++on;
        if (!ok) break;
        tc_fence_after();
      }
      __nv_bfloat16* dst;
      bool store = row < mine;
      if (w.whole()) {
        dst = O + ((size_t)(b.tok + tok0 + row) * kH + head0 + b.head(t, w.i, heads)) * kD;
      } else {
        const size_t at = (size_t)(pair * 2 + (w.j0 > 0 ? 0 : 1)) * SLOT_ROWS +
                          (t * 2 + rank) * kRows + row;
        parts.lse[at] = l == 0.f ? -INFINITY : m + log2f(l);
        dst = parts.o + at * kD;
        store = store && nt > 0;
      }
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld32(to + c, o);
          tc_wait_ld();
        }
        if (moved) {
          const float4* const src = acc_of(parts.acc);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 v = __ldcg(src + (c / 4 + k) * 128);
            o[4 * k] = f2u(u2f(o[4 * k]) + v.x * a);
            o[4 * k + 1] = f2u(u2f(o[4 * k + 1]) + v.y * a);
            o[4 * k + 2] = f2u(u2f(o[4 * k + 2]) + v.z * a);
            o[4 * k + 3] = f2u(u2f(o[4 * k + 3]) + v.w * a);
          }
        }
        if (store) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (lim > 0)
              v = make_uint4(pack_bf16x2(u2f(o[8 * e]) * inv, u2f(o[8 * e + 1]) * inv),
                             pack_bf16x2(u2f(o[8 * e + 2]) * inv, u2f(o[8 * e + 3]) * inv),
                             pack_bf16x2(u2f(o[8 * e + 4]) * inv, u2f(o[8 * e + 5]) * inv),
                             pack_bf16x2(u2f(o[8 * e + 6]) * inv, u2f(o[8 * e + 7]) * inv));
            *reinterpret_cast<uint4*>(dst + c + 8 * e) = v;
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // a warp that gave up may leave loads in flight, which land within
    // microseconds: a millisecond before the pair leaves
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000) {
    }
  }
  cluster_sync_all();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
  cluster_sync_all();  // neither CTA leaves before both have released
}

// ===========================================================================
// join_kernel: the outputs of the items that several pairs worked on,
//   O = sum_s 2^(lse_s - max) O_s / sum_s 2^(lse_s - max)
// Grid (pairs - 1 boundaries, query tile and CTA, four groups of 32 rows); a
// boundary that cuts no item, or one that an earlier boundary cuts too, has
// nothing to do.  256 threads: a row's sixteen 16-byte pieces.
// ===========================================================================
__global__ void __launch_bounds__(256) join_kernel(const Layout ly, const attn::Parts parts,
                                                    int pairs, int head0, int heads,
                                                    __nv_bfloat16* __restrict__ O) {
  using namespace attn;
  pdl_trigger();
  // the layout, complete before the attention let this kernel start (not through L1)
  auto cut_at = [&](int i) {
    const int2 v = __ldcg(reinterpret_cast<const int2*>(ly.cut + i));
    return Cut{v.x, v.y};
  };
  const int c = blockIdx.x + 1, t = blockIdx.y >> 1, rank = blockIdx.y & 1;
  const Cut cut = cut_at(c), before = cut_at(c - 1);
  const bool mine_to_do = cut.j > 0 && !(before.g == cut.g && before.j > 0);
  const int per = heads / 2;
  // The pairs that hold a piece of the item, in its order.  Not all from the first
  // to the last do: with less work than pairs neighbouring cuts coincide, and the
  // pair between them has nothing and writes nothing.
  __shared__ int piece[kPairs], pieces;
  Block b = {};
  if (mine_to_do) {
    if (threadIdx.x == 0) {
      int n = 0;
      piece[n++] = c - 1;
      Cut at = cut;
      for (int s = c; s < pairs && at.g == cut.g && at.j > 0; ++s) {
        const Cut next = cut_at(s + 1);
        if (next.g != at.g || next.j != at.j) piece[n++] = s;
        at = next;
      }
      pieces = n;
    }
    static_assert(sizeof(Block) == 24 && sizeof(Cut) == 8, "read in pairs of words");
    const int2* src = reinterpret_cast<const int2*>(ly.block + cut.g / per);
    const int2 x = __ldcg(src), y = __ldcg(src + 1), z = __ldcg(src + 2);
    b = {x.x, x.y, y.x, y.y, z.x, z.y};
  }
  __syncthreads();
  // every block waits: the kernel after this one relies on it
  pdl_wait();
  if (!mine_to_do) return;
  const int n = pieces;  // two or more
  const int w = b.width(), tok0 = b.first(t) + rank * w;
  const int mine = min(min(b.n, b.first(t) + 2 * w) - tok0, w);
  const int head = head0 + b.head(t, cut.g % per, heads);
  auto at = [&](int k, int row) {  // piece k: the first is its pair's last, the others their pairs' first
    return (size_t)(piece[k] * 2 + (k == 0 ? 1 : 0)) * SLOT_ROWS + (t * 2 + rank) * kRows + row;
  };
  const int chunk = threadIdx.x & 15;
  const int r0 = blockIdx.z * 32 + (threadIdx.x >> 4);  // rows r0 and r0 + 16
  // the first two pieces (mostly all) with their sums, before anything waits for them
  float l[2][2];
  uint4 v[2][2];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const size_t x = at(k, r0 + 16 * r);
      l[r][k] = parts.lse[x];
      v[r][k] = ld_global_nc_v4(parts.o + x * kD + chunk * 8);
    }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = r0 + 16 * r;
    if (row >= mine) continue;
    float top = fmaxf(l[r][0], l[r][1]);
    for (int k = 2; k < n; ++k) top = fmaxf(top, parts.lse[at(k, row)]);
    float sum = 0.f, acc[8] = {};
    auto add = [&](float lse, const uint4& o) {
      if (lse == -INFINITY) return;  // (its output is not written)
      const float f = exp2f(lse - top);
      const uint32_t p[4] = {o.x, o.y, o.z, o.w};
      sum += f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e] += f * u2f(p[e] << 16);
        acc[2 * e + 1] += f * u2f(p[e] & 0xffff0000u);
      }
    };
    add(l[r][0], v[r][0]);
    add(l[r][1], v[r][1]);
    for (int k = 2; k < n; ++k) {
      const size_t x = at(k, row);
      add(parts.lse[x], ld_global_nc_v4(parts.o + x * kD + chunk * 8));
    }
    const float inv = sum > 0.f ? 1.f / sum : sum;  // (0: the token sees nothing; NaN stays)
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    *reinterpret_cast<uint4*>(O + ((size_t)(b.tok + tok0 + row) * kH + head) * kD + chunk * 8) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ===========================================================================
// host
// ===========================================================================

// The first part of a workspace: the layout and the gathered rows.
struct RowsWs {
  size_t row, kv, block, start, cut, rows, total;
  int64_t max_rows;
};

static RowsWs rows_ws(int N, int S, int max_kv) {
  RowsWs w;
  // (a pair's second CTA may reach 128 rows past the last sequence)
  w.max_rows = (int64_t)S * ((max_kv + kRows - 1) / kRows * kRows);
  w.max_rows = (w.max_rows + 2 * kRows - 1) / (2 * kRows) * (2 * kRows);
  w.row = 0;
  w.kv = round_up((size_t)(S + 1) * 4, 256);
  w.block = round_up(w.kv + (size_t)S * 4, 256);
  w.start = round_up(w.block + ((size_t)N / kTile + S) * sizeof(Block), 256);
  w.cut = round_up(w.start + ((size_t)N / kTile + S) * 4, 256);
  w.rows = round_up(w.cut + (kPairs + 1) * sizeof(Cut), 256);
  w.total = round_up(w.rows + (size_t)w.max_rows * MLA_ROW * 2, 256);
  return w;
}

struct Ws {
  RowsWs r;
  size_t k, v, parts, lse, acc, total;
  int heads;  // of a group
};

// (By the bound, which is all the host knows: under one far above the lengths the
// groups are small and what a group costs at least shows.  256 tokens over 1500
// positions: 110 us under a bound of 65,536 positions, 150 under 131,072, 193 under
// 262,144, 596 from 524,289 on, where sixteen groups of eight heads follow each other.)
static Ws layout(int N, int S, int max_kv) {
  Ws w;
  w.r = rows_ws(N, S, max_kv);
  w.heads = kH;
  while (w.heads > 8 && (size_t)w.r.max_rows * w.heads * 2 * kD * 2 > kGroupBytes) w.heads /= 2;
  w.k = w.r.total;
  w.v = w.k + (size_t)w.r.max_rows * w.heads * kD * 2;
  w.parts = w.v + (size_t)w.r.max_rows * w.heads * kD * 2;
  w.lse = w.parts + (size_t)kPairs * 2 * attn::SLOT_ROWS * kD * 2;
  w.acc = w.lse + (size_t)kPairs * 2 * attn::SLOT_ROWS * 4;
  w.total = w.acc + (max_kv > kRun * kRows ? (size_t)kPairs * 4 * attn::ACC * 4 : 0);
  return w;
}

bool fits(int S, int max_kv, int64_t rows) {
  return (int64_t)S * ((max_kv + kRows - 1) / kRows * kRows) <= rows;
}

size_t workspace_bytes(int N, int S, int max_kv) { return layout(N, S, max_kv).total; }

static Layout make_layout(const RowsWs& w, uint8_t* ws) {
  Layout ly;
  ly.row = reinterpret_cast<int32_t*>(ws + w.row);
  ly.kv = reinterpret_cast<int32_t*>(ws + w.kv);
  ly.block = reinterpret_cast<Block*>(ws + w.block);
  ly.start = reinterpret_cast<int32_t*>(ws + w.start);
  ly.cut = reinterpret_cast<Cut*>(ws + w.cut);
  return ly;
}

static int pairs_of(int sms) { return sms / 2 < kPairs ? sms / 2 : kPairs; }

// layout_kernel and gather_kernel
static int gather_rows(const RowsWs& w, const Pool& pool, const Seqs& q, uint8_t* ws,
                       int32_t* table, int max_pages, int heads, int sms, int32_t* status,
                       cudaStream_t st) {
  const Layout ly = make_layout(w, ws);
  __nv_bfloat16* rows = reinterpret_cast<__nv_bfloat16*>(ws + w.rows);
  layout_kernel<<<1, 1024, 0, st>>>(q, pool, ly, heads / 2, pairs_of(sms));
  if (int e = launch_status()) return e;
  const int64_t want = (w.max_rows + 7) / 8;
  const int blocks = (int)(want < sms * 32 ? want : sms * 32);
  if (pool.kind == MLA_PAGE_E4M3)
    return launch_pdl(gather_kernel<true>, dim3(blocks), dim3(256), 0, st, pool, ly, q.S, rows,
                      table, max_pages, status);
  return launch_pdl(gather_kernel<false>, dim3(blocks), dim3(256), 0, st, pool, ly, q.S, rows,
                    table, max_pages, status);
}

static int staged_pages(int max_kv) {
  return (max_kv + kRows - 1) / kRows * (kRows / kStagedPage);
}

size_t staged_bytes(int N, int S, int max_kv) {
  return rows_ws(N, S, max_kv).total + round_up((size_t)S * staged_pages(max_kv) * 4, 256);
}

int stage(const Pool& pool, const Seqs& q, uint8_t* ws, int32_t* status, cudaStream_t st,
          Pool* staged) {
  const RowsWs w = rows_ws(q.N, q.S, q.max_kv);
  int sms = 0;
  if (int e = check_device(&sms)) return e;
  int32_t* table = reinterpret_cast<int32_t*>(ws + w.total);
  staged->base = ws + w.rows;
  staged->kind = MLA_PAGE_BF16;
  staged->num_pages = (int)(w.max_rows / kStagedPage);
  staged->page_size = staged->pitch = kStagedPage;
  staged->row_stride = MLA_ROW * 2;
  staged->rows = (int)w.max_rows;
  staged->table = table;
  staged->max_pages = staged_pages(q.max_kv);
  paged::set_division(staged);
  return gather_rows(w, pool, q, ws, table, staged->max_pages, 2, sms, status, st);
}

int run(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
        const paged::Pool& pool, const paged::Seqs& q, float scale, mla_bf16_t* O, uint8_t* ws,
        int32_t* status, cudaStream_t st) {
  const Ws L = layout(q.N, q.S, q.max_kv);
  int sms = 0;
  if (int e = check_device(&sms)) return e;
  if (int e = gather_rows(L.r, pool, q, ws, nullptr, 0, L.heads, sms, status, st)) return e;
  const Layout ly = make_layout(L.r, ws);
  __nv_bfloat16* rows = reinterpret_cast<__nv_bfloat16*>(ws + L.r.rows);
  __nv_bfloat16* k = reinterpret_cast<__nv_bfloat16*>(ws + L.k);
  __nv_bfloat16* v = reinterpret_cast<__nv_bfloat16*>(ws + L.v);

  alignas(64) CUtensorMap map_c, map_w, map_sk, map_k, map_v, map_r, map_qn, map_qr;
  const uint64_t R = (uint64_t)L.r.max_rows;
  if (int e = bf16_map_2d(&map_c, rows, kC, R, MLA_ROW * 2, 64, kRows)) return e;
  if (int e = bf16_map_2d(&map_w, wkv_b, kC, kH * 256, kC * 2, 64, 128)) return e;
  // keys and values: [head][half of the columns][row][64]
  if (int e = bf16_map_3d(&map_sk, k, 64, R, 2 * L.heads, 128, R * 128, 64, kRows, 1)) return e;
  if (int e = bf16_map_3d(&map_k, k, 64, R, 2 * L.heads, 128, R * 128, 64, 64, 2)) return e;
  if (int e = bf16_map_3d(&map_v, v, 64, R, 2 * L.heads, 128, R * 128, 64, kRows, 1)) return e;
  if (int e = bf16_map_2d(&map_r, rows + kC, kR, R, MLA_ROW * 2, 64, 64)) return e;
  if (int e = bf16_map_3d(&map_qn, q_nope, kD, kH, q.N, kD * 2, kH * kD * 2, 64, 1, kRows))
    return e;
  if (int e = bf16_map_3d(&map_qr, q_pe, kR, kH, q.N, kR * 2, kH * kR * 2, 64, 1, kRows)) return e;
  static std::atomic<unsigned long long> gemm_attr{0}, attn_attr{0};
  if (int e = ensure_smem_attr(expand_kernel, gemm::SMEM, &gemm_attr)) return e;
  if (int e = ensure_smem_attr(chunk_kernel, attn::SMEM, &attn_attr)) return e;
  const dim3 grid(2 * (sms / 2));
  const int pairs = pairs_of(sms);
  const attn::Parts parts = {reinterpret_cast<__nv_bfloat16*>(ws + L.parts),
                             reinterpret_cast<float*>(ws + L.lse),
                             reinterpret_cast<float*>(ws + L.acc)};
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(O);
  for (int h0 = 0; h0 < kH; h0 += L.heads) {
    if (int e = launch_pdl(expand_kernel, grid, dim3(gemm::THREADS), gemm::SMEM, st, map_c, map_w,
                           map_sk, map_v, (const int32_t*)(ly.row + q.S), h0, L.heads, status))
      return e;
    if (int e = launch_pdl(chunk_kernel, dim3(2 * pairs), dim3(attn::THREADS), attn::SMEM, st,
                           map_qn, map_qr, map_k, map_r, map_v, ly, parts, h0, L.heads,
                           scale * 1.4426950408889634f, out, status))
      return e;
    // (no item is cut that has fewer key tiles than two pieces)
    if (q.max_kv > (2 * kMinPiece - 1) * kRows && pairs > 1)
      if (int e = launch_pdl(join_kernel, dim3(pairs - 1, 4, 4), dim3(256), 0, st, ly, parts, pairs,
                             h0, L.heads, out))
        return e;
  }
  return MLA_OK;
}

}  // namespace expand
}  // namespace shla
