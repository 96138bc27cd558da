// Attention of new tokens over a paged latent cache, absorbed form.  For each
// new token and head h, over the positions t < lim the token sees:
//   q~ = q_nope W_UK[h];  s_t = (q~ . c_t + q_pe . kpe_t) * scale
//   O = W_UV[h] (softmax(s) c)
// Five kernels on the caller's stream:
//
//   (fold)           q~ per head, as in mla_decode
//   plan_kernel      one block, while the fold runs: each token's sequence and
//                    limit, the prefix sum of the tokens' 128-key tiles, its cut
//                    into one range of equal cost per CTA pair, and the list of
//                    tokens that a cut splits
//   absorbed_kernel  persistent CTA pairs over their ranges
//   merge_kernel     log-sum-exp merge of the tokens that several pairs held
//   value_kernel     O = W_UV O~ per head
#include <math.h>

#include "attend_paged.cuh"
#include "expand.h"
#include "fold.h"
#include "pair.cuh"
#include "tma_map.h"

namespace shla {
namespace paged {

// ===========================================================================
// plan
// ===========================================================================

constexpr int KT = 128;  // keys per tile
// Fixed cost of a token in tiles: its query load and its output's write-out.
constexpr int kTokenCost = 2;

struct Plan {
  int32_t* seq;     // [N] sequence of each token
  int32_t* lim;     // [N] positions it sees
  int32_t* tstart;  // [N + 1] its first tile in the flattened list
  int32_t* tb;      // [nc + 1] first tile of each pair's range
  int32_t* crow;    // [nc + 1] the token that holds that tile
  int32_t* split;   // [nc] pairs after whose range a token is cut for the first time
  int32_t* nact;    // [2] tokens of the sequences (those behind the last one are padding); entries of split
};

constexpr int kMaxPairs = 512;

// Every token has at least one tile, so that one that sees nothing still gets
// its zero output.
__global__ void __launch_bounds__(1024) plan_kernel(const Seqs q, const Pool pool, const Plan pl,
                                                     int nc) {
  __shared__ int part[1024];
  __shared__ int tb_s[kMaxPairs + 1], nsplit;
  const int tid = threadIdx.x;
  pdl_trigger();
  const int nact = min(q.N, q.q0(q.S));
  const int per = (nact + 1023) / 1024;
  const int lo = min(nact, tid * per), hi = min(nact, lo + per);
  int sum = 0;
  if (lo < hi) {
    // the last sequence that starts at or before token lo
    int a = 0, e = q.S;
    while (e - a > 1) {
      const int m = (a + e) >> 1;
      if (q.q0(m) <= lo) a = m; else e = m;
    }
    int begin = q.q0(a), end = q.q0(a + 1), kv = q.kv(a, pool);
    for (int r = lo; r < hi; ++r) {
      while (r >= end && a + 1 < q.S) {
        ++a;
        begin = q.q0(a);
        end = q.q0(a + 1);
        kv = q.kv(a, pool);
      }
      const int lim = max(0, min(kv, kv - (end - begin) + (r - begin) + 1));
      pl.seq[r] = a;
      pl.lim[r] = lim;
      sum += max(1, (lim + KT - 1) / KT);
    }
  }
  part[tid] = sum;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int v = tid >= o ? part[tid - o] : 0;
    __syncthreads();
    part[tid] += v;
    __syncthreads();
  }
  int run = part[tid] - sum;
  for (int r = lo; r < hi; ++r) {
    pl.tstart[r] = run;
    run += max(1, (pl.lim[r] + KT - 1) / KT);
  }
  const int tot = part[1023];
  for (int r = nact + tid; r <= q.N; r += 1024) pl.tstart[r] = tot;
  if (tid == 0) {
    pl.nact[0] = nact;
    nsplit = 0;
  }
  __syncthreads();  // tstart, written by the block, is visible to it
  // Cost units: token r spans kTokenCost units of its own, then one per tile,
  // from u(r) = tstart[r] + r * kTokenCost.  Pair c takes the units
  // [c U / nc, (c + 1) U / nc); a range that starts in a token's own units
  // starts at its first tile.
  const long long U = (long long)tot + (long long)nact * kTokenCost;
  int mine = -1;  // the token that holds the first tile of this thread's range (nc < 1024)
  if (tid <= nc) {
    const int c = tid;
    int t = tot, b = nact;
    if (c < nc && nact > 0) {
      const long long u = (long long)c * U / nc;
      int a = 0, e = nact;  // u(a) <= u < u(e)
      while (e - a > 1) {
        const int m = (a + e) >> 1;
        if ((long long)pl.tstart[m] + (long long)m * kTokenCost <= u) a = m; else e = m;
      }
      const long long into = u - ((long long)pl.tstart[a] + (long long)a * kTokenCost);
      t = pl.tstart[a] + (into > kTokenCost ? (int)(into - kTokenCost) : 0);
      b = a;
      mine = a;
    }
    pl.tb[c] = tb_s[c] = t;
    pl.crow[c] = b;
  }
  __syncthreads();
  // boundary c cuts its token, and no earlier one does (the order of the list
  // changes nothing but the order of the merge's work)
  if (mine >= 0 && tid > 0) {
    const int rs = pl.tstart[mine];
    if (rs < tb_s[tid] && tb_s[tid - 1] <= rs) pl.split[atomicAdd(&nsplit, 1)] = tid;
  }
  __syncthreads();
  if (tid == 0) pl.nact[1] = nsplit;
  // the fold before this kernel has finished too when it has
  pdl_wait();
}

// ===========================================================================
// absorbed_kernel: persistent CTA pairs (tcgen05 cta_group::2)
//
// A token's fp32 accumulator, 128 heads x 512 latent columns, is a CTA's whole
// TMEM.  So a pair shares a token: CTA r has heads [64r, +64), whose 64 rows of
// scores and of output a pair's M = 128 product leaves in its own TMEM, each
// row in two lanes: lane h the first half of the columns, lane 64 + h the
// second.  No score ever crosses between the CTAs.  Per tile of 128 keys:
//   S = Q~ K^T   M = 128, N = 128 keys, K = 576.  A: 64 rows of Q~ in each CTA.
//                B: CTA r holds keys [64r, +64), all 576 columns.
//   O += P V     M = 128, N = 2 x 256, K = 128 keys.  A: 64 rows of P in each
//                CTA.  B: CTA r holds all 128 keys' latent columns [256r, +256),
//                read MN-major.
// A row's two lanes hold 64 keys' scores each; they agree on the maximum
// through shared memory.  fp32 online softmax: the running maximum is raised
// only once a tile exceeds it by more than 8 log2 units; P = 2^(s-m) is rounded
// to bf16 as a tensor-core operand (its row sum is of the fp32 P).
//
// Bounds, per tile and pair: 147 KB of cache (1.67 us at the measured copy rate
// for 16-bit pages), 2228 cycles of products (measured alone, and not slower
// with the loads running: 36 x 33 + 16 x 65; 1.16 us at 1.92 GHz).  Shared
// memory holds one tile of keys and one of values, in three chunks of 192
// columns and two of 64 keys, each reloaded as soon as its products are done:
// the next tile's first chunk lands while this tile's last is in use, so the
// reload waits neither for the softmax nor for the rest of the tile.
// Measured (clock stamps of every pair): 64 sequences of 1000 to 8000 positions,
// 16-bit pages, one token each: 82 us for 348 MB (4.2 TB/s; 55% of the tensor pipe's
// cycles), 28 to 33 tiles a pair in 132,000 cycles at 1.68 GHz: 15,000 until the first
// tile's values are multiplied, 3200 a tile after another of the same token (3600
// with the slow ones), 9300 where the token changes, 6400 from the last tile to the
// end.  What a tile takes beyond its products is its chain from scores to weights to
// values and the reload of its keys.  8-bit pages, 128 sequences up to 16000: 444 us,
// 114 to 120 tiles a pair in 803,000 cycles, 6700 a tile, 14,500 at a change.
// There a tile's place in shared memory is filled by the converting warps, and
// waiting for the place, loading, converting (50 of 280 us, with four tokens each),
// storing (40) and the softmax add up; tiles of 64 keys with two places took longer.
// (Two rings of 64-key tiles took 2450 cycles a 64-key tile, waiting for the
// reload of keys.  A pair that splits the latent for the scores too holds each
// value once but must exchange 32 KB of partial scores per 64 keys; st.async
// moves them at 23 bytes a cycle while the SM's other shared-memory accesses
// wait: 3600 cycles.)
//
// Roles (640 threads a CTA; 896 for 8-bit pages, which have eight warps for keys
// and eight for values):
//   warps 0-7    softmax, two groups of four warps that take every other tile, a
//                lane of TMEM per thread.  The running maximum goes from group
//                to group (published as soon as a tile's is known, before its
//                exponentials); row sums stay with the group until the token ends.
//   warps 8-11   keys; 12-15 values.  16-bit pages: a warp for each chunk, TMA (one
//                warp for all chunks took 700 cycles for each, in turn).  8-bit:
//                loads, exact conversion to bf16 and swizzled stores.
//   then one warp each that issues the score products (first CTA; TMEM owner),
//                loads queries (TMA), issues the value products (first CTA) and
//                loads the rotary keys of 8-bit pages (TMA)
// TMEM (512 columns): four score tiles [0,256), output [256,512).
// ===========================================================================

constexpr int HH = kH / 2;             // heads of a CTA
constexpr int NSB = 4;                 // score tiles in TMEM (64 columns each)
constexpr int NKC = 3;                 // chunks of a tile's keys (192 columns); values: two of 64 keys
constexpr int Q_ATOM = HH * 128;       // 64 columns of 64 rows, 128 B swizzle
constexpr int K_ATOM = KT / 2 * 128;   // 64 columns of this CTA's 64 keys
constexpr int V_ATOM = 64 * 128;       // 64 columns of a chunk's 64 keys
constexpr int Q_BYTES = 9 * Q_ATOM, K_BYTES = 9 * K_ATOM, V_CHUNK = 4 * V_ATOM;
constexpr int P_BYTES = HH * 128;      // 64 rows of 64 weights
constexpr int OFF_K = Q_BYTES;
constexpr int OFF_V = OFF_K + K_BYTES;
constexpr int OFF_P = OFF_V + 2 * V_CHUNK;
constexpr int SMEM_BYTES = OFF_P + 2 * P_BYTES;
constexpr uint32_t T_S = 0, T_O = 256, TMEM_COLS = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int ACC = 128 * 256 + 128;  // [256 / 4 columns][128 lanes][4], then the lanes' maxima
static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_P % 1024 == 0, "alignment");
static_assert(T_S + NSB * KT / 2 <= T_O, "TMEM plan");
constexpr int KEY_WARP0 = 8;
template <bool kE4M3>
struct Roles {
  static constexpr int load_warps = kE4M3 ? 8 : 4;  // of keys, and of values
  static constexpr int val0 = KEY_WARP0 + load_warps, s = val0 + load_warps, q = s + 1, o = s + 2, rope = s + 3;
  static constexpr int threads = 32 * (s + 4);
  // registers: an equal share at launch, then by role (in groups of four warps)
  static constexpr int groups = threads / 128, share = 65536 / threads / 8 * 8;
  static constexpr int soft = kE4M3 ? 80 : 128, load = kE4M3 ? 72 : 80, rest = kE4M3 ? 56 : 64;
  static_assert(2 * soft + load_warps / 2 * load + rest <= groups * share, "register split");
};

struct Params {
  const __nv_bfloat16* q_tilde;  // [N][128][512]
  const __nv_bfloat16* q_pe;     // [N][128][64]
  Pool pool;
  Plan plan;
  int N;
  int box;                       // rows of a TMA box that no page boundary cuts (64, 32, 16; 0: none)
  float scale_log2;              // softmax scale * log2(e)
  __nv_bfloat16* opart;          // [pairs][2 slots][128][512], normalised per segment
  float* lse;                    // [pairs][2 slots][128], log2 units of scaled scores
  __nv_bfloat16* omerged;        // [N][128][512]
  float* acc;                    // [pairs][2 CTAs] x ACC: accumulators taken out of TMEM
  int32_t* status;
};

// "first CTA": waited on by the issuer only, arrived on from both CTAs;
// "both": committed to both CTAs by the issuer; the others are each CTA's own
struct alignas(16) Bars {
  uint64_t q_full, q_free;           // first CTA / both
  uint64_t k_full[NKC], k_empty[NKC];  // first CTA / both
  uint64_t v_full[2];                // by half of the keys (two chunks)
  uint64_t s_full[NSB];              // both: scores of tile i in buffer i % NSB
  uint64_t s_empty[NSB];             // first CTA: ... read by all softmax warps
  uint64_t p_full[2][2];             // first CTA, by group: [0] first half of P written and all of O
                                     // free to be added to, [1] second half written
  uint64_t pv_done[2][2];            // both: tile i's value products of a half of the keys done, by
                                     // i & 1 and half: their P and values are free; [.][1]: O~ holds tile i
  uint64_t m_full[2][4];             // running maxima after tile i, by group and lane quarter
  uint64_t x_full[2][2];             // tile maxima of both lanes of a row (by quarter & 1)
  uint64_t l_full[2][4];             // row sums after tile i
  uint64_t flushed[4];               // a token's output has left TMEM, by lane quarter
  uint64_t drain[2];                 // both
  uint32_t tmem_base;
  int abort;
  // by group: running maxima of the heads, tile maxima and row sums of the lanes
  float m[2][HH], x[2][128], l[2][128];
};

static_assert((sizeof(Bars) + 1023) / 1024 * 1024 + SMEM_BYTES <= 232448,
              "shared memory budget");

// Dynamic shared memory: the operands from the first 1024-byte boundary after
// the kernel's static part, which is Bars.
static constexpr int dynamic_smem() {
  return SMEM_BYTES + (1024 - (int)(sizeof(Bars) % 1024)) % 1024;
}

struct Pos {
  int bb, jt, nr;  // token, tile within it, its tile count
};

template <bool kE4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Roles<kE4M3>::threads, 1)
    absorbed_kernel(const Params p, const __grid_constant__ CUtensorMap map_qt,
                    const __grid_constant__ CUtensorMap map_qr,
                    const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v,
                    const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_1) {
  using R = Roles<kE4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ Bars bars;
  volatile int* abort = &bars.abort;

  // (the static part begins on such a boundary; were it not so, nothing runs)
  if (smem + SMEM_BYTES > smem_raw + dynamic_smem()) {
    report_timeout(p.status);
    return;
  }
  const uint32_t rank = cluster_ctarank();
  const int cid = blockIdx.x >> 1;
  pdl_wait();  // the plan, and the fold before it
  const int t_begin = ld_global_nc_s32_early(p.plan.tb + cid);
  const int n = ld_global_nc_s32_early(p.plan.tb + cid + 1) - t_begin;
  const int bb0 = min(ld_global_nc_s32_early(p.plan.crow + cid), p.N - 1);
  const int jt0 = t_begin - ld_global_nc_s32_early(p.plan.tstart + bb0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  const uint32_t sbase = smem_u32(smem);
  // (one past the last token only where the range ends: any count will do)
  auto tiles_of = [&](int bb) {
    return bb < p.N ? ld_global_nc_s32_early(p.plan.tstart + bb + 1) -
                          ld_global_nc_s32_early(p.plan.tstart + bb)
                    : 1;
  };
  auto lim_of = [&](int bb) { return bb < p.N ? ld_global_nc_s32_early(p.plan.lim + bb) : 0; };
  // a barrier of the pair's first CTA
  auto first_cta = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };

  if (warp == R::s) tmem_alloc2(&bars.tmem_base, TMEM_COLS);
  if (tid == 0) {
    constexpr int fill = kE4M3 ? 2 * Roles<true>::load_warps : 1;  // warps of both CTAs, or one arrival and bytes
    constexpr int rope_fill = kE4M3 ? 1 : 0;  // (the last chunk also a box of rotary keys)
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q_free, 1);
    for (int i = 0; i < NKC; ++i) {
      mbar_init(&bars.k_full[i], fill + (i == NKC - 1 ? rope_fill : 0));
      mbar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.p_full[i][0], 8);  // the four warps of a group in each CTA
      mbar_init(&bars.p_full[i][1], 4);  // the two of the second half
      mbar_init(&bars.v_full[i], kE4M3 ? Roles<true>::load_warps : 1);
      mbar_init(&bars.pv_done[i][0], 1);
      mbar_init(&bars.pv_done[i][1], 1);
      mbar_init(&bars.x_full[i][0], 2);
      mbar_init(&bars.x_full[i][1], 2);
      for (int q = 0; q < 4; ++q) {
        mbar_init(&bars.m_full[i][q], 1);
        mbar_init(&bars.l_full[i][q], 1);
      }
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_empty[i], 8);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&bars.flushed[q], 1);
    mbar_init(&bars.drain[0], 1);
    mbar_init(&bars.drain[1], 1);
    bars.abort = 0;
    fence_mbarrier_init_cluster();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  // (through a shuffle: the compiler then keeps it in a uniform register, as the
  // products want it)
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem_base, 0);

  if (n <= 0) {
    // an empty range (fewer tiles than pairs): nothing to do
  } else if (warp >= KEY_WARP0 && warp < R::s) {
    // ---------------- keys and values ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::load));
    const bool val = warp >= R::val0;
    const int wl = warp - (val ? R::val0 : KEY_WARP0);
    int bb = bb0, jt = jt0 - 1, nr = tiles_of(bb0), lim = 0, bad = 0;
    const int32_t* trow = nullptr;
    bool last = false;  // the token sees all its sequence's positions: count its bad pages
    auto enter = [&]() {
      if (bb >= p.N) return;
      const int s = ld_global_nc_s32_early(p.plan.seq + bb);
      lim = lim_of(bb);
      trow = p.pool.table + (long long)s * p.pool.max_pages;
      last = bb + 1 >= ld_global_nc_s32_early(p.plan.nact) ||
             ld_global_nc_s32_early(p.plan.seq + bb + 1) != s;
    };
    auto advance = [&]() {  // to the next tile
      if (++jt == nr) {
        jt = 0;
        nr = tiles_of(++bb);
        enter();
      }
    };
    // the pool row of position k, whose page is pg; an entry outside the pool
    // counts once for each page of a sequence
    auto row_at = [&](int pg, int k, bool count) {
      const bool in = pg >= 0 && pg < p.pool.num_pages;
      const int off = k - page_of(p.pool, k) * p.pool.page_size;
      if (count && !in && off == 0) ++bad;
      return in ? pg * p.pool.pitch + off : p.pool.rows;
    };
    enter();
    if constexpr (!kE4M3) {
      const int chunk = wl;  // of the keys' columns, or of the values' keys
      if (chunk < (val ? 2 : NKC)) {
        const int sub = val ? chunk * 64 : rank * 64;  // this chunk's first key in a tile
        uint64_t* const full = val ? &bars.v_full[chunk] : &bars.k_full[chunk];
        const uint32_t bar = first_cta(full);
        const uint32_t dst = sbase + (val ? OFF_V + chunk * V_CHUNK : OFF_K + chunk * 3 * K_ATOM);
        const int bytes = val ? V_CHUNK : 3 * K_ATOM, atoms = val ? 4 : 3;
        const int atom0 = val ? rank * 4 : chunk * 3;  // 64-column atom of the row
        const CUtensorMap* const map = val ? &map_v : &map_k;
        const bool counts = val && rank == 0;  // the values' warps of one CTA see every key once
        // The page of a box of 64 keys is looked up a tile ahead.
        int pg = -1;
        auto lookup = [&]() {
          advance();
          const int k = jt * KT + sub;
          if (p.box == 64 && k + 64 <= lim) pg = ld_global_nc_s32_early(trow + page_of(p.pool, k));
        };
        lookup();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int k0 = jt * KT + sub, left = lim - k0;
          const bool whole = p.box == 64 && left >= 64;
          int y0 = 0, r0 = p.pool.rows, r1 = p.pool.rows;  // rows of keys k0, k0 + lane, k0 + 32 + lane
          if (whole) {
            y0 = row_at(pg, k0, counts && last && lane == 0);
          } else {
            const int ka = k0 + lane, kb = ka + 32;
            if (ka < lim)
              r0 = row_at(ld_global_nc_s32_early(trow + page_of(p.pool, ka)), ka, counts && last);
            if (kb < lim)
              r1 = row_at(ld_global_nc_s32_early(trow + page_of(p.pool, kb)), kb, counts && last);
          }
          if (i + 1 < n) lookup();
          const bool ok =
              val ? i == 0 || warp_wait(&bars.pv_done[(i - 1) & 1][chunk], ((i - 1) >> 1) & 1,
                                        abort, p.status)
                  : warp_wait(&bars.k_empty[chunk], (i & 1) ^ 1, abort, p.status);
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(full, 2 * bytes);
          __syncwarp();
          if (whole) {
            if (elect_one()) tma_load_3d_pair(dst, map, 0, y0, atom0, bar);
          } else if (p.box && left >= 64) {
            // pages of a multiple of 16 or 32 rows: a box for each column atom
            const int per = 64 / p.box, k = (lane % per) * p.box, a = lane / per;
            const int ya = __shfl_sync(0xffffffffu, r0, k & 31);
            const int yb = __shfl_sync(0xffffffffu, r1, k & 31);
            if (a < atoms)
              tma_load_2d_pair(dst + a * 8192 + k * 128, &map_b, (atom0 + a) * 64,
                               k < 32 ? ya : yb, bar);
          } else {
            // row by row, four rows a load: the rows past the limit read as
            // zeros, so that nothing stored there can reach a product
            const int g = lane & 15;  // rows 4g .. 4g+3
            int y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int ya = __shfl_sync(0xffffffffu, r0, (4 * g + j) & 31);
              const int yb = __shfl_sync(0xffffffffu, r1, (4 * g + j) & 31);
              y[j] = g < 8 ? ya : yb;
            }
#pragma unroll 1
            for (int a = lane >> 4; a < atoms; a += 2)
              tma_gather4_pair(dst + a * 8192 + g * 512, &map_1, (atom0 + a) * 64, y[0], y[1],
                               y[2], y[3], bar);
          }
          __syncwarp();
        }
      }
    } else {
      // 8-bit: a warp takes 8 rows x 512 codes of the keys, or 16 x 256 of the
      // values: eight loads of 16 codes a thread, each instruction two rows' 256
      // contiguous bytes (four cache lines; a thread's codes side by side would
      // be 16 lines an instruction), and one scale, passed on by shuffles.  A
      // tile is converted as soon as its place is free; then the next one's loads
      // are issued, 64 KB an SM in flight.  The rotary keys come by TMA.
      const int hi = lane >> 4, ch = lane & 15;        // row of an instruction's pair, unit
      const int rows = val ? 16 : 8, hf = val ? wl >> 2 : 0;
      const int row0 = wl * rows;                      // of the tile's (this CTA's) rows
      const int yl = lane & (rows - 1);                // the row whose page this lane looks up
      const int key = row0 + yl + (val ? 0 : rank * 64);
      uint64_t* const full = val ? &bars.v_full[hf] : &bars.k_full[0];
      const uint32_t full0 = first_cta(full);
      // 16-byte piece of the first pair's row: pair j's is at (d0 ^ (j << 5)) + 256 j
      // (j < 4), the piece after it at address ^ 16
      const uint32_t d0 = sbase + (val ? OFF_V + hf * V_CHUNK : OFF_K) + (ch >> 2) * K_ATOM +
                          sw128_off((row0 & 63) + hi, (ch & 3) * 2);
      const int coff = (val ? rank * 256 : 0) + ch * 16;
      const int srow = val ? lane >> 1 : lane >> 2;    // row and group of this lane's scale
      const int soff = pages::kScaleOff + (val ? rank * 2 + (lane & 1) : lane & 3) * 4;
      // lane that holds the scale of unit it
      const int s0 = val ? hi * 2 + (ch >> 3) : hi * 4 + (ch >> 3);
      uint4 code[8];
      float sc = 0.f;
      int y = 0, pg = -2;  // pool row of the tile loaded, page of the next (this lane's row)
      auto lookup = [&]() {
        advance();
        const int k = jt * KT + key;
        pg = -2;
        if (k < lim) pg = ld_global_nc_s32_early(trow + page_of(p.pool, k));
      };
      auto ptr = [&](int l) {  // the row of lane l (an absent one: any, it gets the factor 0)
        const int r = __shfl_sync(0xffffffffu, y, l);
        return p.pool.base + (long long)(r < p.pool.rows ? r : 0) * p.pool.row_stride;
      };
      auto load = [&]() {
        const int k = jt * KT + key;
        y = row_at(pg, k, val && rank == 0 && lane < rows && last && k < lim);
#pragma unroll
        for (int it = 0; it < 8; ++it)
          code[it] = ld_global_nc_v4(val ? ptr(it * 2 + hi) + coff
                                         : ptr((it >> 1) * 2 + hi) + coff + (it & 1) * 256);
        const uint8_t* src = ptr(srow);
        sc = *reinterpret_cast<const float*>(src + soff);
      };
      lookup();
      load();
      if (n > 1) lookup();
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        // (keys: the last chunk's products are the last to finish)
        const bool ok =
            val ? i == 0 || warp_wait(&bars.pv_done[(i - 1) & 1][hf], ((i - 1) >> 1) & 1, abort,
                                      p.status)
                : warp_wait(&bars.k_empty[NKC - 1], (i & 1) ^ 1, abort, p.status);
        if (!ok) break;
        if (__shfl_sync(0xffffffffu, y, srow) >= p.pool.rows) sc = 0.f;
        const bool fp32 = __any_sync(0xffffffffu, pages::needs_fp32(sc));
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int j = val ? it & 3 : it >> 1;  // pair of rows (mod 8 rows)
          const uint32_t off = j * 256 + (val ? (it >> 2) * 1024 : (it & 1) * 4 * K_ATOM);
          const float f = __shfl_sync(0xffffffffu, sc, s0 + (val ? it * 4 : j * 8 + (it & 1) * 2));
          uint4 o0, o1;
          // (an absent row: whatever its codes are, under the factor 0 the exact product is 0)
          pages::dequant16(code[it], pages::Factor(f), fp32 && f != 0.f, o0, o1);
          st_shared_v4((d0 ^ (j << 5)) + off, o0.x, o0.y, o0.z, o0.w);
          st_shared_v4((d0 ^ (j << 5) ^ 16u) + off, o1.x, o1.y, o1.z, o1.w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_pair(full0);
          if (!val)
            for (int k = 1; k < NKC; ++k) mbar_arrive_pair(full0 + k * 8);
        }
        if (i + 1 < n) {
          load();
          if (i + 2 < n) lookup();
        }
      }
    }
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0 && bad && p.status) atomicAdd(p.status + 1, bad);
  } else if (kE4M3 && warp == R::rope) {
    // ---------------- rotary keys of 8-bit pages: the last atom of the last chunk ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::rest));
    int bb = bb0, jt = jt0 - 1, nr = tiles_of(bb0), lim = 0;
    const int32_t* trow = nullptr;
    auto enter = [&]() {
      if (bb >= p.N) return;
      lim = lim_of(bb);
      trow = p.pool.table + (long long)ld_global_nc_s32_early(p.plan.seq + bb) * p.pool.max_pages;
    };
    enter();
    const uint32_t bar = first_cta(&bars.k_full[NKC - 1]), dst = sbase + OFF_K + 8 * K_ATOM;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (++jt == nr) {
        jt = 0;
        nr = tiles_of(++bb);
        enter();
      }
      const int k0 = jt * KT + rank * 64 + lane, first = k0 - lane;
      const int r0 = k0 < lim ? row_of(p.pool, trow, k0) : p.pool.rows;
      const int r1 = k0 + 32 < lim ? row_of(p.pool, trow, k0 + 32) : p.pool.rows;
      if (!warp_wait(&bars.k_empty[NKC - 1], (i & 1) ^ 1, abort, p.status)) break;
      if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bars.k_full[NKC - 1], 2 * K_ATOM);
      __syncwarp();
      if (p.box && first + 64 <= lim) {
        const int k = lane * p.box & 63;
        const int ya = __shfl_sync(0xffffffffu, r0, k & 31);
        const int yb = __shfl_sync(0xffffffffu, r1, k & 31);
        if (lane * p.box < 64) tma_load_2d_pair(dst + k * 128, &map_b, 0, k < 32 ? ya : yb, bar);
      } else {
        const int g = lane & 15;
        int y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ya = __shfl_sync(0xffffffffu, r0, (4 * g + j) & 31);
          const int yb = __shfl_sync(0xffffffffu, r1, (4 * g + j) & 31);
          y[j] = g < 8 ? ya : yb;
        }
        if (lane < 16) tma_gather4_pair(dst + g * 512, &map_1, 0, y[0], y[1], y[2], y[3], bar);
      }
      __syncwarp();
    }
  } else if (warp == R::q) {
    // ---------------- queries: this CTA's 64 heads of each token ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::rest));
    const uint32_t bar = first_cta(&bars.q_full);
    int bb = bb0, i = 0, use = 0;  // use: tiles of the segment before
    for (int seg = 0; i < n; ++seg, ++bb) {
      if (!warp_wait(&bars.q_free, (seg & 1) ^ 1, abort, p.status, queries_limit_ns(use))) break;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(&bars.q_full, 2 * Q_BYTES);
        for (int a = 0; a < 8; ++a)
          tma_load_3d_pair(sbase + a * Q_ATOM, &map_qt, a * 64, rank * HH, bb, bar);
        tma_load_3d_pair(sbase + 8 * Q_ATOM, &map_qr, 0, rank * HH, bb, bar);
      }
      __syncwarp();
      use = tiles_of(bb) - (seg == 0 ? jt0 : 0);
      i += use;
    }
  } else if (warp == R::s) {
    // ---------------- score products ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::rest));
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, KT, 0, 0);
      constexpr uint32_t hi128 = desc_hi(1024, kSwizzle128B);
      const uint32_t lo_q = desc_lo(sbase, 16), lo_k = desc_lo(sbase + OFF_K, 16);
      int bb = bb0, jt = jt0, nr = tiles_of(bb0), seg = 0;
      bool ok = true, fresh = true;  // fresh: the segment's queries have not been waited for
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        if (fresh) ok = warp_wait(&bars.q_full, seg & 1, abort, p.status);
        fresh = false;
        const int sb = i % NSB;
        const bool ends = jt == nr - 1;
        ok = ok && warp_wait(&bars.s_empty[sb], ((i / NSB) & 1) ^ 1, abort, p.status);
        const uint32_t ts = tmem + T_S + sb * (KT / 2);
#pragma unroll 1
        for (int c = 0; c < NKC && ok; ++c) {
          ok = warp_wait(&bars.k_full[c], i & 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a = lo_q + c * (3 * Q_ATOM / 16), b = lo_k + c * (3 * K_ATOM / 16);
            // (12 products at once: 5 us of 119 against three times four)
#pragma unroll
            for (int ks = 0; ks < 12; ++ks)
              tc_mma2(ts, desc_join(a + (ks / 4 * Q_ATOM + ks % 4 * 32) / 16, hi128),
                      desc_join(b + (ks / 4 * K_ATOM + ks % 4 * 32) / 16, hi128), idesc,
                      ks > 0 || c > 0 ? 1u : 0u);
            tc_commit2(&bars.k_empty[c]);
            if (c == NKC - 1) {
              tc_commit2(&bars.s_full[sb]);
              if (ends) tc_commit2(&bars.q_free);
            }
          }
          __syncwarp();
        }
        if (++jt == nr) {
          jt = 0;
          nr = tiles_of(++bb);
          ++seg;
          fresh = true;
        }
      }
      // everything issued so far has finished before TMEM is released
      if (elect_one()) tc_commit2(&bars.drain[0]);
      __syncwarp();
      warp_wait(&bars.drain[0], 0, nullptr, p.status);
    }
  } else if (warp == R::o) {
    // ---------------- value products ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::rest));
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 256, 0, 1);
      constexpr uint32_t hi128 = desc_hi(1024, kSwizzle128B);
      const uint32_t lo_v = desc_lo(sbase + OFF_V, V_ATOM), lo_p = desc_lo(sbase + OFF_P, 16);
      int bb = bb0, jt = jt0, nr = tiles_of(bb0);
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t first = (jt - (bb == bb0 ? jt0 : 0)) % kRun == 0 ? 1u : 0u;
#pragma unroll 1
        for (int c = 0; c < 2 && ok; ++c) {  // half of the keys
          ok = warp_wait(&bars.v_full[c], i & 1, abort, p.status) &&
               warp_wait(&bars.p_full[i & 1][c], (i >> 1) & 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = lo_p + c * (P_BYTES / 16), v = lo_v + c * (V_CHUNK / 16);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                tc_mma2(tmem + T_O + j * 128, desc_join(a + ks * 2, hi128),
                        desc_join(v + (j * 2 * V_ATOM + ks * 2048) / 16, hi128), idesc,
                        ks > 0 || c > 0 ? 1u : first ^ 1u);
            tc_commit2(&bars.pv_done[i & 1][c]);
          }
          __syncwarp();
        }
        if (++jt == nr) {
          jt = 0;
          nr = tiles_of(++bb);
        }
      }
      if (elect_one()) tc_commit2(&bars.drain[1]);
      __syncwarp();
      warp_wait(&bars.drain[1], 0, nullptr, p.status);
    }
  } else if (warp >= KEY_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::rest));  // (idle)
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::soft));
    // ---------------- softmax: group g = tiles i with i % 2 == g ----------------
    // Thread = TMEM lane: head h = lane % 64 of this CTA's, keys (and latent
    // columns) of half lane / 64.
    const int g = warp >> 2, q4 = warp & 3;
    const int ln = q4 * 32 + lane, h = ln & 63, half = ln >> 6;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t to = tmem + lane_base + T_O;
    const uint32_t p_row = sbase + OFF_P + half * P_BYTES;
    const uint32_t p_bar0 = first_cta(&bars.p_full[g][0]), p_bar = p_bar0 + half * 8;
    const uint32_t s_bar = first_cta(&bars.s_empty[0]);
    auto wait_pv = [&](int t) -> bool {  // the value product of tile t has completed
      if (!warp_wait(&bars.pv_done[t & 1][1], (t >> 1) & 1, abort, p.status)) return false;
      tc_fence_after();
      return true;
    };
    // 32 scores of the lane; the first `left` of them are of keys the token sees
    auto load_scores = [](uint32_t taddr, int left, float (&x)[32]) {
      tmem_ld32(taddr, reinterpret_cast<uint32_t*>(x));
      tc_wait_ld();
      if (left < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= left) x[j] = -INFINITY;
      }
    };
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    auto publish_m = [&](float m) {  // the running maximum after this group's tile
      bars.m[g][h] = m;  // (both lanes of the head: the same value)
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.m_full[g][q4]);
    };
    float l = 0.f, lm = -INFINITY;  // this lane's and group's part of the row sum, its maximum
    int bb = bb0, jt = jt0, nr = tiles_of(bb0), lim = lim_of(bb0);
    int nseg = 0;  // tokens whose last tile came before this one
    int lseg = 0;  // the segment that l belongs to
    // this lane's part of the accumulator's copy and the maximum it refers to.  A
    // segment's runs end at every kRun-th tile, always of the same group: each thread
    // reads what it wrote, and what the other group's wrote only at the segment's end.
    static_assert(kRun % 2 == 0, "runs end at tiles of one group");
    float* const acc = p.acc + (size_t)blockIdx.x * ACC;
    float4* const acc4 = reinterpret_cast<float4*>(acc) + ln;
    float* const acc_m = acc + 128 * 256 + ln;
    auto step = [&]() {
      if (++jt == nr) {
        jt = 0;
        ++nseg;
        nr = tiles_of(++bb);
        lim = lim_of(bb);
      }
    };
    if (g == 1) step();
#pragma unroll 1
    for (int i = g; i < n; i += 2) {
      const int ph = (i >> 1) & 1;
      const int js = jt - (nseg == 0 ? jt0 : 0);     // tile of the segment
      const bool first = js == 0;
      const bool ends = jt == nr - 1 || i == n - 1;  // ... its last
      if (nseg != lseg) {  // this group's first tile of the segment
        lseg = nseg;
        l = 0.f;
        lm = -INFINITY;
      }
      if (!warp_wait(&bars.s_full[i % NSB], (i / NSB) & 1, abort, p.status)) break;
      tc_fence_after();
      const uint32_t ts = tmem + lane_base + T_S + (i % NSB) * (KT / 2);
      const int left = lim - jt * KT - half * 64;  // keys of this lane's 64 that the token sees
      float mt = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        float x[32];
        load_scores(ts + c, left - c, x);
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int j = 4; j < 28; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[j + e], x[j + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[28 + e]);
        mt = max3(max3(mt, mx[0], mx[1]), mx[2], mx[3]);
      }
      mt *= p.scale_log2;  // log2 units (the scale is positive)
      // The running maximum after tile i - 1, from the other group.  Waited for
      // before this tile's maxima are exchanged: whoever passes the exchange
      // then knows that both lanes' warps of the other group are done with
      // tile i - 1, and a segment's last tile publishes only after it has
      // read the sums of all four.
      float m = -INFINITY;
      if (i > 0) {
        if (!warp_wait(&bars.m_full[g ^ 1][q4], ((i - 1) >> 1) & 1, abort, p.status)) break;
        if (!first) m = *(volatile float*)&bars.m[g ^ 1][h];
      }
      // the tile's maximum over both lanes of the row
      bars.x[g][ln] = mt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.x_full[g][q4 & 1]);
      if (!warp_wait(&bars.x_full[g][q4 & 1], ph, abort, p.status)) break;
      mt = fmaxf(mt, *(volatile float*)&bars.x[g][ln ^ 64]);
      const bool raise = mt > m + kRescaleThreshold;
      const float mn = raise ? mt : m;
      if (!ends) publish_m(mn);
      if (!first && js % kRun == 0) {
        // a run ends: O~, which holds all tiles up to i - 1, moves to its copy
        if (!wait_pv(i - 1)) break;
        const bool more = js > kRun;
        float a = 0.f;
        if (more) {
          const float am = __ldcg(acc_m);
          a = am == m ? 1.f : fast_exp2(am - m);
        }
#pragma unroll 1
        for (int cc = 0; cc < 256; cc += 16) {
          uint32_t r[16];
          tmem_ld16(to + cc, r);
          tc_wait_ld();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float4 v = more ? __ldcg(acc4 + (cc / 4 + k) * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
            v.x = v.x * a + u2f(r[4 * k]);
            v.y = v.y * a + u2f(r[4 * k + 1]);
            v.z = v.z * a + u2f(r[4 * k + 2]);
            v.w = v.w * a + u2f(r[4 * k + 3]);
            __stcg(acc4 + (cc / 4 + k) * 128, v);
          }
        }
        __stcg(acc_m, m);
      } else if (!first && __any_sync(0xffffffffu, raise)) {
        // O~ must hold the value product of tile i - 1 before it is scaled
        if (!wait_pv(i - 1)) break;
        const float a = raise ? fast_exp2(m - mn) : 1.f;
#pragma unroll 1
        for (int cc = 0; cc < 256; cc += 16) {
          uint32_t r[16];
          tmem_ld16(to + cc, r);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = f2u(u2f(r[j]) * a);
          tmem_st16(to + cc, r);
        }
        tc_wait_st();
      }
      if (lm != mn) {  // the sum so far refers to a lower maximum (or is empty)
        l *= lm == -INFINITY ? 0.f : fast_exp2(lm - mn);
        lm = mn;
      }
      // (a row that has seen no key yet has m = -inf: its P is exp2(-inf) = 0)
      const float d = mn == -INFINITY ? 0.f : -mn;
      // the previous token's output has left TMEM before this one's first
      // value product (the other group writes it out)
      if (first && i > 0 &&
          !warp_wait(&bars.flushed[q4], (nseg - 1) & 1, abort, p.status))
        break;
      // (an arrival below is for this tile's phase: the group's last one, of
      // tile i - 2, is over once its value product has used the first half)
      if (i >= 2 && !warp_wait(&bars.pv_done[g][0], ((i - 2) >> 1) & 1, abort, p.status)) break;
      // The first half's products write all lanes of O: the second half's warps'
      // lanes are ready, so those products need not wait for their P.
      tc_fence_before();
      __syncwarp();
      if (half == 1 && lane == 0) mbar_arrive_pair(p_bar0);
      // This half of P has been used by tile i - 1's value product.  (A barrier
      // for each parity of tiles: a group waits on every phase of its own, and
      // one that both waited on could be two phases behind what a wait expects.)
      if (i > 0 && !warp_wait(&bars.pv_done[g ^ 1][half], ((i - 1) >> 1) & 1, abort, p.status))
        break;
      // (The scores are read from TMEM again, in a rolled loop.  The roles run
      // different code on the same schedulers: with a lane's 64 scores unrolled
      // they waited 5.8 cycles an issue for instructions, 6900 cycles a tile.)
      uint64_t s2 = 0;
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        float x[32];
        load_scores(ts + c, left - c, x);
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float e0, e1;
          unpack2(fma2(pack2(x[2 * j], x[2 * j + 1]), scale2, pack2(d, d)), e0, e1);
          e0 = fast_exp2(e0);
          e1 = fast_exp2(e1);
          s2 = add2(s2, pack2(e0, e1));
          w[j] = pack_bf16x2(e0, e1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          st_shared_v4(p_row + sw128_off(h, (c >> 3) + k), w[4 * k], w[4 * k + 1], w[4 * k + 2],
                       w[4 * k + 3]);
      }
      {
        float e0, e1;
        unpack2(s2, e0, e1);
        l += e0 + e1;
      }
      bars.l[g][ln] = l;
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_pair(p_bar);
        mbar_arrive(&bars.l_full[g][q4]);
        mbar_arrive_pair(s_bar + (i % NSB) * 8);
      }
      if (ends) {
        // the segment's end: the sums of both lanes and groups, then this lane's
        // half of O~ / l into the token's output (a token held whole by this
        // pair), or rounded to bf16 into the pair's slot (0: the range's first
        // segment, 1: its last) with the segment's log-sum-exps
        if (!warp_wait(&bars.l_full[g][q4 ^ 2], ph, abort, p.status)) break;
        volatile float* sum = bars.l[g];
        float lt = sum[h] + sum[h + 64];
        if (!first) {
          // tile i - 1 was the other group's, of the same segment: its sums refer
          // to the maximum it published (and publishes again only after this one)
          const int ph1 = ((i - 1) >> 1) & 1;
          if (!warp_wait(&bars.l_full[g ^ 1][q4], ph1, abort, p.status) ||
              !warp_wait(&bars.l_full[g ^ 1][q4 ^ 2], ph1, abort, p.status))
            break;
          sum = bars.l[g ^ 1];
          const float l2 = sum[h] + sum[h + 64];
          if (m != -INFINITY) lt += l2 * fast_exp2(m - mn);
        }
        publish_m(mn);
        if (!wait_pv(i)) break;
        const bool partial = (nseg == 0 && jt0 > 0) || jt != nr - 1;
        const int slot = 2 * cid + (nseg == 0 ? 0 : 1);
        const int head = rank * HH + h;
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        const bool moved = js >= kRun;  // earlier runs' part is in the copy
        float a = 0.f;
        if (moved) {
          const float am = __ldcg(acc_m);
          a = am == mn ? 1.f : fast_exp2(am - mn);
        }
        __nv_bfloat16* dst = (!partial ? p.omerged + ((size_t)bb * kH + head) * kC
                                       : p.opart + ((size_t)slot * kH + head) * kC) +
                             half * 256;
#pragma unroll 1
        for (int cc = 0; cc < 256; cc += 32) {
          uint32_t r[32];
          tmem_ld32(to + cc, r);
          tc_wait_ld();
          if (moved) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 v = __ldcg(acc4 + (cc / 4 + k) * 128);
              r[4 * k] = f2u(u2f(r[4 * k]) + v.x * a);
              r[4 * k + 1] = f2u(u2f(r[4 * k + 1]) + v.y * a);
              r[4 * k + 2] = f2u(u2f(r[4 * k + 2]) + v.z * a);
              r[4 * k + 3] = f2u(u2f(r[4 * k + 3]) + v.w * a);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(dst + cc + 8 * j) = make_uint4(
                pack_bf16x2(u2f(r[8 * j]) * inv, u2f(r[8 * j + 1]) * inv),
                pack_bf16x2(u2f(r[8 * j + 2]) * inv, u2f(r[8 * j + 3]) * inv),
                pack_bf16x2(u2f(r[8 * j + 4]) * inv, u2f(r[8 * j + 5]) * inv),
                pack_bf16x2(u2f(r[8 * j + 6]) * inv, u2f(r[8 * j + 7]) * inv));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.flushed[q4]);
        if (partial && half == 0)
          p.lse[(size_t)slot * kH + head] = lt == 0.f ? -INFINITY : mn + log2f(lt);
      }
      step();
      step();
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
  if (warp == R::s) {
    tc_fence_after();
    tmem_dealloc2(tmem, TMEM_COLS);
  }
  cluster_sync_all();  // neither CTA leaves before both have released
}

// ===========================================================================
// merge: O~ = sum_s 2^(lse_s - max) O~_s / sum_s 2^(lse_s - max) over the
// segments of the tokens that several pairs held (the plan's list).  Many split
// tokens: a warp for each token and head (or a few heads of it), without a barrier,
// its first segments' outputs loaded with their weights.  Few (then each has many
// segments): a block for two heads, 256 threads: a head's 64 16-byte chunks, four
// threads for each chunk's segments.  The plan, which was complete before the
// attend kernel let this one start, is read before the wait for its outputs.
// Bound by latency: 2 x 1 KB a head and segment.  (A block for each boundary and
// head, most of them with nothing to do, took 25 us; one for eight heads of a token,
// four at once, 14.)
// ===========================================================================
DEV int plan_entry(const int32_t* p) { return __ldcg(p); }  // (not through L1)

// Segments in pair order of the token b that boundary cb is the first to cut: slot
// 1 of pair cb - 1 (slot 0 when the token starts its range), slot 0 of every later
// pair whose range starts inside the token and is not empty.  Called by a warp.
DEV int segments_of(const Plan& pl, int nc, int cb, int b, uint16_t* slots) {
  const int lane = threadIdx.x & 31;
  const int rs = plan_entry(pl.tstart + b), re = plan_entry(pl.tstart + b + 1);
  int have = 1;
  if (lane == 0) slots[0] = 2 * (cb - 1) + (rs > plan_entry(pl.tb + cb - 1) ? 1 : 0);
  for (int c0 = cb; c0 < nc; c0 += 32) {
    const int c = c0 + lane;
    const int a = c < nc ? plan_entry(pl.tb + c) : re;
    const int e = c < nc ? plan_entry(pl.tb + c + 1) : re;
    const bool in = a < re && e > a;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) slots[have + __popc(m & ((1u << lane) - 1u))] = 2 * c;
    have += __popc(m);
    if (!__all_sync(0xffffffffu, a < re)) break;
  }
  __syncwarp();
  return have;
}
// the segments' weights of head h into w, by a warp -> their sum
DEV float segment_weights(const float* lse, const uint16_t* slots, int n, int h, float* w) {
  const int lane = threadIdx.x & 31;
  float mx = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float l = lse[(size_t)slots[i] * kH + h];
    w[i] = l;
    mx = fmaxf(mx, l);  // (drops a NaN, which the weights below keep)
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float e = w[i] == -INFINITY ? 0.f : exp2f(w[i] - mx);
    w[i] = e;
    sum += e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  return sum;
}
DEV void add_segment(float (&acc)[8], const uint4& v, float w) {
  const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[2 * e] += w * u2f(p[e] << 16);
    acc[2 * e + 1] += w * u2f(p[e] & 0xffff0000u);
  }
}
DEV void store_merged(__nv_bfloat16* dst, const float (&acc)[8], float sum) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                 pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
}

constexpr int kMergeMany = 16;  // split tokens

__global__ void __launch_bounds__(256) merge_kernel(const __nv_bfloat16* __restrict__ opart,
                                                     const float* __restrict__ lse, const Plan pl,
                                                     int nc, __nv_bfloat16* __restrict__ omerged) {
  __shared__ uint16_t slots[8][kMaxPairs];
  __shared__ float w[8][kMaxPairs];
  __shared__ int count;
  __shared__ float wsum, acc_s[3][64][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  const int nsplit = plan_entry(pl.nact + 1);
  if (nsplit >= kMergeMany) {
    int heads = 1;  // of a warp
    while (heads < kH && (long long)gridDim.x * 8 * heads < (long long)nsplit * kH) heads *= 2;
    const int unit = (blockIdx.x * 8 + warp) * heads, ti = unit / kH;
    int b = 0, n = 0;
    if (ti < nsplit) {
      const int cb = plan_entry(pl.split + ti);
      b = plan_entry(pl.crow + cb);
      n = segments_of(pl, nc, cb, b, slots[warp]);
    }
    // every block waits, those with nothing to merge too: the value kernel
    // relies on this grid's completion implying the attend kernel's
    pdl_wait();
    for (int h = unit % kH; n > 0 && h < unit % kH + heads; ++h) {
      const __nv_bfloat16* src = opart + (size_t)h * kC + lane * 8;
      uint4 v[3][2];
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            v[i][k] = ld_global_nc_v4(src + (size_t)slots[warp][i] * kH * kC + k * 256);
      const float sum = segment_weights(lse, slots[warp], n, h, w[warp]);
      float acc[2][8] = {};
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n)
#pragma unroll
          for (int k = 0; k < 2; ++k) add_segment(acc[k], v[i][k], w[warp][i]);
      for (int i = 3; i < n; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          add_segment(acc[k],
                      ld_global_nc_v4(src + (size_t)slots[warp][i] * kH * kC + k * 256),
                      w[warp][i]);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        store_merged(omerged + ((size_t)b * kH + h) * kC + k * 256 + lane * 8, acc[k], sum);
      __syncwarp();
    }
    return;
  }
  // a token and two heads, in turn
  const int ch = tid & 63, g = tid >> 6;
  bool waited = false;
  for (int u = blockIdx.x; u < nsplit * (kH / 2); u += gridDim.x) {
    const int cb = plan_entry(pl.split + u / (kH / 2));
    const int b = plan_entry(pl.crow + cb);
    if (warp == 0) {
      const int have = segments_of(pl, nc, cb, b, slots[0]);
      if (lane == 0) count = have;
    }
    __syncthreads();
    const int n = count;
    if (!waited) pdl_wait();
    waited = true;
    for (int h = u % (kH / 2) * 2, last = h + 1; h <= last; ++h) {
      const __nv_bfloat16* src = opart + (size_t)h * kC + ch * 8;
      uint4 v[2];  // the thread's first segments: g and g + 4
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (g + 4 * k < n) v[k] = ld_global_nc_v4(src + (size_t)slots[0][g + 4 * k] * kH * kC);
      if (warp == 0) {
        const float sum = segment_weights(lse, slots[0], n, h, w[0]);
        if (lane == 0) wsum = sum;
      }
      __syncthreads();
      float acc[8] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (g + 4 * k < n) add_segment(acc, v[k], w[0][g + 4 * k]);
#pragma unroll 4
      for (int i = g + 8; i < n; i += 4)
        add_segment(acc, ld_global_nc_v4(src + (size_t)slots[0][i] * kH * kC), w[0][i]);
      if (g > 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc_s[g - 1][ch][e] = acc[e];
      __syncthreads();
      if (g == 0) {
        for (int k = 0; k < 3; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += acc_s[k][ch][e];
        store_merged(omerged + ((size_t)b * kH + h) * kC + ch * 8, acc, wsum);
      }
      __syncthreads();  // w, acc_s and slots may be written again
    }
  }
  if (!waited) pdl_wait();
}

// ===========================================================================
// value_kernel: O = W_UV O~ per head, D^T[d, token] = sum_c W_UV[h][d][c] O~[token][h][c]
//   A = W_UV[h] (M = 128 value dims, K = c), B = O~ rows (N = tokens), both K-major
// Grid (heads, blocks of NB tokens), 128 threads.  All of K = 512 is loaded at
// once in eight 64-wide chunks with a barrier each; the weight's loads are in
// flight before the kernel waits for the kernel that writes O~.  Rows of
// padding tokens are not written.
// ===========================================================================
template <int NB>
__global__ void __launch_bounds__(128) value_kernel(const __grid_constant__ CUtensorMap map_w,
                                                     const __grid_constant__ CUtensorMap map_o,
                                                     const int32_t* __restrict__ nact,
                                                     __nv_bfloat16* __restrict__ O,
                                                     int32_t* status) {
  constexpr uint32_t NCOLS = NB < 32 ? 32 : NB;
  constexpr int A_CHUNK = 128 * 128, B_CHUNK = NB * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sA = smem_u32(smem), sB = sA + 8 * A_CHUNK;
  __shared__ uint64_t bar[8], bar_mma;
  __shared__ uint32_t tmem_base;
  const int h = blockIdx.x, b0 = blockIdx.y * NB;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    tmem_alloc(&tmem_base, NCOLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(&bar[i], 1);
    mbar_init(&bar_mma, 1);
    fence_mbarrier_init_cluster();
    for (int i = 0; i < 8; ++i) {
      mbar_arrive_expect_tx(&bar[i], A_CHUNK + B_CHUNK);
      tma_load_2d(sA + i * A_CHUNK, &map_w, i * 64, h * 256 + kD, &bar[i]);
    }
  }
  pdl_wait();
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) tma_load_3d(sB + i * B_CHUNK, &map_o, i * 64, h, b0, &bar[i]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if (tid == 0) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, NB, 0, 0);
    for (int i = 0; i < 8; ++i) {
      if (!mbar_wait(&bar[i], 0, nullptr, status)) break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        tc_mma(tmem, smem_desc(sA + i * A_CHUNK + ks * 32, 16, 1024, kSwizzle128B),
               smem_desc(sB + i * B_CHUNK + ks * 32, 16, 1024, kSwizzle128B), idesc,
               (i > 0 || ks > 0) ? 1u : 0u);
    }
    tc_commit(&bar_mma);
  }
  __syncwarp();
  const int n = min(NB, ld_global_nc_s32_early(nact) - b0);  // rows of this block to write
  bool ok = warp_wait(&bar_mma, 0, nullptr, status);
  // (the products have finished, so a chunk that timed out shows here too)
  for (int i = 0; i < 8; ++i) ok = warp_wait(&bar[i], 0, nullptr, status) && ok;
  tc_fence_after();
  // through shared memory as [token][128 d] bf16 rows, then 16-byte stores
  const uint32_t stage = sA;
  if (ok) {
    const int d = warp * 32 + lane;
#pragma unroll 1
    for (int n0 = 0; n0 < NB; n0 += 16) {
      uint32_t r[16];
      tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + n0, r);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const __nv_bfloat16 v = __float2bfloat16_rn(u2f(r[j]));
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(stage + (n0 + j) * 256 + d * 2),
                     "h"(*reinterpret_cast<const unsigned short*>(&v))
                     : "memory");
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (ok) {
    for (int q = tid; q < n * 16; q += 128) {
      const int nn = q >> 4, ch = q & 15;
      const uint4 v = ld_shared_v4(stage + nn * 256 + ch * 16);
      *reinterpret_cast<uint4*>(O + ((size_t)(b0 + nn) * kH + h) * kD + ch * 8) = v;
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, NCOLS);
  }
}

// ===========================================================================
// host
// ===========================================================================

static int max_pairs() {
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 74;
  }
  if (dev < 64) {
    const int c = cached[dev].load(std::memory_order_acquire);
    if (c > 0) return c;
  }
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * kMaxPairs);
  cfg.blockDim = dim3(Roles<true>::threads);
  cfg.dynamicSmemBytes = dynamic_smem();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // (one CTA an SM either way: shared memory)
  if (cudaFuncSetAttribute(absorbed_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           dynamic_smem()) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, absorbed_kernel<true>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    int sms = 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      sms = 148;
    }
    n = sms / 2;
  }
  n = n < kMaxPairs ? n : kMaxPairs;
  if (dev < 64) cached[dev].store(n, std::memory_order_release);
  return n;
}

struct AbsorbedWs {
  size_t q_tilde, opart, lse, acc, omerged, seq, lim, tstart, tb, crow, split, nact, total;
};

static AbsorbedWs absorbed_ws(int N, int nc) {
  AbsorbedWs w;
  w.q_tilde = 0;
  w.opart = round_up((size_t)N * kH * kC * 2, 256);
  w.lse = w.opart + (size_t)nc * 2 * kH * kC * 2;
  w.acc = round_up(w.lse + (size_t)nc * 2 * kH * 4, 256);
  w.omerged = round_up(w.acc + (size_t)nc * 2 * ACC * 4, 256);
  w.seq = round_up(w.omerged + (size_t)N * kH * kC * 2, 256);
  w.lim = round_up(w.seq + (size_t)N * 4, 256);
  w.tstart = round_up(w.lim + (size_t)N * 4, 256);
  w.tb = round_up(w.tstart + (size_t)(N + 1) * 4, 256);
  w.crow = round_up(w.tb + (size_t)(nc + 1) * 4, 256);
  w.split = round_up(w.crow + (size_t)(nc + 1) * 4, 256);
  w.nact = round_up(w.split + (size_t)nc * 4, 256);
  w.total = w.nact + 256;
  return w;
}

template <int NB>
static int launch_value_nb(const __nv_bfloat16* wkv_b, const __nv_bfloat16* omerged, int N,
                           const int32_t* nact, __nv_bfloat16* O, int32_t* status,
                           cudaStream_t st) {
  alignas(64) CUtensorMap map_w, map_o;
  if (int e = bf16_map_2d(&map_w, wkv_b, kC, kH * 256, kC * 2, 64, 128)) return e;
  if (int e = bf16_map_3d(&map_o, omerged, kC, kH, N, kC * 2, kH * kC * 2, 64, 1, NB)) return e;
  const int smem = 8 * (128 * 128 + NB * 128) + 1024;
  static std::atomic<unsigned long long> attr_done{0};
  if (int e = ensure_smem_attr(value_kernel<NB>, smem, &attr_done)) return e;
  return launch_pdl(value_kernel<NB>, dim3(kH, (N + NB - 1) / NB), dim3(128), smem, st, map_w,
                    map_o, nact, O, status);
}

template <bool kE4M3>
static int launch_absorbed(const Params& p, int nc, cudaStream_t st) {
  alignas(64) CUtensorMap map_qt, map_qr, map_k = {}, map_v = {}, map_b = {}, map_1 = {};
  if (int e = bf16_map_3d(&map_qt, p.q_tilde, kC, kH, p.N, kC * 2, kH * kC * 2, 64, HH, 1))
    return e;
  if (int e = bf16_map_3d(&map_qr, p.q_pe, kR, kH, p.N, kR * 2, kH * kR * 2, 64, HH, 1)) return e;
  if (!kE4M3) {
    // rows as [9 column atoms][rows][64]: a box takes several atoms at once
    const uint64_t rows = p.pool.rows, rb = p.pool.row_stride;
    if (int e = bf16_map_3d(&map_k, p.pool.base, 64, rows, 9, rb, 128, 64, 64, 3)) return e;
    if (int e = bf16_map_3d(&map_v, p.pool.base, 64, rows, 9, rb, 128, 64, 64, 4)) return e;
    if (int e = bf16_map_2d(&map_b, p.pool.base, MLA_ROW, rows, rb, 64, p.box ? p.box : 1)) return e;
    if (int e = bf16_map_2d(&map_1, p.pool.base, MLA_ROW, rows, rb, 64, 1)) return e;
  } else {
    const uint64_t rows = p.pool.rows, rb = p.pool.row_stride;
    const uint8_t* rope = p.pool.base + pages::kRopeOff;
    if (int e = bf16_map_2d(&map_b, rope, kR, rows, rb, 64, p.box ? p.box : 1)) return e;
    if (int e = bf16_map_2d(&map_1, rope, kR, rows, rb, 64, 1)) return e;
  }
  static std::atomic<unsigned long long> attr_done{0};
  if (int e = ensure_smem_attr(absorbed_kernel<kE4M3>, dynamic_smem(), &attr_done)) return e;
  return launch_pdl(absorbed_kernel<kE4M3>, dim3(2 * nc), dim3(Roles<kE4M3>::threads), dynamic_smem(), st, p,
                    map_qt, map_qr, map_k, map_v, map_b, map_1);
}

// 8-bit pages that several tokens a sequence read are converted to bf16 rows
// first.  Measured over 128 sequences up to 16000 positions, in microseconds
// without / with it: 2 tokens each 905 / 873, 3 1421 / 1211, 4 1784 / 1413; its
// two launches take 10 at least (32 sequences up to 500, 2 tokens: 51 / 63; one of
// 60000, 4 tokens: 143 / 121).  So from 3 tokens a sequence, and where what is
// saved (0.24 ns a token and position, half of max_kv on average) pays for the
// launches; and not where the rows could pass 4 GiB.
static bool stages(int kind, int N, int S, int max_kv) {
  return kind == MLA_PAGE_E4M3 && N >= 3 * (int64_t)S && (int64_t)N * max_kv >= (1 << 18) &&
         (int64_t)S * (max_kv + 127) * (MLA_ROW * 2) <= (4ll << 30);
}

static int run_absorbed(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
                        const Pool& pages, const Seqs& seqs, float scale, mla_bf16_t* O,
                        uint8_t* ws, int32_t* status, cudaStream_t st) {
  const int nc = max_pairs();
  const AbsorbedWs L = absorbed_ws(seqs.N, nc);
  Pool pool = pages;
  Seqs q = seqs;
  if (stages(pages.kind, q.N, q.S, q.max_kv)) {
    if (int e = expand::stage(pages, q, ws + round_up(L.total, 256), status, st, &pool)) return e;
    // (the staged table may have room for positions that the caller's has not)
    const int64_t cap = (int64_t)pages.max_pages * pages.page_size;
    if (cap < q.max_kv) q.max_kv = (int)cap;
  }
  Plan pl;
  pl.seq = reinterpret_cast<int32_t*>(ws + L.seq);
  pl.lim = reinterpret_cast<int32_t*>(ws + L.lim);
  pl.tstart = reinterpret_cast<int32_t*>(ws + L.tstart);
  pl.tb = reinterpret_cast<int32_t*>(ws + L.tb);
  pl.crow = reinterpret_cast<int32_t*>(ws + L.crow);
  pl.split = reinterpret_cast<int32_t*>(ws + L.split);
  pl.nact = reinterpret_cast<int32_t*>(ws + L.nact);
  __nv_bfloat16* q_tilde = reinterpret_cast<__nv_bfloat16*>(ws + L.q_tilde);
  // The fold waits for the stream's earlier work as usual; the others may start
  // while their predecessor drains.
  if (int e = launch_fold(reinterpret_cast<const __nv_bfloat16*>(q_nope),
                          reinterpret_cast<const __nv_bfloat16*>(wkv_b), q_tilde, q.N, status, st))
    return e;
  if (int e = launch_pdl(plan_kernel, dim3(1), dim3(1024), 0, st, q, pool, pl, nc)) return e;
  Params p;
  p.q_tilde = q_tilde;
  p.q_pe = reinterpret_cast<const __nv_bfloat16*>(q_pe);
  p.pool = pool;
  p.plan = pl;
  p.N = q.N;
  p.box = pool.page_size % 64 == 0 ? 64 : pool.page_size % 32 == 0 ? 32
          : pool.page_size % 16 == 0 ? 16 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.opart = reinterpret_cast<__nv_bfloat16*>(ws + L.opart);
  p.lse = reinterpret_cast<float*>(ws + L.lse);
  p.acc = reinterpret_cast<float*>(ws + L.acc);
  p.omerged = reinterpret_cast<__nv_bfloat16*>(ws + L.omerged);
  p.status = status;
  if (int e = pool.kind == MLA_PAGE_E4M3 ? launch_absorbed<true>(p, nc, st)
                                         : launch_absorbed<false>(p, nc, st))
    return e;
  if (nc > 1)
    if (int e = launch_pdl(merge_kernel, dim3(8 * nc), dim3(256), 0, st,
                           (const __nv_bfloat16*)p.opart, (const float*)p.lse, pl, nc, p.omerged))
      return e;
  const __nv_bfloat16* w = reinterpret_cast<const __nv_bfloat16*>(wkv_b);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(O);
  if (q.N <= 16) return launch_value_nb<16>(w, p.omerged, q.N, pl.nact, out, status, st);
  if (q.N <= 32) return launch_value_nb<32>(w, p.omerged, q.N, pl.nact, out, status, st);
  return launch_value_nb<64>(w, p.omerged, q.N, pl.nact, out, status, st);
}

}  // namespace paged
}  // namespace shla

using namespace shla;

// The absorbed form's list of (token, 128-key tile) is counted in 32 bits.
static bool absorbed_fits(int N, int max_kv) {
  return (int64_t)N * ((max_kv + 127) / 128) <= 0x3fffffff;
}

// The form of a call: as asked, or by the new tokens per sequence.  Past
// kAutoRows positions in all the expanded form's workspace decides, not its time.
static int form_of(int form, int N, int S, int max_kv) {
  if (form != MLA_FORM_AUTO) return form;
  if ((int64_t)N < (int64_t)S * expand::min_tokens(max_kv)) return MLA_FORM_ABSORBED;
  return expand::fits(S, max_kv, expand::kAutoRows) ||
                 (!absorbed_fits(N, max_kv) && expand::fits(S, max_kv))
             ? MLA_FORM_EXPANDED
             : MLA_FORM_ABSORBED;
}

static int check_sizes(int N, int S, int max_kv, int kind, int form) {
  if (kind != MLA_PAGE_BF16 && kind != MLA_PAGE_E4M3) return MLA_ERR_SHAPE;
  if (N < 1 || N > 65535 || S < 1 || S > 65535 || max_kv < 1 || max_kv > (1 << 24))
    return MLA_ERR_SHAPE;
  if (form < MLA_FORM_AUTO || form > MLA_FORM_EXPANDED) return MLA_ERR_SHAPE;
  if (form_of(form, N, S, max_kv) == MLA_FORM_EXPANDED ? !expand::fits(S, max_kv)
                                                       : !absorbed_fits(N, max_kv))
    return MLA_ERR_SHAPE;
  return MLA_OK;
}

extern "C" size_t mla_attend_paged_workspace_bytes(int N, int S, int max_kv, int kind, int form) {
  if (check_sizes(N, S, max_kv, kind, form) != MLA_OK) return 0;
  if (form_of(form, N, S, max_kv) == MLA_FORM_EXPANDED) return expand::workspace_bytes(N, S, max_kv);
  const size_t own = round_up(paged::absorbed_ws(N, paged::max_pairs()).total, 256);
  return own + (paged::stages(kind, N, S, max_kv) ? expand::staged_bytes(N, S, max_kv) : 0);
}

extern "C" int mla_attend_paged(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe,
                                const mla_bf16_t* wkv_b, const void* pool, int kind,
                                int num_pages, int page_size, int64_t page_stride, int row_stride,
                                const int32_t* page_table, int max_pages, const int32_t* cu_q,
                                const int32_t* kv_len, int S, int N, int max_kv, float scale,
                                int form, mla_bf16_t* O, void* ws, size_t ws_bytes,
                                int32_t* status, void* stream) {
  if (!q_nope || !q_pe || !wkv_b || !page_table || !cu_q || !kv_len || !O) return MLA_ERR_NULL;
  if (int e = pages::check_pool(pool, kind, num_pages, page_size, page_stride, row_stride))
    return e;
  if (int e = check_sizes(N, S, max_kv, kind, form)) return e;
  // (written so that a NaN is refused too)
  if (max_pages < 1 || !(scale > 0.f && scale <= 3.0e38f)) return MLA_ERR_SHAPE;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(wkv_b) || !aligned16(O))
    return MLA_ERR_ALIGN;
  if (!ws || !aligned256(ws)) return MLA_ERR_WORKSPACE;
  const size_t need = mla_attend_paged_workspace_bytes(N, S, max_kv, kind, form);
  // (the expanded form stores outputs while other SMs still load queries, and reads
  // all others after its first ones too)
  const size_t row = (size_t)MLA_HEADS * 2 * MLA_NOPE, out_bytes = N * row;
  const struct {
    const void* p;
    size_t bytes;
  } inputs[] = {{q_nope, N * row},
                {q_pe, (size_t)N * MLA_HEADS * 2 * MLA_ROPE},
                {wkv_b, (size_t)MLA_HEADS * 256 * MLA_LATENT * 2},
                {page_table, (size_t)S * max_pages * 4},
                {cu_q, ((size_t)S + 1) * 4},
                {kv_len, (size_t)S * 4}};
  for (const auto& in : inputs)
    if (overlap(O, out_bytes, in.p, in.bytes) || overlap(ws, need, in.p, in.bytes))
      return MLA_ERR_OVERLAP;
  if (overlap(O, out_bytes, ws, need)) return MLA_ERR_OVERLAP;
  if (int e = check_device()) return e;
  if (ws_bytes < need) return MLA_ERR_WORKSPACE;
  paged::Pool p;
  p.base = static_cast<const uint8_t*>(pool);
  p.kind = kind;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.pitch = (int)(page_stride / row_stride);
  p.row_stride = row_stride;
  p.rows = (num_pages - 1) * p.pitch + page_size;
  p.table = page_table;
  paged::set_division(&p);
  p.max_pages = max_pages;
  paged::Seqs q;
  q.cu_q = cu_q;
  q.kv_len = kv_len;
  q.S = S;
  q.N = N;
  q.max_kv = max_kv;
  if (form_of(form, N, S, max_kv) == MLA_FORM_EXPANDED)
    return expand::run(q_nope, q_pe, wkv_b, p, q, scale, O, static_cast<uint8_t*>(ws), status,
                       as_stream(stream));
  return paged::run_absorbed(q_nope, q_pe, wkv_b, p, q, scale, O, static_cast<uint8_t*>(ws),
                             status, as_stream(stream));
}
