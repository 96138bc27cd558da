// Attention of new tokens over a paged latent cache, absorbed form.  For each
// new token and head h, over the positions t < lim the token sees:
//   q~ = q_nope W_UK[h];  s_t = (q~ . c_t + q_pe . kpe_t) * scale
//   O = W_UV[h] (softmax(s) c)
// Five kernels on the caller's stream:
//
//   plan_kernel      one block: each token's sequence and limit, the prefix sum
//                    of the tokens' 64-key tiles, and its cut into one range
//                    of equal cost per CTA pair
//   (fold)           q~ per head, as in mla_decode
//   absorbed_kernel  persistent CTA pairs over their ranges
//   merge_kernel     log-sum-exp merge of the tokens that several pairs held
//   value_kernel     O = W_UV O~ per head
#include <math.h>

#include "attend_paged.cuh"
#include "expand.h"
#include "tma_map.h"

namespace shla {
namespace paged {

// ===========================================================================
// plan
// ===========================================================================

constexpr int KT = 64;  // keys per tile
// Fixed cost of a token in tiles: its query load and its output's write-out.
constexpr int kTokenCost = 4;

struct Plan {
  int32_t* seq;     // [N] sequence of each token
  int32_t* lim;     // [N] positions it sees
  int32_t* tstart;  // [N + 1] its first tile in the flattened list
  int32_t* tb;      // [nc + 1] first tile of each pair's range
  int32_t* crow;    // [nc + 1] the token that holds that tile
  int32_t* nact;    // [1] tokens of the sequences (those behind the last one are padding)
};

// Every token has at least one tile, so that one that sees nothing still gets
// its zero output.
__global__ void __launch_bounds__(1024) plan_kernel(const Seqs q, const Pool pool, const Plan pl,
                                                     int nc) {
  __shared__ int part[1024];
  const int tid = threadIdx.x;
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
  if (tid == 0) *pl.nact = nact;
  __syncthreads();  // tstart, written by the block, is visible to it
  // Cost units: token r spans kTokenCost units of its own, then one per tile,
  // from u(r) = tstart[r] + r * kTokenCost.  Pair c takes the units
  // [c U / nc, (c + 1) U / nc); a range that starts in a token's own units
  // starts at its first tile.
  const long long U = (long long)tot + (long long)nact * kTokenCost;
  for (int c = tid; c <= nc; c += 1024) {
    if (c == nc || nact == 0) {
      pl.tb[c] = tot;
      pl.crow[c] = nact;
      continue;
    }
    const long long u = (long long)c * U / nc;
    int a = 0, e = nact;  // u(a) <= u < u(e)
    while (e - a > 1) {
      const int m = (a + e) >> 1;
      if ((long long)pl.tstart[m] + (long long)m * kTokenCost <= u) a = m; else e = m;
    }
    const long long into = u - ((long long)pl.tstart[a] + (long long)a * kTokenCost);
    pl.tb[c] = pl.tstart[a] + (into > kTokenCost ? (int)(into - kTokenCost) : 0);
    pl.crow[c] = a;
  }
}

// ===========================================================================
// absorbed_kernel: persistent 2-CTA clusters
//
// One CTA's TMEM cannot hold the 128 x 512 fp32 accumulator of a token's 128
// heads and anything else, so a pair of CTAs splits the latent: CTA r holds
// latent columns [256r, 256r+256) and rotary columns [32r, 32r+32) of q~ and
// of every key.  Per tile of 64 keys:
//   S_r  = Q~_r K_r^T      M = 128 heads, N = 64, K = 288; A = Q~ in TMEM
//   the two exchange their fp32 partial scores (st.async into the peer's
//   shared memory), add them (a + b in one CTA, b + a in the other: the same
//   numbers) and both run the same fp32 online softmax: running maximum,
//   raised only once a tile exceeds it by more than 8 log2 units; P = 2^(s-m)
//   rounded to bf16 as a tensor-core operand (its row sum is of the fp32 P)
//   O_r += P V_r           M = 128, N = 256, K = 64; A = P in TMEM, V = the
//   key tile itself, read MN-major
//
// Roles (640 threads):
//   warps 0-7    softmax, 16 head rows each, four threads per row: own partial
//                scores from TMEM + the peer's from shared memory
//   warps 8-11   senders, one lane quarter each: own partial scores to the
//                peer; the next token's queries
//   warps 12-18  keys: TMA boxes of up to 64 rows (16-bit pages; one warp), or
//                loads, exact conversion to bf16 and swizzled stores (8-bit)
//   warp 19      TMEM owner and MMA issuer
// The senders never wait for the peer's scores and the softmax warps never
// send: the exchange is a pipeline stage, not a round trip.  Scores are
// double-buffered and P overlays the scores it came from, so the score
// product of tile i + 1 runs while tile i is in the softmax.
// TMEM (512 columns): Q~ half [0,128) as bf16 pairs, two score tiles [128,256)
// (their first 32 columns become P), the output half in fp32 [256,512).
// ===========================================================================

constexpr int NST = 4;                 // key ring depth
constexpr int NSOFT = 8;               // softmax warps
constexpr int SEND_WARP0 = 8;
constexpr int KEY_WARP0 = 12;
constexpr int NKEY = 7;
constexpr int MMA_WARP = 19;
constexpr int NTHREADS = 32 * (MMA_WARP + 1);
constexpr int ST_ATOM = KT * 128;      // one 64-column latent atom of a tile (128 B swizzle)
constexpr int ST_KR = 4 * ST_ATOM;     // rotary half of a tile (64 B swizzle)
constexpr int ST_BYTES = ST_KR + KT * 64;
constexpr int OFF_QR = NST * ST_BYTES; // rotary half of Q: 128 rows x 64 B, 64 B swizzle
constexpr int OFF_XS = OFF_QR + 128 * 64;
constexpr int XS_BYTES = NSOFT * 8 * 32 * 16;  // the peer's partial scores: [warp][8][32 lanes][16 B]
constexpr int OFF_ROWSTART = OFF_XS + 2 * XS_BYTES;  // per stage: the tile starts its token
constexpr int SMEM_BYTES = OFF_ROWSTART + NST * 4 + 1024;  // + alignment slack
constexpr uint32_t T_Q = 0, T_S = 128, T_O = 256, TMEM_COLS = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
static_assert(ST_BYTES % 1024 == 0 && OFF_QR % 1024 == 0 && OFF_XS % 16 == 0, "alignment");
static_assert(SMEM_BYTES + 512 <= 232448, "shared memory budget");
static_assert(T_Q + 128 <= T_S && T_S + 2 * KT <= T_O && T_O + 256 <= TMEM_COLS, "TMEM plan");

struct Params {
  const __nv_bfloat16* q_tilde;  // [N][128][512]
  const __nv_bfloat16* q_pe;     // [N][128][64]
  Pool pool;
  Plan plan;
  int N;
  int box;                       // rows of a TMA box (16, 32 or 64; 0: row by row)
  float scale_log2;              // softmax scale * log2(e)
  __nv_bfloat16* opart;          // [pairs][2 slots][128][512], normalised per segment
  float* lse;                    // [pairs][2 slots][128], log2 units of scaled scores
  __nv_bfloat16* omerged;        // [N][128][512]
  int32_t* status;
};

struct Bars {
  uint64_t full[NST], empty[NST];  // key ring
  uint64_t s_full[2];              // score tile of tile i in buffer i & 1
  uint64_t sent[2];                // ... read by the senders
  uint64_t xs_full[2], xs_free[2]; // the peer's partial scores landed / the peer has read ours
  uint64_t p_full[2], o_done[2];   // P written over the scores / its value product done
  uint64_t q_ready;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// one lane of a converged warp, the same every time
DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, the accumulate flag at run time
DEV void tc_mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

DEV float u2f(uint32_t x) { return __uint_as_float(x); }
DEV uint32_t f2u(float x) { return __float_as_uint(x); }

struct Pos {
  int bb, jt, nr;  // token, tile within it, its tile count
};

template <bool kE4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    absorbed_kernel(const Params p, const __grid_constant__ CUtensorMap map_c,
                    const __grid_constant__ CUtensorMap map_r,
                    const __grid_constant__ CUtensorMap map_c1,
                    const __grid_constant__ CUtensorMap map_r1) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ Bars bars;
  volatile int* abort = &bars.abort;

  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  const int cid = blockIdx.x >> 1;
  // (the plan was complete before the fold kernel began)
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

  if (warp == MMA_WARP) {
    tmem_alloc(&bars.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars.full[s], kE4M3 ? NKEY : 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.sent[i], 4);
      mbar_init(&bars.xs_full[i], 1);      // own expect_tx arrival + the peer's bytes
      mbar_init(&bars.xs_free[i], NSOFT);  // one arrival per softmax warp of the peer
      mbar_init(&bars.p_full[i], NSOFT);
      mbar_init(&bars.o_done[i], 1);
    }
    mbar_init(&bars.q_ready, 4);
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbarrier_init_cluster();
    for (int i = 0; i < 2 && i < n; ++i) mbar_arrive_expect_tx(&bars.xs_full[i], XS_BYTES);
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  if (n <= 0) {
    // an empty range (fewer tiles than pairs): nothing to do
  } else if (warp >= KEY_WARP0 && warp < MMA_WARP) {
    // ---------------- keys ----------------
    const int kw = warp - KEY_WARP0;
    if (kE4M3 || kw == 0) {
      int bb = bb0, jt = jt0 - 1, nr = tiles_of(bb0), lim = 0, issued = 0, bad = 0;
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
      enter();
      int ra = 0, rb = 0, key0 = 0;  // rows of keys lane and 32 + lane of the current tile
      bool start = false;
      auto next_tile = [&]() {
        if (++jt == nr) {
          jt = 0;
          nr = tiles_of(++bb);
          enter();
        }
        key0 = jt * KT;
        start = jt == 0;
        ra = rb = p.pool.rows;
        if (key0 + lane < lim) ra = row_of(p.pool, trow, key0 + lane);
        if (key0 + 32 + lane < lim) rb = row_of(p.pool, trow, key0 + 32 + lane);
      };
      // entries outside the pool, each page of a sequence once
      auto count_bad = [&]() {
        if (rank == 0 && kw == 0 && last) {
          const int a = key0 + lane, b = a + 32;
          bad += a < lim && ra == p.pool.rows && a % p.pool.page_size == 0;
          bad += b < lim && rb == p.pool.rows && b % p.pool.page_size == 0;
        }
      };
      if constexpr (!kE4M3) {
        next_tile();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int s = i % NST;
          count_bad();
          const int xa = ra, xb = rb;
          const bool boxes = p.box && key0 + KT <= lim;
          const uint32_t st_start = i == 0 || start ? 1u : 0u;
          if (i + 1 < n) next_tile();
          if (!warp_wait(&bars.empty[s], ((i / NST) & 1) ^ 1, abort, p.status)) break;
          if (lane == 0) {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(sbase + OFF_ROWSTART + s * 4),
                         "r"(st_start)
                         : "memory");
            mbar_arrive_expect_tx(&bars.full[s], ST_BYTES);
          }
          __syncwarp();
          const uint32_t stage = sbase + s * ST_BYTES;
          if (boxes) {
            // whole boxes of rows: every page boundary is a box boundary
            const int k0 = (lane * p.box) & 63;
            const int ya = __shfl_sync(0xffffffffu, xa, k0 & 31);
            const int yb = __shfl_sync(0xffffffffu, xb, k0 & 31);
            const int y = k0 < 32 ? ya : yb;
            if (lane * p.box < KT) {
#pragma unroll
              for (int a = 0; a < 4; ++a)
                tma_load_2d(stage + a * ST_ATOM + k0 * 128, &map_c, rank * 256 + a * 64, y,
                            &bars.full[s]);
              tma_load_2d(stage + ST_KR + k0 * 64, &map_r, rank * 32, y, &bars.full[s]);
            }
          } else {
            // row by row: the tile's rows past the limit read as zeros, so
            // that nothing stored there can reach a product
            const int k0 = 4 * (lane & 15), src = k0 & 31;
            int y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int ya = __shfl_sync(0xffffffffu, xa, src + j);
              const int yb = __shfl_sync(0xffffffffu, xb, src + j);
              y[j] = k0 < 32 ? ya : yb;
            }
            if (lane < 16) {
#pragma unroll
              for (int a = 0; a < 4; ++a)
                tma_gather4(stage + a * ST_ATOM + k0 * 128, &map_c1, rank * 256 + a * 64, y[0],
                            y[1], y[2], y[3], &bars.full[s]);
              tma_gather4(stage + ST_KR + k0 * 64, &map_r1, rank * 32, y[0], y[1], y[2], y[3],
                          &bars.full[s]);
            }
          }
          issued = i + 1;
        }
        // on an abort, the loads still in flight land before the CTA can leave
        for (int t = max(0, issued - NST); t < issued; ++t)
          warp_wait(&bars.full[t % NST], (t / NST) & 1, nullptr, nullptr);
      } else {
        // two rows per warp and step: lane = (row of the pair, 16-code chunk)
        constexpr int STEPS = (KT / 2 + NKEY - 1) / NKEY;
        const int rsel = lane >> 4, ch = lane & 15;
        uint4 code[STEPS], rope[2];
        float sc[STEPS];
        auto load = [&]() {
#pragma unroll
          for (int it = 0; it < STEPS; ++it) {
            const int row = 2 * (kw + NKEY * it) + rsel;
            const int ya = __shfl_sync(0xffffffffu, ra, row & 31);
            const int yb = __shfl_sync(0xffffffffu, rb, row & 31);
            const int y = row < 32 ? ya : yb;
            code[it] = make_uint4(0, 0, 0, 0);
            sc[it] = 1.f;
            if (row < KT && y < p.pool.rows) {
              const uint8_t* src = p.pool.base + (long long)y * p.pool.row_stride;
              code[it] = ld_global_nc_v4(src + rank * 256 + ch * 16);
              sc[it] = u2f((uint32_t)ld_global_nc_s32_early(reinterpret_cast<const int32_t*>(
                  src + pages::kScaleOff + (rank * 2 + (ch >> 3)) * 4)));
            }
          }
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int u = kw * 32 + lane + it * NKEY * 32;  // (row, 16-byte chunk) of the rotary half
            const int row = (u >> 2) & 63;
            const int ya = __shfl_sync(0xffffffffu, ra, row & 31);
            const int yb = __shfl_sync(0xffffffffu, rb, row & 31);
            const int y = row < 32 ? ya : yb;
            rope[it] = make_uint4(0, 0, 0, 0);
            if (u < KT * 4 && y < p.pool.rows)
              rope[it] = ld_global_nc_v4(p.pool.base + (long long)y * p.pool.row_stride +
                                         pages::kRopeOff + rank * 64 + (u & 3) * 16);
          }
        };
        next_tile();
        load();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int s = i % NST;
          count_bad();
          const uint32_t st_start = i == 0 || start ? 1u : 0u;
          if (i + 1 < n) next_tile();
          if (!warp_wait(&bars.empty[s], ((i / NST) & 1) ^ 1, abort, p.status)) break;
          const uint32_t stage = sbase + s * ST_BYTES;
          if (kw == 0 && lane == 0)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(sbase + OFF_ROWSTART + s * 4),
                         "r"(st_start)
                         : "memory");
#pragma unroll
          for (int it = 0; it < STEPS; ++it) {
            const int row = 2 * (kw + NKEY * it) + rsel;
            if (row >= KT) continue;
            uint4 o0, o1;
            pages::dequant16(code[it], sc[it], o0, o1);
            const uint32_t atom = stage + (ch >> 2) * ST_ATOM;
            const int c2 = (ch & 3) * 2;
            st_shared_v4(atom + sw128_off(row, c2), o0.x, o0.y, o0.z, o0.w);
            st_shared_v4(atom + sw128_off(row, c2 + 1), o1.x, o1.y, o1.z, o1.w);
          }
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int u = kw * 32 + lane + it * NKEY * 32;
            if (u < KT * 4)
              st_shared_v4(stage + ST_KR + sw64_off(u >> 2, u & 3), rope[it].x, rope[it].y,
                           rope[it].z, rope[it].w);
          }
          if (i + 1 < n) load();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.full[s]);
        }
      }
      bad = __reduce_add_sync(0xffffffffu, bad);
      if (lane == 0 && bad && p.status) atomicAdd(p.status + 1, bad);
    }
  } else if (warp == MMA_WARP) {
    // ---------------- MMA issuer ----------------
    // A value product goes first whenever its P is ready; the score product of
    // tile i + 2 follows the value product of tile i, whose P it overwrites
    // (products of one thread run in the order they are issued).  The whole
    // warp runs the loop and an elected lane issues: under elect.sync the
    // compiler keeps descriptors in uniform registers, 20 cycles an issue
    // against 50 from a branch on the lane number, which was more than the 32
    // cycles such a product takes.
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, KT, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 256, 0, 1);
    constexpr uint32_t hi_k128 = desc_hi(1024, kSwizzle128B);
    constexpr uint32_t hi_k64 = desc_hi(512, kSwizzle64B);
    const uint32_t lo_qr = desc_lo(sbase + OFF_QR, 16);
    auto test = [](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0;
    };
    int qk = 0, pv = 0, idle = 0, qseg = -1;
    int qs = 0, qph = 0, ps = 0;
    uint64_t t_idle = 0;
#pragma unroll 1
    while (pv < n) {
      bool did = false;
      if (pv < qk && test(&bars.p_full[pv & 1], (pv >> 1) & 1)) {
        tc_fence_after();
        const uint32_t lo = desc_lo(sbase + ps * ST_BYTES, ST_ATOM);  // V, MN-major
        const uint32_t tp = tmem + T_S + (pv & 1) * KT;
        const uint32_t first = ld_shared_u32(sbase + OFF_ROWSTART + ps * 4);
        if (elect_one()) {
          tc_mma_tmem_a(tmem + T_O, tp, desc_join(lo, hi_k128), idesc_pv, first ^ 1u);
#pragma unroll
          for (int ks = 1; ks < KT / 16; ++ks)
            tc_mma_tmem_a_c<true>(tmem + T_O, tp + ks * 8,
                                  desc_join(lo + ks * (2048 >> 4), hi_k128), idesc_pv);
          tc_commit(&bars.o_done[pv & 1]);
          tc_commit(&bars.empty[ps]);
        }
        __syncwarp();
        ++pv;
        if (++ps == NST) ps = 0;
        did = true;
      }
      if (qk < n && qk < pv + 2 && test(&bars.full[qs], qph)) {
        const int seg = ld_shared_u32(sbase + OFF_ROWSTART + qs * 4) ? qseg + 1 : qseg;
        if (seg == qseg || test(&bars.q_ready, seg & 1)) {
          qseg = seg;
          tc_fence_after();
          const uint32_t st = sbase + qs * ST_BYTES;
          const uint32_t lo = desc_lo(st, 16), lo_r = desc_lo(st + ST_KR, 16);
          const uint32_t ts = tmem + T_S + (qk & 1) * KT;
          if (elect_one()) {
            tc_mma_tmem_a_c<false>(ts, tmem + T_Q, desc_join(lo, hi_k128), idesc_qk);
#pragma unroll
            for (int ks = 1; ks < 16; ++ks)
              tc_mma_tmem_a_c<true>(
                  ts, tmem + T_Q + ks * 8,
                  desc_join(lo + (((ks >> 2) * ST_ATOM + (ks & 3) * 32) >> 4), hi_k128), idesc_qk);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              tc_mma_c<true>(ts, desc_join(lo_qr + ks * 2, hi_k64),
                             desc_join(lo_r + ks * 2, hi_k64), idesc_qk);
            tc_commit(&bars.s_full[qk & 1]);
          }
          __syncwarp();
          ++qk;
          if (++qs == NST) {
            qs = 0;
            qph ^= 1;
          }
          did = true;
        }
      }
      if (did) {
        idle = 0;
        t_idle = 0;
      } else if (++idle >= 64) {
        idle = 0;
        if (__any_sync(0xffffffffu, *abort != 0)) break;
        const uint64_t now = __shfl_sync(0xffffffffu, globaltimer_ns(), 0);
        if (t_idle == 0) {
          t_idle = now;
        } else if (now - t_idle > kWaitLimitNs) {
          if (lane == 0) {
            *abort = 1;
            report_timeout(p.status);
          }
          break;
        }
      }
    }
    // everything issued so far has finished before TMEM is released
    if (elect_one()) tc_commit(&bars.drain);
    __syncwarp();
    warp_wait(&bars.drain, 0, nullptr, p.status);
  } else if (warp >= SEND_WARP0) {
    // ---------------- senders ----------------
    // Lane quarter q as two 16-lane halves in the 16x256b fragment order of
    // softmax warps q and q + 4: register 4k + e of half hf is 16-byte chunk k
    // of softmax warp q + 4 hf.
    const int q4 = warp - SEND_WARP0;
    const uint32_t xs_peer = mapa_shared(sbase + OFF_XS + lane * 16, peer);
    const uint32_t xs_full_peer = mapa_shared(smem_u32(&bars.xs_full[0]), peer);
    // the quarter's 32 rows of this CTA's half of Q~ for token bb (one row
    // per thread): latent values into TMEM as bf16 pairs, rotary values into
    // the swizzled shared tile
    auto load_q = [&](int bb) {
      const int h = q4 * 32 + lane;
      const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
      const __nv_bfloat16* qrow = p.q_tilde + ((size_t)bb * kH + h) * kC + rank * 256;
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        uint4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = ld_global_nc_v4(qrow + c * 64 + i * 8);
#pragma unroll
        for (int hc = 0; hc < 2; ++hc) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r[4 * i] = v[8 * hc + i].x;
            r[4 * i + 1] = v[8 * hc + i].y;
            r[4 * i + 2] = v[8 * hc + i].z;
            r[4 * i + 3] = v[8 * hc + i].w;
          }
          tmem_st32(tmem + lane_base + T_Q + (c + hc) * 32, r);
        }
      }
      const __nv_bfloat16* rrow = p.q_pe + ((size_t)bb * kH + h) * kR + rank * 32;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = ld_global_nc_v4(rrow + c * 8);
        st_shared_v4(sbase + OFF_QR + sw64_off(h, c), v.x, v.y, v.z, v.w);
      }
      fence_proxy_async_smem();
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_ready);
    };
    // this thread's part of the next token's queries into L2, a token ahead
    auto prefetch_q = [&](int i, const Pos& c) {
      if (i + c.nr - c.jt >= n) return;
      const int h = q4 * 32 + lane;
      const __nv_bfloat16* qrow = p.q_tilde + ((size_t)(c.bb + 1) * kH + h) * kC + rank * 256;
#pragma unroll
      for (int j = 0; j < 4; ++j) prefetch_l2(qrow + j * 64);
      prefetch_l2(p.q_pe + ((size_t)(c.bb + 1) * kH + h) * kR + rank * 32);
    };
    pdl_wait();  // q~ is the fold kernel's output (the other roles read only inputs and the plan)
    load_q(bb0);
    Pos c = {bb0, jt0, tiles_of(bb0)};
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int b = i & 1, ph = (i >> 1) & 1;
      if (i == 0 || c.jt == 0) prefetch_q(i, c);
      if (!warp_wait(&bars.s_full[b], ph, abort, p.status)) break;
      tc_fence_after();
      uint32_t r[2][32];
      tmem_ld_16x256b_x8(tmem + ((uint32_t)(q4 * 32) << 16) + T_S + b * KT, r[0]);
      tmem_ld_16x256b_x8(tmem + ((uint32_t)(q4 * 32 + 16) << 16) + T_S + b * KT, r[1]);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      // relaxed: the tcgen05 loads have completed (waited for above)
      if (lane == 0) mbar_arrive_relaxed(&bars.sent[b]);
      // the peer has read its buffer of tile i - 2
      if (!warp_wait<true>(&bars.xs_free[b], ph ^ 1, abort, p.status)) break;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          st_async_u4(xs_peer + b * XS_BYTES + (q4 + 4 * hf) * 4096 + k * 512, r[hf][4 * k],
                      r[hf][4 * k + 1], r[hf][4 * k + 2], r[hf][4 * k + 3],
                      xs_full_peer + b * 8);
      // the token's last score product is done: its queries make room for the
      // next token's
      if (c.jt == c.nr - 1 && i + 1 < n) load_q(c.bb + 1);
      if (++c.jt == c.nr) {
        c.jt = 0;
        c.nr = tiles_of(++c.bb);
      }
    }
  } else {
    // ---------------- softmax: rows [32q + 16h, +16), all keys ----------------
    // Through the 16x256b TMEM shape thread t holds rows t/4 and t/4 + 8 of
    // its 16 and, of each 8-key block j, keys 8j + 2(t%4) and 8j + 2(t%4) + 1:
    // register 4j+e is (row t/4 + 8 (e/2), key 8j + 2(t%4) + e%2).
    const int q4 = warp & 3, hf = warp >> 2;
    const int c4 = lane & 3;
    const int row0 = q4 * 32 + hf * 16 + (lane >> 2), row1 = row0 + 8;
    const uint32_t frag = (uint32_t)(q4 * 32 + hf * 16) << 16;
    const uint32_t xs_own = sbase + OFF_XS + warp * 4096 + lane * 16;
    const uint32_t xs_free_peer = mapa_shared(smem_u32(&bars.xs_free[0]), peer);
    bool alive = true;

    auto wait_pv = [&](int t) -> bool {  // the value product of tile t has completed
      if (!warp_wait(&bars.o_done[t & 1], (t >> 1) & 1, abort, p.status)) return false;
      tc_fence_after();
      return true;
    };
    auto rescale_o = [&](float a0, float a1) {
#pragma unroll 1
      for (int cc = 0; cc < 256; cc += 32) {
        uint32_t r[16];
        const uint32_t ta = tmem + frag + T_O + cc;
        tmem_ld_16x256b_x4(ta, r);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[4 * j] = f2u(u2f(r[4 * j]) * a0);
          r[4 * j + 1] = f2u(u2f(r[4 * j + 1]) * a0);
          r[4 * j + 2] = f2u(u2f(r[4 * j + 2]) * a1);
          r[4 * j + 3] = f2u(u2f(r[4 * j + 3]) * a1);
        }
        tmem_st_16x256b_x4(ta, r);
      }
      tc_wait_st();
    };
    float m0 = -INFINITY, m1 = -INFINITY;  // running maxima of the two rows (log2 units)
    float l0 = 0.f, l1 = 0.f;              // this thread's parts of their row sums
    // A segment's end: this thread's rows of this CTA's half of O~ / l into the
    // token's output (a token held whole by this pair), or rounded to bf16 into
    // the pair's slot (0: the range's first segment, 1: its last) with the
    // segment's log-sum-exps
    auto flush = [&](int i_last, int bb, bool partial, int slot1) -> bool {
      float t0 = l0 + __shfl_xor_sync(0xffffffffu, l0, 1);
      t0 += __shfl_xor_sync(0xffffffffu, t0, 2);
      float t1 = l1 + __shfl_xor_sync(0xffffffffu, l1, 1);
      t1 += __shfl_xor_sync(0xffffffffu, t1, 2);
      if (!wait_pv(i_last)) return false;
      const int slot = 2 * cid + slot1;
      const float inv0 = t0 > 0.f ? 1.f / t0 : (t0 == 0.f ? 0.f : t0);
      const float inv1 = t1 > 0.f ? 1.f / t1 : (t1 == 0.f ? 0.f : t1);
      __nv_bfloat16* dst0 = (!partial ? p.omerged + ((size_t)bb * kH + row0) * kC
                                      : p.opart + ((size_t)slot * kH + row0) * kC) +
                            rank * 256 + 2 * c4;
      __nv_bfloat16* dst1 = dst0 + 8 * kC;
      uint32_t r[16];
#pragma unroll 1
      for (int cc = 0; cc < 256; cc += 32) {
        tmem_ld_16x256b_x4(tmem + frag + T_O + cc, r);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          *reinterpret_cast<uint32_t*>(dst0 + cc + 8 * j) =
              pack_bf16x2(u2f(r[4 * j]) * inv0, u2f(r[4 * j + 1]) * inv0);
          *reinterpret_cast<uint32_t*>(dst1 + cc + 8 * j) =
              pack_bf16x2(u2f(r[4 * j + 2]) * inv1, u2f(r[4 * j + 3]) * inv1);
        }
      }
      tc_fence_before();
      if (partial && rank == 0 && c4 == 0) {
        float* lse = p.lse + (size_t)slot * kH;
        lse[row0] = t0 == 0.f ? -INFINITY : m0 + log2f(t0);
        lse[row1] = t1 == 0.f ? -INFINITY : m1 + log2f(t1);
      }
      return true;
    };
    float x[32];
    Pos c = {bb0, jt0, tiles_of(bb0)};
    int lim = lim_of(bb0);
    int prev_bb = bb0, nx = 0;
    bool open = false;  // the last tile processed is not its token's last
    int nseg = 0;       // segments written out
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int b = i & 1, ph = (i >> 1) & 1;
      const bool first = i == 0 || c.jt == 0;
      if (first && i > 0) {
        if (!flush(i - 1, prev_bb, nseg == 0 && jt0 > 0, 0)) { alive = false; break; }
        ++nseg;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
      }
      if (!warp_wait(&bars.s_full[b], ph, abort, p.status)) { alive = false; break; }
      tc_fence_after();
      {
        uint32_t own[32];
        tmem_ld_16x256b_x8(tmem + frag + T_S + b * KT, own);
        if (!warp_wait<true>(&bars.xs_full[b], ph, abort, p.status)) { alive = false; break; }
        nx = i + 1;
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = ld_shared_v4(xs_own + b * XS_BYTES + k * 512);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[4 * k] = u2f(own[4 * k]) + u2f(v[k].x);
          x[4 * k + 1] = u2f(own[4 * k + 1]) + u2f(v[k].y);
          x[4 * k + 2] = u2f(own[4 * k + 2]) + u2f(v[k].z);
          x[4 * k + 3] = u2f(own[4 * k + 3]) + u2f(v[k].w);
        }
      }
      // the sums are computed (so the buffer's loads have returned) before the
      // relaxed arrives below
#pragma unroll
      for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(x[j]));
      __syncwarp();
      if (lane == 0) {
        if (warp == 0 && i + 2 < n) mbar_arrive_expect_tx_relaxed(&bars.xs_full[b], XS_BYTES);
        mbar_arrive_cluster_relaxed(xs_free_peer + b * 8);
      }
      // scale to log2 units; mask the token's last tile; row maxima
      const int left = lim - c.jt * KT;
      float mt0 = -INFINITY, mt1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] *= p.scale_log2;
      if (left < KT) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if ((j >> 2) * 8 + 2 * c4 + (j & 1) >= left) x[j] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mt0 = fmaxf(mt0, fmaxf(x[4 * j], x[4 * j + 1]));
        mt1 = fmaxf(mt1, fmaxf(x[4 * j + 2], x[4 * j + 3]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mt0 = fmaxf(mt0, __shfl_xor_sync(0xffffffffu, mt0, o));
        mt1 = fmaxf(mt1, __shfl_xor_sync(0xffffffffu, mt1, o));
      }
      const bool resc0 = mt0 > m0 + kRescaleThreshold, resc1 = mt1 > m1 + kRescaleThreshold;
      if (!first && __any_sync(0xffffffffu, resc0 || resc1)) {
        // O~ must hold the value product of tile i - 1 before it is scaled
        if (!wait_pv(i - 1)) { alive = false; break; }
        rescale_o(resc0 ? fast_exp2(m0 - mt0) : 1.f, resc1 ? fast_exp2(m1 - mt1) : 1.f);
      }
      if (resc0) {
        l0 *= first ? 0.f : fast_exp2(m0 - mt0);
        m0 = mt0;
      }
      if (resc1) {
        l1 *= first ? 0.f : fast_exp2(m1 - mt1);
        m1 = mt1;
      }
      // P over the scores once the senders have read them too
      {
        // (a row that has seen no key yet has m = -inf: its P is exp2(-inf) = 0)
        const float d0 = m0 == -INFINITY ? 0.f : m0, d1 = m1 == -INFINITY ? 0.f : m1;
        uint32_t w[16];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e0 = fast_exp2(x[4 * j] - d0), e1 = fast_exp2(x[4 * j + 1] - d0);
          const float e2 = fast_exp2(x[4 * j + 2] - d1), e3 = fast_exp2(x[4 * j + 3] - d1);
          s0 += e0 + e1;
          s1 += e2 + e3;
          w[2 * j] = pack_bf16x2(e0, e1);
          w[2 * j + 1] = pack_bf16x2(e2, e3);
        }
        l0 += s0;
        l1 += s1;
        if (!warp_wait(&bars.sent[b], ph, abort, p.status)) { alive = false; break; }
        tc_fence_after();
        tmem_st_16x128b_x8(tmem + frag + T_S + b * KT, w);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[b]);
      prev_bb = c.bb;
      open = c.jt != c.nr - 1;
      if (++c.jt == c.nr) {
        c.jt = 0;
        c.nr = tiles_of(++c.bb);
        lim = lim_of(c.bb);
      }
    }
    // on an abort, partial scores the peer may still be sending land before
    // the CTA can leave: the armed, unconsumed phases (none on the normal path)
    for (int t = nx; t < n && t < nx + 2; ++t)
      warp_wait<true>(&bars.xs_full[t & 1], (t >> 1) & 1, nullptr, nullptr);
    if (__all_sync(0xffffffffu, alive) && !*abort)
      flush(n - 1, prev_bb, (nseg == 0 && jt0 > 0) || open, nseg == 0 ? 0 : 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
  // neither CTA leaves while its peer may still touch its shared memory
  cluster_sync_all();
}

// ===========================================================================
// merge: O~ = sum_s 2^(lse_s - max) O~_s / sum_s 2^(lse_s - max) over the
// segments of a token that several pairs held.  Grid (range boundaries
// 1 .. pairs-1, heads); boundary c serves the token it falls inside when it is
// the token's first one.  256 threads: 64 16-byte chunks of the head's latent,
// four threads each over every fourth segment.
// ===========================================================================
constexpr int kMaxPairs = 512;

__global__ void __launch_bounds__(256) merge_kernel(const __nv_bfloat16* __restrict__ opart,
                                                     const float* __restrict__ lse, const Plan pl,
                                                     int nc, __nv_bfloat16* __restrict__ omerged) {
  __shared__ float w[kMaxPairs];
  __shared__ int slots[kMaxPairs];
  __shared__ int count;
  __shared__ float acc_s[3][64][8];
  __shared__ float wsum;
  const int cb = blockIdx.x + 1, h = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  // every block waits, those with nothing to merge too: the value kernel
  // relies on this grid's completion implying the attend kernel's
  pdl_wait();
  const int t = ld_global_nc_s32_early(pl.tb + cb);
  const int b = ld_global_nc_s32_early(pl.crow + cb);
  if (b >= ld_global_nc_s32_early(pl.nact)) return;
  const int rs = ld_global_nc_s32_early(pl.tstart + b);
  const int re = ld_global_nc_s32_early(pl.tstart + b + 1);
  const int before = ld_global_nc_s32_early(pl.tb + cb - 1);
  if (rs == t || before > rs) return;
  // segments in pair order: slot 1 of pair cb - 1 (slot 0 when the token
  // starts its range), slot 0 of every later pair whose range starts inside
  // the token and is not empty
  if (tid < 32) {
    int have = 1;
    if (tid == 0) slots[0] = 2 * (cb - 1) + (rs > before ? 1 : 0);
    for (int c0 = cb; c0 < nc; c0 += 32) {
      const int c = c0 + tid;
      const int a = c < nc ? ld_global_nc_s32_early(pl.tb + c) : re;
      const int e = c < nc ? ld_global_nc_s32_early(pl.tb + c + 1) : re;
      const bool in = a < re && e > a;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      const int at = have + __popc(m & ((1u << tid) - 1u));
      if (in) slots[at] = 2 * c;
      have += __popc(m);
      if (!__any_sync(0xffffffffu, a < re)) break;
    }
    __syncwarp();
    float mx = -INFINITY;
    for (int i = tid; i < have; i += 32) {
      const float l = lse[(size_t)slots[i] * kH + h];
      w[i] = l;
      mx = fmaxf(mx, l);  // (drops a NaN, which the weights below keep)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float s = 0.f;
    for (int i = tid; i < have; i += 32) {
      const float e = w[i] == -INFINITY ? 0.f : exp2f(w[i] - mx);
      w[i] = e;
      s += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tid == 0) {
      count = have;
      wsum = s;
    }
  }
  __syncthreads();
  const int n = count;
  const int ch = tid & 63, g = tid >> 6;
  const __nv_bfloat16* src = opart + (size_t)h * kC + ch * 8;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = g; i < n; i += 4) {
    const uint4 v = ld_global_nc_v4(src + (size_t)slots[i] * kH * kC);
    const float wi = w[i];
    const __nv_bfloat162* pv = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(pv[e]);
      acc[2 * e] += wi * f.x;
      acc[2 * e + 1] += wi * f.y;
    }
  }
  if (g > 0)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc_s[g - 1][ch][e] = acc[e];
  __syncthreads();
  if (g == 0) {
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += acc_s[k][ch][e];
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    uint4 o;
    o.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    o.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    o.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    o.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4*>(omerged + ((size_t)b * kH + h) * kC + ch * 8) = o;
  }
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
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(absorbed_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SMEM_BYTES) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, absorbed_kernel<false>, &cfg) != cudaSuccess || n < 1) {
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
  size_t q_tilde, opart, lse, omerged, seq, lim, tstart, tb, crow, nact, total;
};

static AbsorbedWs absorbed_ws(int N, int nc) {
  AbsorbedWs w;
  w.q_tilde = 0;
  w.opart = round_up((size_t)N * kH * kC * 2, 256);
  w.lse = w.opart + (size_t)nc * 2 * kH * kC * 2;
  w.omerged = round_up(w.lse + (size_t)nc * 2 * kH * 4, 256);
  w.seq = round_up(w.omerged + (size_t)N * kH * kC * 2, 256);
  w.lim = round_up(w.seq + (size_t)N * 4, 256);
  w.tstart = round_up(w.lim + (size_t)N * 4, 256);
  w.tb = round_up(w.tstart + (size_t)(N + 1) * 4, 256);
  w.crow = round_up(w.tb + (size_t)(nc + 1) * 4, 256);
  w.nact = round_up(w.crow + (size_t)(nc + 1) * 4, 256);
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
  alignas(64) CUtensorMap map_c = {}, map_r = {}, map_c1 = {}, map_r1 = {};
  if (!kE4M3) {
    const uint8_t* lat = p.pool.base;
    const uint8_t* rot = p.pool.base + kC * 2;
    const uint64_t rows = p.pool.rows, rb = p.pool.row_stride;
    const int box = p.box ? p.box : 1;
    const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    if (int e = bf16_map_2d(&map_c, lat, kC, rows, rb, 64, box, CU_TENSOR_MAP_SWIZZLE_128B, l2))
      return e;
    if (int e = bf16_map_2d(&map_r, rot, kR, rows, rb, 32, box, CU_TENSOR_MAP_SWIZZLE_64B, l2))
      return e;
    if (int e = bf16_map_2d(&map_c1, lat, kC, rows, rb, 64, 1, CU_TENSOR_MAP_SWIZZLE_128B, l2))
      return e;
    if (int e = bf16_map_2d(&map_r1, rot, kR, rows, rb, 32, 1, CU_TENSOR_MAP_SWIZZLE_64B, l2))
      return e;
  }
  static std::atomic<unsigned long long> attr_done{0};
  if (int e = ensure_smem_attr(absorbed_kernel<kE4M3>, SMEM_BYTES, &attr_done)) return e;
  return launch_pdl(absorbed_kernel<kE4M3>, dim3(2 * nc), dim3(NTHREADS), SMEM_BYTES, st, p, map_c,
                    map_r, map_c1, map_r1);
}

static int run_absorbed(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
                        const Pool& pool, const Seqs& q, float scale, mla_bf16_t* O, uint8_t* ws,
                        int32_t* status, cudaStream_t st) {
  const int nc = max_pairs();
  const AbsorbedWs L = absorbed_ws(q.N, nc);
  Plan pl;
  pl.seq = reinterpret_cast<int32_t*>(ws + L.seq);
  pl.lim = reinterpret_cast<int32_t*>(ws + L.lim);
  pl.tstart = reinterpret_cast<int32_t*>(ws + L.tstart);
  pl.tb = reinterpret_cast<int32_t*>(ws + L.tb);
  pl.crow = reinterpret_cast<int32_t*>(ws + L.crow);
  pl.nact = reinterpret_cast<int32_t*>(ws + L.nact);
  __nv_bfloat16* q_tilde = reinterpret_cast<__nv_bfloat16*>(ws + L.q_tilde);
  // plain launch: complete before the fold starts, so the attend kernel, which
  // may start during the fold, finds the plan
  plan_kernel<<<1, 1024, 0, st>>>(q, pool, pl, nc);
  if (int e = launch_status()) return e;
  if (int e = mla_fold_wuk(q_nope, wkv_b, q.N, reinterpret_cast<mla_bf16_t*>(q_tilde), st))
    return e;
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
  p.omerged = reinterpret_cast<__nv_bfloat16*>(ws + L.omerged);
  p.status = status;
  if (int e = pool.kind == MLA_PAGE_E4M3 ? launch_absorbed<true>(p, nc, st)
                                         : launch_absorbed<false>(p, nc, st))
    return e;
  if (nc > 1)
    if (int e = launch_pdl(merge_kernel, dim3(nc - 1, kH), dim3(256), 0, st,
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

// The form of a call: as asked, or by the new tokens per sequence.
static int form_of(int form, int N, int S) {
  if (form != MLA_FORM_AUTO) return form;
  return (int64_t)N >= (int64_t)S * expand::kMinTokens ? MLA_FORM_EXPANDED : MLA_FORM_ABSORBED;
}

static int check_sizes(int N, int S, int max_kv, int form) {
  if (N < 1 || N > 65535 || S < 1 || S > 65535 || max_kv < 1 || max_kv > (1 << 24))
    return MLA_ERR_SHAPE;
  if (form < MLA_FORM_AUTO || form > MLA_FORM_EXPANDED) return MLA_ERR_SHAPE;
  // absorbed: the flattened list of (token, 64-key tile) is counted in 32 bits
  if (form_of(form, N, S) == MLA_FORM_EXPANDED ? !expand::fits(S, max_kv)
                                               : (int64_t)N * ((max_kv + 63) / 64) > 0x3fffffff)
    return MLA_ERR_SHAPE;
  return MLA_OK;
}

extern "C" size_t mla_attend_paged_workspace_bytes(int N, int S, int max_kv, int form) {
  if (check_sizes(N, S, max_kv, form) != MLA_OK) return 0;
  if (form_of(form, N, S) == MLA_FORM_EXPANDED) return expand::workspace_bytes(N, S, max_kv);
  return paged::absorbed_ws(N, paged::max_pairs()).total;
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
  if (int e = check_sizes(N, S, max_kv, form)) return e;
  // (written so that a NaN is refused too)
  if (max_pages < 1 || !(scale > 0.f && scale <= 3.0e38f)) return MLA_ERR_SHAPE;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(wkv_b) || !aligned16(O))
    return MLA_ERR_ALIGN;
  if (!ws || !aligned256(ws)) return MLA_ERR_WORKSPACE;
  if (int e = check_device()) return e;
  if (ws_bytes < mla_attend_paged_workspace_bytes(N, S, max_kv, form)) return MLA_ERR_WORKSPACE;
  paged::Pool p;
  p.base = static_cast<const uint8_t*>(pool);
  p.kind = kind;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.pitch = (int)(page_stride / row_stride);
  p.row_stride = row_stride;
  p.rows = (num_pages - 1) * p.pitch + page_size;
  p.table = page_table;
  p.max_pages = max_pages;
  paged::Seqs q;
  q.cu_q = cu_q;
  q.kv_len = kv_len;
  q.S = S;
  q.N = N;
  q.max_kv = max_kv;
  if (form_of(form, N, S) == MLA_FORM_EXPANDED)
    return expand::run(q_nope, q_pe, wkv_b, p, q, scale, O, static_cast<uint8_t*>(ws), status,
                       as_stream(stream));
  return paged::run_absorbed(q_nope, q_pe, wkv_b, p, q, scale, O, static_cast<uint8_t*>(ws),
                             status, as_stream(stream));
}
