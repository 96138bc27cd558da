/*
 * libshla -- absorbed sparse multi-head latent attention decode for B200
 * (sm_100a): the decode step of DeepSeek-V3.2-Exp's sparse latent attention,
 * with W_UK folded into the queries and W_UV applied after the latent mix.
 *
 * C ABI.  All tensor arguments are DEVICE pointers owned by the caller; the
 * library never allocates, frees or keeps per-call state, and it keeps no
 * pointer after a call returns.  Every compute entry point only enqueues work
 * on the given CUDA stream (``stream`` is a cudaStream_t; NULL = legacy
 * default stream) and returns at once.
 *
 * Element types:
 *   bf16  = 16-bit brain float, passed as raw bits (mla_bf16_t)
 *   fp32  = IEEE float
 *   int32 = int32_t
 * All arrays are row-major.  Unless a stride argument says otherwise, they are
 * contiguous.  Base pointers and row strides of every bf16/fp32 array must be
 * 16-byte aligned (MLA_ERR_ALIGN otherwise).
 *
 * Model dimensions are fixed ("Key heads" page, MLA init listing; "KV
 * compression" page):
 *   H  = 128 heads
 *   C  = 512 latent width (kv_lora_rank)
 *   R  = 64 shared rotary key width (qk_rope_head_dim)
 *   Dn = 128 non-rotary query/key width, Dv = 128 value width
 *   DIM = 7168 model width
 *
 * Return value: MLA_OK (0), or a negative MLA_ERR_* code for a synchronous
 * error found before anything was enqueued.  Asynchronous conditions go into
 * an optional caller-owned device int32 status[2]:
 *   status[0] |= MLA_STATUS_TIMEOUT  if a kernel gave up a bounded wait (the
 *                                    output is then undefined);
 *   status[1] += count of top-k entries that are neither -1 nor inside
 *                [0, min(end_pos[b], T)) (they are ignored).
 * The library never clears the status word.
 */
#ifndef SHLA_H_
#define SHLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t mla_bf16_t;

enum {
  MLA_OK = 0,
  MLA_ERR_NULL = -1,        /* a required pointer is NULL */
  MLA_ERR_SHAPE = -2,       /* a size or stride is out of range */
  MLA_ERR_ALIGN = -3,       /* a pointer or stride breaks 16-byte alignment */
  MLA_ERR_WORKSPACE = -4,   /* workspace pointer NULL or too small */
  MLA_ERR_UNSUPPORTED = -5, /* device is not sm_100 */
  MLA_ERR_CUDA = -6,        /* a CUDA launch or attribute call failed */
  MLA_ERR_OVERLAP = -7      /* an output or the workspace shares memory with another argument */
};

#define MLA_STATUS_TIMEOUT 1

#define MLA_HEADS 128
#define MLA_LATENT 512
#define MLA_ROPE 64
#define MLA_NOPE 128
#define MLA_VDIM 128
#define MLA_ROW 576
#define MLA_DIM 7168

/* Kinds of cache pages (mla_page_write) and forms of mla_attend_paged. */
#define MLA_PAGE_BF16 0
#define MLA_PAGE_E4M3 1
#define MLA_PAGE_ROW8 656
#define MLA_FORM_AUTO 0
#define MLA_FORM_ABSORBED 1
#define MLA_FORM_EXPANDED 2

/* Human-readable text for a return code.  Static storage; never NULL. */
const char* mla_status_string(int code);

/*
 * Rotary embedding of feature pairs ("Rotated shared key" page,
 * the apply_rotary_emb code excerpt).
 *   x    bf16  [B, S, Hx, 64]
 *   rope fp32  [S, 32, 2]: (cos, sin) of the angle for sequence slot s and
 *              pair j; slot s of x uses row s (the caller offsets the table to
 *              the first position)
 *   interleaved != 0: pair j = (x[2j], x[2j+1]); result written back to
 *              (2j, 2j+1).  interleaved == 0: pair j = (x[j], x[j+32]); result
 *              written as all real parts then all imaginary parts.
 *   y    bf16  [B, S, Hx, 64]; may equal x (in place)
 * Rotation in fp32, one rounding to bf16.
 */
int mla_rope(const mla_bf16_t* x, const float* rope, int B, int S, int Hx, int interleaved,
             mla_bf16_t* y, void* stream);

/*
 * Cache write for new positions ("KV compression" page: the key-value
 * down-projection code excerpt, and its Explanation of the 576 values cached
 * per position):
 *   kv = x W_KVa (fp32 accumulation); latent = RMSNorm(kv[0:512]) * norm_w
 *   (y = v / sqrt(mean(v^2) + eps) * w, fp32); k_pe = interleaved RoPE of
 *   kv[512:576] at the row's position; both stored as bf16.
 *   x       bf16 [B, S, 7168]
 *   w_kva   bf16 [7168, 576]   (x W form: row i holds input feature i)
 *   norm_w  bf16 [512]
 *   rope    fp32 [S, 32, 2]    coefficients of positions start_pos .. start_pos+S-1
 *   c_kv    bf16 latent cache: element (b, t, c) at c_kv[b*ckv_bstride + t*ckv_rstride + c]
 *   k_pe    bf16 rotary cache: element (b, t, r) at k_pe[b*kpe_bstride + t*kpe_rstride + r]
 *           (fused [B, T, 576] rows: k_pe = c_kv + 512, both rstrides 576)
 *   T       cache capacity; requires 0 <= start_pos, start_pos + S <= T
 *   ws      device workspace of at least mla_cache_write_workspace_bytes(B*S)
 *           bytes, 256-byte aligned; contents need not be initialised
 * Requires 1 <= B*S <= 4096.
 * Two kernels are enqueued on `stream`: a split-K GEMM, then the finalize
 * kernel under programmatic dependent launch (it waits for the GEMM before
 * reading its partials).  For the caller nothing changes: work enqueued
 * after the call starts when the finalize kernel has finished.
 */
size_t mla_cache_write_workspace_bytes(int rows);
int mla_cache_write(const mla_bf16_t* x, const mla_bf16_t* w_kva, const mla_bf16_t* norm_w,
                    float eps, const float* rope, int B, int S, int start_pos,
                    mla_bf16_t* c_kv, int64_t ckv_bstride, int ckv_rstride,
                    mla_bf16_t* k_pe, int64_t kpe_bstride, int kpe_rstride, int T,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * The cache write above without a workspace argument, for callers that
 * cannot allocate device memory when they call it: code running inside
 * callbacks of graph-based or embedding runtimes, decode loops whose runtime
 * forbids allocation after start-up, and hosts whose device memory belongs to
 * another allocator.  The pages describe no such variant; it exists only for
 * those callers.
 *
 * The split-K partial products go to one fixed device array inside this
 * library (MLA_NOALLOC_MAX_ROWS rows of partials, 4,128,768 bytes), which every
 * GPU that loads the library holds until the process exits.  Arguments,
 * layouts and results are those of mla_cache_write; B*S above
 * MLA_NOALLOC_MAX_ROWS returns MLA_ERR_SHAPE without touching the GPU.  The
 * function allocates nothing.
 *
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  The address belongs to the device's context: a call made after
 * the context was replaced (cudaDeviceReset and a new context) looks it up
 * again.  All calls share the array and it keeps the last call's contents;
 * every value a call reads from it is written earlier in the same call, so
 * nothing needs clearing, but calls that can overlap on the GPU (different
 * streams, or different host threads) race on it and must be serialised by
 * the caller.
 */
#define MLA_NOALLOC_MAX_ROWS 64
int mla_cache_write_noalloc(const mla_bf16_t* x, const mla_bf16_t* w_kva,
                            const mla_bf16_t* norm_w, float eps, const float* rope, int B, int S,
                            int start_pos, mla_bf16_t* c_kv, int64_t ckv_bstride,
                            int ckv_rstride, mla_bf16_t* k_pe, int64_t kpe_bstride,
                            int kpe_rstride, int T, void* stream);

/*
 * Absorbed sparse decode, one query per batch row ("Mix and project" page,
 * decode ("MQA decode") code excerpt):
 *   q~[b,h,:]  = q_nope[b,h,:] W_UK[h]            W_UK[h] = wkv_b[h, 0:128, :]
 *   s[b,h,t]   = (q~[b,h,:].c_KV[b,t,:] + q_pe[b,h,:].k_pe[b,t,:]) * scale
 *                for t in the selected set of row b
 *   A          = softmax_t(s)
 *   O~[b,h,:]  = sum_t A[b,h,t] c_KV[b,t,:]
 *   O[b,h,:]   = W_UV[h] O~[b,h,:]                W_UV[h] = wkv_b[h, 128:256, :]
 * The selected keys of row b are the entries of topk[b, :] inside
 * [0, min(end_pos[b], T)); -1 entries are padding.  Other entries are
 * ignored and counted in status[1].  A row with no valid entry gets O = 0.
 * The pages' index mask is a set (a position listed twice is selected once);
 * this call does not look for repeats: each valid entry is one key, so a
 * position listed twice counts twice.  Callers pass distinct positions (an
 * indexer's top-k does), and then the two agree.
 *   q_nope  bf16 [B, 128, 128]
 *   q_pe    bf16 [B, 128, 64]   (already rotated)
 *   wkv_b   bf16 [128, 256, 512] ([out, in] storage of the 512 -> 128*256 projection)
 *   c_kv, k_pe, strides, T: cache as in mla_cache_write (read only)
 *   topk    int32 [B, k]   positions, in any order; distinct (see above)
 *   end_pos int32 [B]
 *   scale   softmax scale (192^-0.5 * mscale^2 in the model)
 *   O       bf16 [B, 128, 128]
 *   ws      device workspace of at least mla_decode_workspace_bytes(B, k) bytes,
 *           256-byte aligned; contents need not be initialised
 *   status  optional int32[2] (see top of file), may be NULL
 * Requires 1 <= B <= 65535 and 1 <= k <= 65536.
 *
 * Arithmetic: the scores are accumulated in fp32 by the tensor cores (each CTA
 * of a pair over half of the 576 columns; the two fp32 partial sums are added
 * in fp32), then scaled, masked, maximised, shifted by the running maximum
 * and exponentiated in fp32; row sums, the output accumulator and the
 * rescaling are fp32.  Rounded to bf16, as tensor-core operands: q~ (the
 * fold's output), the softmax weights P = 2^(s - m) (at most 2^8: the running
 * maximum is raised once a tile's maximum exceeds it by more than 8 log2
 * units), and the per-split partial outputs that the merge reads.  O is
 * rounded to bf16 once, at the end.
 *
 * Work split: the flattened list of (row, 64-key tile) is cut into equal
 * contiguous ranges, one per SM pair; a row cut between two ranges is merged
 * from their partial results by log-sum-exp.  The ranges depend on the
 * number of SM pairs the device runs the kernel on, so on devices with
 * different SM counts the split rows (and the last bits of their outputs)
 * may differ; on one device the result is the same on every call.
 *
 * The call enqueues three or four kernels on `stream`.  The first waits for
 * the stream's earlier work as usual.  The later ones use programmatic
 * dependent launch: each may start its set-up while its predecessor drains,
 * and reads that predecessor's results only once it has finished.  For the
 * caller nothing changes: work enqueued after the call starts when the call's
 * last kernel has finished, and the inputs must not be modified before then.
 */
size_t mla_decode_workspace_bytes(int B, int k);
int mla_decode(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
               const mla_bf16_t* c_kv, int64_t ckv_bstride, int ckv_rstride,
               const mla_bf16_t* k_pe, int64_t kpe_bstride, int kpe_rstride, int T,
               const int32_t* topk, int k, const int32_t* end_pos, int B, float scale,
               mla_bf16_t* O, void* ws, size_t ws_bytes, int32_t* status, void* stream);

/*
 * Several query rows per cache batch row: query row r (0 <= r < B) reads
 * cache batch row r / queries_per_row, with its own q_nope[r], q_pe[r],
 * topk[r, :] and end_pos[r]; everything else is mla_decode's definition
 * (mla_decode is the case queries_per_row = 1).  Two uses:
 *
 *   multi-query decode: S new tokens of one sequence scored in one step
 *   (speculative or multi-token-prediction tokens); row b * S + s holds token
 *   s of sequence b, end_pos[b * S + s] its causal limit.
 *
 *   sparse prefill ("Mix and project" page, the MHA prefill branch of the
 *   forward excerpt, with the index mask added to the causal mask): a prompt
 *   of S tokens of sequence b, cached at positions 0 .. S-1, gives rows
 *   b * S + s with end_pos = s + 1.  The prefill branch expands per-head keys
 *   k = [c_KV W_UK[h] ; k_pe] and values c_KV W_UV[h] and scores every prompt
 *   position under the mask; folding W_UK into the query and W_UV after the
 *   mix gives the same result in exact arithmetic ("Key heads" page), and
 *   only the selected positions are read.  Entries past the causal limit are
 *   excluded as the mask excludes them (and counted in status[1] like any
 *   entry outside [0, end_pos)); pass -1 for them to keep the count clean.
 *
 *   q_nope, q_pe, topk, end_pos, O: B query rows, layouts as mla_decode
 *   c_kv, k_pe, strides, T: B / queries_per_row cache batch rows
 *   ws: mla_decode_workspace_bytes(B, k) bytes
 *
 * Ragged lists: the lists of prefill tokens and new tokens end in -1 padding
 * of different lengths.  Two small kernels run first: one counts, per query
 * row, the 64-entry tiles up to the last one that holds an entry other than
 * -1 (at least one), and one prefix-sums the counts and cuts the work into
 * ranges that balance the tiles plus a fixed cost per row; the tiles after a
 * row's last listed entry are not run.  The split points therefore differ
 * from mla_decode's, and with one query per row the two calls agree within
 * rounding, not bit for bit.
 * Requires queries_per_row >= 1 dividing B, and every cache row in use
 * addressable as a 32-bit row index: (B / queries_per_row - 1) *
 * (ckv_bstride / ckv_rstride) + T <= 2^31 - 1 (else MLA_ERR_SHAPE).
 */
int mla_decode_mq(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
                  const mla_bf16_t* c_kv, int64_t ckv_bstride, int ckv_rstride,
                  const mla_bf16_t* k_pe, int64_t kpe_bstride, int kpe_rstride, int T,
                  const int32_t* topk, int k, const int32_t* end_pos, int B, int queries_per_row,
                  float scale, mla_bf16_t* O, void* ws, size_t ws_bytes, int32_t* status,
                  void* stream);

/*
 * The same call split into its three phases, for timing one of them alone:
 *   phase 1: fold of W_UK into the queries (writes q~ into ws)
 *   phase 2: gather + scores + softmax + latent mix (reads q~; writes the
 *            mixed latent O~ of each row held by one cluster, and the
 *            partial O~ and log-sum-exp of each segment of a split row, into ws)
 *   phase 3: log-sum-exp merge of the split rows (one launch, skipped when no
 *            row is split), then O = O~ W_UV^T (reads ws, writes O)
 *   phase 0: all three (identical to mla_decode)
 * Phases must run in order on one stream with the same arguments and
 * workspace; each phase alone leaves O undefined until phase 3 has run.
 */
int mla_decode_phase(int phase, const mla_bf16_t* q_nope, const mla_bf16_t* q_pe,
                     const mla_bf16_t* wkv_b, const mla_bf16_t* c_kv, int64_t ckv_bstride,
                     int ckv_rstride, const mla_bf16_t* k_pe, int64_t kpe_bstride,
                     int kpe_rstride, int T, const int32_t* topk, int k, const int32_t* end_pos,
                     int B, float scale, mla_bf16_t* O, void* ws, size_t ws_bytes,
                     int32_t* status, void* stream);

/*
 * Fold of W_UK into the queries, the first step of mla_decode ("Mix and
 * project" page, decode branch: einsum bshd,hdc->bshc):
 *   q_tilde[b,h,c] = sum_d q_nope[b,h,d] wkv_b[h,d,c]     bf16 [B, 128, 512]
 * fp32 accumulation, one rounding to bf16.  Requires 1 <= B <= 65535.
 */
int mla_fold_wuk(const mla_bf16_t* q_nope, const mla_bf16_t* wkv_b, int B,
                 mla_bf16_t* q_tilde, void* stream);

/*
 * Test hook: the decode index mask ("Mix and project" page, decode branch:
 * a -inf row over [0, end_pos) with the indexer's positions scattered to 0).
 *   mask uint8 [B, T]: 1 where t is listed in topk[b] and t < end_pos[b], else 0.
 * Invalid entries are counted in status[1] (status may be NULL).
 */
int mla_index_mask(const int32_t* topk, int B, int k, const int32_t* end_pos, int T,
                   uint8_t* mask, int32_t* status, void* stream);

/*
 * Test hook: the row gather of mla_decode.  rows[b, j, :] = the 576 cached
 * values (latent then rotary key) of position topk[b, j], or zeros when the
 * entry is -1 or invalid (invalid ones are counted in status[1]).
 *   rows bf16 [B, k, 576]
 */
int mla_gather_rows(const mla_bf16_t* c_kv, int64_t ckv_bstride, int ckv_rstride,
                    const mla_bf16_t* k_pe, int64_t kpe_bstride, int kpe_rstride, int T,
                    const int32_t* topk, int B, int k, const int32_t* end_pos,
                    mla_bf16_t* rows, int32_t* status, void* stream);

/*
 * Test hook: the expiry path of the bounded waits.  Every wait in the
 * library's kernels (mbarrier phases, the MMA issuer's event loop) gives up
 * after 1 s, sets MLA_STATUS_TIMEOUT in status[0] and lets its kernel wind
 * down, so that a lost arrival ends as an error the host can read instead of
 * a hung GPU.  This call launches one block of two warps that wait, through
 * the same code, on an mbarrier that nothing arrives on; it returns after the
 * limit with status[0] |= MLA_STATUS_TIMEOUT and gave_up[0] += 2 (one per
 * warp).  The GPU context stays usable.
 *   status  int32[2] device (status[1] untouched); gave_up int32[1] device
 */
int mla_wait_limit_check(int32_t* status, int32_t* gave_up, void* stream);

/* The most ranges (SM pairs) that share one row in mla_decode's work split
 * for (B, k) on the current device (1: no row is split). */
int mla_decode_num_splits(int B, int k);

/*
 * Output projection of the attention block ("Mix and project" page: the
 * output projection wo, the only step that mixes heads, 16,384 x 7,168
 * weights; the decode excerpt applies it as wo(x.flatten(2))):
 *   Delta[b, n] = sum over h, d of O[b, h, d] W_O[n, h * 128 + d]
 *     O      bf16 [B, 128, 128]   (the mla_decode output; flattened head-major)
 *     w_o    bf16 [7168, 16384]   ([out, in] storage)
 *     delta  bf16 [B, 7168]
 * fp32 accumulation.  A row tile of W_O whose K range is split between CTAs
 * is summed from fp32 partials in a fixed order, so the result is the same
 * on every run.  Requires 1 <= B <= 65535 and a caller-owned device
 * workspace of at least mla_out_proj_workspace_bytes(B) bytes, 256-byte
 * aligned (MLA_ERR_WORKSPACE otherwise).  status may be NULL (see above).
 * Two kernels are enqueued; the second uses programmatic dependent launch
 * (as described for mla_decode), with the same stream semantics for the
 * caller.
 */
size_t mla_out_proj_workspace_bytes(int B);
int mla_out_proj(const mla_bf16_t* O, const mla_bf16_t* w_o, int B, mla_bf16_t* delta, void* ws,
                 size_t ws_bytes, int32_t* status, void* stream);

/*
 * Query path ("Query rotary up-projection" page: the MLA init and forward
 * excerpts; W_QR is output features 128-191 of each head's 192 in wq_b):
 *   qr[b, :]   = RMSNorm(x[b] wq_a^T) * q_norm_w   (fp32 norm, qr rounded to bf16)
 *   q[b, h, :] = (qr[b] wq_b^T)[192 h .. 192 h + 191]
 *   q_nope[b, h, :] = q[b, h, 0:128]
 *   q_pe[b, h, :]   = interleaved rotation of q[b, h, 128:192] by rope[pos[b]]
 *     x        bf16 [B, 7168]
 *     wq_a     bf16 [1536, 7168]       ([out, in])
 *     q_norm_w bf16 [1536], eps >= 0   (RMSNorm y = x / sqrt(mean(x^2) + eps) * w)
 *     wq_b     bf16 [24576, 1536]      ([out, in], 128 heads x (128 + 64))
 *     rope     fp32 [T, 32, 2]         ((cos, sin) per position and pair)
 *     pos      int32 [B]               (the query position of each row)
 *     q_nope   bf16 [B, 128, 128], q_pe bf16 [B, 128, 64]: the mla_decode inputs
 * A row whose pos is outside [0, T) gets q_pe = 0 and is counted in
 * status[1].  Partials are summed in a fixed order (results identical on
 * every run).  Requires 1 <= B <= 65535 and a device workspace of at least
 * mla_query_proj_workspace_bytes(B) bytes, 256-byte aligned.  Four kernels
 * are enqueued; the last three use programmatic dependent launch (as
 * described for mla_decode), with the same stream semantics for the caller.
 */
size_t mla_query_proj_workspace_bytes(int B);
int mla_query_proj(const mla_bf16_t* x, const mla_bf16_t* wq_a, const mla_bf16_t* q_norm_w,
                   float eps, const mla_bf16_t* wq_b, const float* rope, int T,
                   const int32_t* pos, int B, mla_bf16_t* q_nope, mla_bf16_t* q_pe, void* ws,
                   size_t ws_bytes, int32_t* status, void* stream);

/*
 * Paged latent cache.  A pool holds num_pages pages of page_size rows; a row
 * holds the 576 cached values of one position ("KV compression" page), in
 * one of two kinds:
 *   MLA_PAGE_BF16   576 bf16 values (1152 bytes), as in the contiguous cache
 *   MLA_PAGE_E4M3   656 bytes: 512 latent codes (e4m3: sign, 4 exponent and 3
 *                   mantissa bits), 4 fp32 scales, 64 bf16 rotary values.  Scale g
 *                   belongs to latent values 128g .. 128g+127; a value is
 *                   code * scale.
 * The pages described on the method's pages are contiguous bf16 only.  The 656
 * bytes are laid out as in the 8-bit rows that public serving code for latent
 * attention stores; its scales are commonly max / 448, this library's powers of
 * two.
 *   pool         16-byte aligned; page p, row o at pool + p*page_stride + o*row_stride
 *   page_stride, row_stride   bytes, multiples of 16; row_stride >= 1152 / 656;
 *                page_stride a multiple of row_stride holding page_size rows;
 *                fewer than 2^31 - 256 rows in all
 *   slot         p * page_size + o
 * No alignment of page_size is required; 16 or more, a multiple of 16, is
 * fastest for mla_attend_paged on bf16 pages.
 *
 * mla_page_write stores rows into slots (MLA_PAGE_E4M3 quantises them as they
 * are written):
 *   rows   bf16, row i at rows + i*rstride (rstride in elements, a multiple of 8, >= 576)
 *   slots  int32 [N]; -1 skips the row, any other slot outside the pool is
 *          skipped and counted in status[1].  Slots are distinct: of a slot
 *          listed twice, each 16-byte piece holds one of the two rows'.  Rows
 *          may themselves lie in the pool (a page copied to another), but not
 *          in a slot that the call writes.
 * The scale of a group is the least power of two 2^n, -117 <= n <= 119, with
 * max |x| <= 448 * 2^n over the group; a code is x / scale (exact) rounded to
 * nearest even, saturated at 448.  A group with an infinity or NaN gets the
 * scale NaN and codes 0: all its values read as NaN.  A power of two makes code
 * * scale exact in bf16, so the rounding to a code is the only one.  N >= 0.
 * Rows written by other means may hold any fp32 scale: wherever rows are read, a
 * value is then code * scale in fp32, rounded once more, to bf16.  They hold no
 * NaN codes (0x7f, 0xff): under a power-of-two scale these read as numbers.
 *
 * mla_page_read returns the rows of slots as bf16 [N] rows (code * scale, exactly
 * for rows of mla_page_write); slot -1, and any other slot outside the pool
 * (counted in status[1]), gives a row of zeros.  The rows written share no memory
 * with the slots read.
 *
 * Both enqueue one kernel and use no workspace.
 */
int mla_page_write(const mla_bf16_t* rows, int64_t rstride, const int32_t* slots, int N,
                   void* pool, int kind, int num_pages, int page_size, int64_t page_stride,
                   int row_stride, int32_t* status, void* stream);
int mla_page_read(const void* pool, int kind, int num_pages, int page_size, int64_t page_stride,
                  int row_stride, const int32_t* slots, int N, mla_bf16_t* rows, int64_t rstride,
                  int32_t* status, void* stream);

/*
 * Attention of the new tokens of S sequences over their paged cache, all
 * cached positions, causal among the new tokens ("Mix and project" page, both
 * branches of the forward excerpt without the index mask): one token a
 * sequence (decode), a few (drafted tokens to verify) or a chunk or the whole
 * of a prompt, mixed freely.  The new tokens' own rows are in the cache
 * already (mla_page_write).
 *   Sequence s has the tokens r = cu_q[s] .. cu_q[s+1]-1 and kv_len[s] cached
 *   positions; position t is row t % page_size of page
 *   page_table[s, t / page_size].  Its token number i sees the positions
 *   t < kv_len[s] - (cu_q[s+1] - cu_q[s]) + i + 1:
 *     s[h,t] = (q_nope[r,h] . W_UK[h] c_t + q_pe[r,h] . kpe_t) * scale
 *     O[r,h] = sum_t softmax_t(s)[h,t] W_UV[h] c_t
 *   A token that sees nothing gets O = 0.
 *   q_nope     bf16 [N, 128, 128], q_pe bf16 [N, 128, 64] (rotated), O bf16 [N, 128, 128]
 *   wkv_b      bf16 [128, 256, 512], as in mla_decode
 *   pool, kind, num_pages, page_size, strides: as above (read only)
 *   page_table int32 [S, max_pages]
 *   cu_q       int32 [S + 1], cu_q[0] = 0, not decreasing, cu_q[S] <= N: rows of O
 *              from cu_q[S] on (the padding of a captured call) are left as they are
 *   kv_len     int32 [S]; a length above max_kv or the table's reach is cut to it
 *   scale      softmax scale, > 0 (else MLA_ERR_SHAPE)
 *   max_kv     the host's bound on the lengths; sets the workspace's size and, in
 *              the expanded form, how many heads are worked on at a time: close
 *              to the lengths is faster (256 tokens over 1500 positions: 110 us
 *              with a bound of 1500 to 65,536, 596 us from 524,289 on)
 *   form       MLA_FORM_ABSORBED folds W_UK into the queries and applies W_UV
 *              after the mix (278,528 flop per token and position).
 *              MLA_FORM_EXPANDED computes every position's keys and values of
 *              the 128 heads once (33.6 Mflop a position) and attends to those
 *              (81,920 flop per token and position).  MLA_FORM_AUTO takes the
 *              expanded form from an average of 112 (max_kv <= 1024), 160
 *              (<= 4096) or 208 new tokens a sequence on, where S * max_kv, each
 *              length rounded up to 128, is at most 2^21 (its workspace then
 *              takes up to 11 GB) or the absorbed form is refused.  The forms
 *              agree within rounding.  One form serves the whole call: decode
 *              tokens and a prompt chunk are faster in a call each (63 tokens
 *              over 1000 to 7820 positions with a chunk of 512 over 6000: 743
 *              us in one, 592 in two).
 *   ws         at least mla_attend_paged_workspace_bytes(N, S, max_kv, kind,
 *              form) bytes, 256-byte aligned; contents need not be initialised
 *   O and ws   share no memory with each other and with the arguments that are
 *              read (else MLA_ERR_OVERLAP; the pool's rows, which may lie among
 *              other memory, are not looked at)
 *   status     optional int32[2].  An entry of page_table outside [0, num_pages)
 *              for a page below the length of a sequence with new tokens reads
 *              as a page of zeros and is counted once in status[1].
 * Cached values at positions below kv_len[s] are taken to be finite: a NaN
 * there makes the tokens that see it NaN, an infinity may, and both may do so to
 * earlier tokens of the same sequence in the call.  What the pages hold from
 * kv_len[s] on does not matter.
 * 1 <= N <= 65535, 1 <= S <= 65535, 1 <= max_kv <= 2^24; absorbed: N *
 * ceil(max_kv / 128) < 2^30; expanded: S * max_kv, each length rounded up to
 * 128, at most 2^26 (else MLA_ERR_SHAPE).  The expanded form's workspace holds
 * 1152 bytes for each of those positions and the keys and values of as many
 * heads as fit 4 GiB, at least 8 (4 KB a position) and at most 128 (64 KB),
 * and 20 MB of partial outputs (40 MB for max_kv above 2^17).
 * The absorbed form on 8-bit pages with three tokens a sequence or more on
 * average (N >= 3 S, N * max_kv >= 2^18) converts the positions to bf16 in the
 * workspace first, 1152 bytes each, where that is 4 GiB at most.
 *
 * Arithmetic: scores, softmax statistics and outputs accumulate in fp32; the
 * tensor cores' additions truncate, so an output's sum is moved to another one,
 * added to nearest, every 2^17 positions.
 * Rounded to bf16, as tensor-core operands: softmax weights; absorbed: q~, the
 * mixed latent and a split token's partial mixed latents; expanded: keys,
 * values and the partial outputs of work that is split between SMs.  On one
 * device a call gives the same bits every time.
 *
 * The kernels of a call are enqueued on `stream`, some under programmatic
 * dependent launch (as described for mla_decode, with the same stream
 * semantics for the caller).  The call can be captured into a graph; graphs
 * that may run at the same time need workspaces of their own.
 */
size_t mla_attend_paged_workspace_bytes(int N, int S, int max_kv, int kind, int form);
int mla_attend_paged(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
                     const void* pool, int kind, int num_pages, int page_size,
                     int64_t page_stride, int row_stride, const int32_t* page_table,
                     int max_pages, const int32_t* cu_q, const int32_t* kv_len, int S, int N,
                     int max_kv, float scale, int form, mla_bf16_t* O, void* ws, size_t ws_bytes,
                     int32_t* status, void* stream);

/*
 * Test hook (host only, no device call): the work split of the
 * weight-streaming GEMM behind mla_out_proj and mla_query_proj for a
 * [n_out, k_in] weight.  Row tile m (128 weight rows) and K chunk j (128
 * columns) form unit m * nch + j; CTA c of a batch block takes units
 * [c * tot / nc, (c + 1) * tot / nc).  Writes plan[0..3] = tot, nc, nch,
 * slots, and for every row tile m first_last[2m], first_last[2m + 1] = the
 * first and last CTA holding a unit of tile m (the partial of CTA c for tile
 * m goes to slot c - first); first_last may be NULL.  Requires
 * n_out % 128 == 0 and k_in % 128 == 0, both positive (else MLA_ERR_SHAPE).
 */
int mla_xwt_plan(int n_out, int k_in, int32_t* plan, int32_t* first_last);

#ifdef __cplusplus
}
#endif

#endif /* SHLA_H_ */
