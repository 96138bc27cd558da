// The expanded form of the attention over a paged cache (expand.cu).
#pragma once

#include "attend_paged.cuh"

namespace shla {
namespace expand {

// Average new tokens per sequence from which MLA_FORM_AUTO expands.  By flops
// alone the forms meet at 33.6e6 / (278,528 - 81,920) = 171 tokens.  Measured, in
// microseconds absorbed / expanded: 32 sequences of 300 positions, 64 new tokens
// each 602 / 638, 96 862 / 638; 8 of 1000, 96 tokens 389 / 447, 128 487 / 421; one
// of 2000, 128 tokens 107 / 128, 160 129 / 128; one of 6000, 160 tokens 248 / 304,
// 256 367 / 306; one of 40000, 160 tokens 1440 / 1971, 256 2215 / 1924.
inline int min_tokens(int max_kv) { return max_kv <= 1024 ? 112 : max_kv <= 4096 ? 160 : 208; }

// Positions of all sequences, each rounded up to 128, that a call may reach.
constexpr int64_t kMaxRows = 1 << 26;
// ... and may reach for MLA_FORM_AUTO to expand: a workspace of 11 GB, 6% of the
// GPU's memory (16 sequences of 131,072 positions, 512 new tokens each: 140 ms
// against 318 absorbed).  It grows by 5.2 KB a position: 176 GB for 256 sequences
// under that bound, however short they are, which the absorbed form serves from 17.
constexpr int64_t kAutoRows = 1 << 21;
bool fits(int S, int max_kv, int64_t rows = kMaxRows);

size_t workspace_bytes(int N, int S, int max_kv);

// The rows of a call's sequences as bf16, one sequence after another in pages of
// 64: a pool and table that the absorbed form reads instead of 8-bit pages.
size_t staged_bytes(int N, int S, int max_kv);
int stage(const paged::Pool& pool, const paged::Seqs& q, uint8_t* ws, int32_t* status,
          cudaStream_t st, paged::Pool* staged);

int run(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
        const paged::Pool& pool, const paged::Seqs& q, float scale, mla_bf16_t* O, uint8_t* ws,
        int32_t* status, cudaStream_t st);

}  // namespace expand
}  // namespace shla
