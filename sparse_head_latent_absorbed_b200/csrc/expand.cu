#include "expand.h"
namespace shla { namespace expand {
size_t workspace_bytes(int N, int S, int max_kv) { return 256; }
int run(const mla_bf16_t* q_nope, const mla_bf16_t* q_pe, const mla_bf16_t* wkv_b,
        const paged::Pool& pool, const paged::Seqs& q, float scale, mla_bf16_t* O, uint8_t* ws,
        int32_t* status, cudaStream_t st) { return MLA_ERR_UNSUPPORTED; }
}}
