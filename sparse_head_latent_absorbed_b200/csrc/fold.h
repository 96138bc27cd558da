// The fold of W_UK into the queries (decode.cu), as the calls that begin with
// it launch it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace shla {

// q~ [B][128][512] from q_nope [B][128][128]: one kernel, an ordinary launch; its
// bounded waits report in `status`.
int launch_fold(const __nv_bfloat16* q_nope, const __nv_bfloat16* wkv_b, __nv_bfloat16* q_tilde,
                int B, int32_t* status, cudaStream_t st);

}  // namespace shla
