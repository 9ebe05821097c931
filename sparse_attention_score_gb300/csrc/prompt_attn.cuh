// prompt_attn.cuh -- parameter block of the packed prompt attention.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dsa_internal.cuh"

namespace dsa {

struct PromptAttnParams {
  const __nv_bfloat16 *q, *k, *v;  // [tokens][heads][dim] with strides in elements
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  const int32_t *cu_q, *cu_k;  // [B + 1] or NULL (one sequence)
  int B, Nq, Nk, Hq, Hk, Dk, Dv;
  float scale_log2;
  __nv_bfloat16* out;
  long long o_ts, o_hs;
  float* lse;  // [Nq][Hq] or NULL
  int* status;
};
// Bytes of a workspace that serves calls of any size, and those of it that this one uses
// (no partial results where there are items for every SM many times over, no sums of
// their own where there are few keys).
size_t prompt_attn_ws();
size_t prompt_attn_uses(int B, int Nq, int Nk, int Hq, int Hk, int Dv);
int launch_prompt_attn(const PromptAttnParams& p, void* ws, cudaStream_t s);

}  // namespace dsa
