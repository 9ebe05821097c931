// cache4.cuh -- the 4-bit cache's row format and the parameter blocks of its
// calls.  A row holds one position of one key head:
//   Dk / 2 bytes  codes of K, two E2M1 codes a byte, the lower dim in the low half
//   Dv / 2        codes of V
//   Dk / 16       E4M3 scales of K, one per group of 16 dims
//   Dv / 16       E4M3 scales of V
//   zeros up to a multiple of 16 bytes
// so group j of the row's (Dk + Dv) / 16 has its codes at 8 j and its scale at
// (Dk + Dv) / 2 + j.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dsa_internal.cuh"

namespace dsa {

inline int cache4_row_bytes(int Dk, int Dv) { return ((Dk + Dv) / 16 * 9 + 15) / 16 * 16; }

// cache4_write and cache4_read
struct Cache4RowsParams {
  LayoutDev lay;
  const int32_t* seq;  // NULL with pos: token i is the newest position of sequence i
  const int32_t* pos;
  int N, Hk, Dk, Dv, row_bytes;
  const __nv_bfloat16 *k, *v;  // rows to write
  long long k_ts, k_hs, v_ts, v_hs;
  const float *k_scale, *v_scale;
  uint8_t* pool;
  __nv_bfloat16 *k_out, *v_out;  // [N][Hk][D]; of a write NULL or the values kept
  int* status;
};
int launch_cache4_rows(const Cache4RowsParams& p, bool write, cudaStream_t s);

// cache4_attn_decode
struct Cache4AttnParams {
  LayoutDev lay;
  const __nv_bfloat16* q;
  const uint8_t* pool;
  const float *k_scale, *v_scale;
  int Hq, Hk, Dk, Dv, row_bytes;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int* status;
};
size_t cache4_attn_ws(int B, int Hq, int Hk, int Dk, int Dv);
int launch_cache4_attn(const Cache4AttnParams& p, void* ws, cudaStream_t s);

}  // namespace dsa
