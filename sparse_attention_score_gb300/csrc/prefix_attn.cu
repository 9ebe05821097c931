// prefix_attn.cu -- exact decode attention over every cached position, for a
// batch that shares a prefix.
//
// One warp per (sequence, head): the positions one after the other through
// the block table, with a running maximum and sum of the softmax; lanes over
// the dims.
#include "device_common.cuh"
#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 576, kMaxV = 512;

__global__ void __launch_bounds__(kWarps * 32) k_prefix_attn(PrefixAttnParams p) {
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= p.lay.batch * p.Hq) return;
  const int b = r / p.Hq;
  long long L = __ldg(&p.lay.seq_lens[b]);
  const long long cap = (long long)p.lay.maxb * p.lay.bs;
  if (L > cap) {
    if (lane == 0) flag_status(p.status, DSA_STATUS_BAD_LENGTH);
    L = cap;
  }
  int src = b;  // block-table row the prefix is read through
  if (L >= p.prefix)
    for (src = 0; __ldg(&p.lay.seq_lens[src]) < p.prefix; ++src) {}
  float q[kMaxD / 32], o[kMaxV / 32];
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.Dqk ? __bfloat162float(p.q[(long long)r * p.Dqk + d]) * p.scale_log2 : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kMaxV / 32; ++i) o[i] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  for (long long pos = 0; pos < L; ++pos) {
    const long long row = phys_row(p.lay.bt, p.lay.maxb, p.lay.bs, p.lay.nb,
                                   pos < p.prefix ? src : b, pos);
    if (row < 0) {
      if (lane == 0) flag_status(p.status, DSA_STATUS_BAD_BLOCK);
      continue;
    }
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
      const int d = lane + 32 * i;
      if (d < p.Dqk) z = fmaf(q[i], __bfloat162float(p.kp[row * p.ks + d]), z);
    }
    z = warp_sum(z);
    const float mn = fmaxf(m, z);
    const float f = m > -INFINITY ? exp2f(m - mn) : 0.0f;
    const float w = mn > -INFINITY ? exp2f(z - mn) : 0.0f;
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kMaxV / 32; ++i) {
      const int d = lane + 32 * i;
      if (d < p.Dv) o[i] = fmaf(w, __bfloat162float(p.vp[row * p.vs + d]), o[i] * f);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxV / 32; ++i) {
    const int d = lane + 32 * i;
    if (d < p.Dv) p.out[(long long)r * p.Dv + d] = __float2bfloat16(o[i] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[r] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t prefix_attn_ws(int, int, int, int, int) { return kWsHeader; }

int launch_prefix_attn(const PrefixAttnParams& p, void*, cudaStream_t s) {
  const int rows = p.lay.batch * p.Hq;
  const cudaError_t e = launch_pdl(k_prefix_attn, dim3((unsigned)((rows + kWarps - 1) / kWarps)),
                                   dim3(kWarps * 32), 0, s, p);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("prefix_attn_decode");
}

}  // namespace dsa
