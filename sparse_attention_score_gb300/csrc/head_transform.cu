// head_transform.cu -- per-head norm and position rotation of new tokens'
// queries and cache rows, written to strided tensors or, through the block
// table, to the paged pools.
//
// A layer's projections hand over raw heads; the indexer and the attention
// ("Day-0 Adaptation of Trillion-Parameter MoE Models on Domestic GPUs",
// section 3) read normed, rotated ones, and the KV cache is written in the
// block layout the gather reads ("Day-0 Adaptation of Ultra-Large-Scale MoE
// Models on Heterogeneous AI Accelerators", section 4).  For one head
// x[0..dim):
//   norm    RMS:   y = x / sqrt(mean(x^2) + eps) * w
//           layer: y = (x - mean) / sqrt(mean((x - mean)^2) + eps) * w + b
//           over the first norm_dim elements (the rest pass through);
//   rotate  the pairs (a, b) of [rope_offset, rope_offset + rope_dim):
//           (a cos t - b sin t, b cos t + a sin t), t = pos * inv_freq[i];
//   store   one rounding, to bf16 or to saturating E4M3.
//
// Angles: t / 2 pi is wanted modulo 1 only, and far positions have t in the
// millions, where an fp32 product is off by whole turns' fractions.  A
// frequency is turned once into a 64-bit fixed-point fraction of a turn (one
// fp64 product, rounded to 2^-64 turns), and pos times that, modulo 2^64, is
// an integer product that wraps where the angle does: for inv_freq <= 1 the
// error is below pos * 2^-54 turns.  Its upper 32 bits go through sincospif.
#include <cuda_runtime.h>

#include <string>

#include "device_common.cuh"
#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxJobs = 2 * DSA_MAX_HEAD_PARTS;
constexpr int kMaxDim = 1024;

struct HeadJob {
  const __nv_bfloat16* in;
  long long in_ts, in_hs;  // elements between tokens / heads
  void* out;
  long long out_ts, out_hs;  // out_ts: between tokens, or between pool rows
  const float* weight;
  const float* bias;
  const float* inv_freq;
  float eps;
  int heads, dim, norm, norm_dim, rope_off, rope_dim;
  int interleaved, fp8, paged;
  int groups;    // head groups per token
  int group;     // heads per group
  int first;     // first item of this job
};

struct HeadParams {
  LayoutDev lay;
  const int32_t* seq;
  const int32_t* pos;  // NULL: append form, position seq_lens[i] - 1 of sequence i
  int N;
  int n_jobs, items;
  int cs_len;     // cos/sin pairs per warp
  int stage_len;  // staged floats per warp
  int* status;
  HeadJob job[kMaxJobs];
};

// Fraction of a turn per position, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  double t = (double)f * 0.15915494309189533577;  // f / 2 pi
  t -= rint(t);  // in [-1/2, 1/2]
  return (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
}

// (cos, sin) of pos * f.
__device__ __forceinline__ float2 rotation(float f, int pos) {
  const unsigned long long u = turns_of(f) * (unsigned long long)(long long)pos;
  const float x = (float)(int)(u >> 32) * 4.6566128730773926e-10f;  // half turns in [-1, 1)
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c, s);
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void store8(const HeadJob& j, long long off, const float (&v)[8]) {
  if (j.fp8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(j.out) + off) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(j.out) + off) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The heads [h0, h1) of one token: L lanes per head, granules of 8 elements,
// J granules per lane.
template <int L, int J>
__device__ void transform(const HeadJob& j, long long tok, int h0, int h1, long long out_base,
                          const float2* cs, float* stage) {
  const int lane = threadIdx.x & 31;
  const int sub = lane / L, li = lane % L;
  constexpr int kRows = 32 / L;
  const int G = j.dim >> 3;
  const int half = j.rope_dim >> 1;
  for (int h = h0; h < h1; h += kRows) {
    const int hh = h + sub;
    const bool live = hh < h1;
    float v[J][8];
#pragma unroll
    for (int k = 0; k < J; ++k) {
      const int g = li + L * k;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (live && g < G)
        raw = *reinterpret_cast<const uint4*>(j.in + tok * j.in_ts + hh * j.in_hs + 8 * g);
      unpack8(raw, v[k]);
    }
    if (j.norm != DSA_NORM_NONE) {
      float mean = 0.0f;
      if (j.norm == DSA_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < J; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (8 * (li + L * k) + i < j.norm_dim) s += v[k][i];
        mean = row_sum<L>(s) / (float)j.norm_dim;
      }
      float q = 0.0f;
#pragma unroll
      for (int k = 0; k < J; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * (li + L * k) + i < j.norm_dim) {
            v[k][i] -= mean;
            q = fmaf(v[k][i], v[k][i], q);
          }
      const float r = 1.0f / sqrtf(row_sum<L>(q) / (float)j.norm_dim + j.eps);
#pragma unroll
      for (int k = 0; k < J; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = 8 * (li + L * k) + i;
          if (e < j.norm_dim) {
            float y = v[k][i] * r;
            if (j.weight) y *= __ldg(&j.weight[e]);
            if (j.bias) y += __ldg(&j.bias[e]);
            v[k][i] = y;
          }
        }
    }
    if (j.rope_dim) {
      if (j.interleaved) {
#pragma unroll
        for (int k = 0; k < J; ++k)
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const int e = 8 * (li + L * k) + i - j.rope_off;
            if (e >= 0 && e < j.rope_dim) {
              const float2 c = cs[e >> 1];
              const float a = v[k][i], b = v[k][i + 1];
              v[k][i] = a * c.x - b * c.y;
              v[k][i + 1] = b * c.x + a * c.y;
            }
          }
      } else {
        float* st = stage + sub * j.rope_dim;
#pragma unroll
        for (int k = 0; k < J; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = 8 * (li + L * k) + i - j.rope_off;
            if (e >= 0 && e < j.rope_dim) st[e] = v[k][i];
          }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < J; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = 8 * (li + L * k) + i - j.rope_off;
            if (e >= 0 && e < j.rope_dim) {
              const bool first = e < half;
              const float2 c = cs[first ? e : e - half];
              const float p = st[first ? e + half : e - half];
              v[k][i] = first ? v[k][i] * c.x - p * c.y : v[k][i] * c.x + p * c.y;
            }
          }
        __syncwarp();
      }
    }
    if (live && out_base >= 0) {
#pragma unroll
      for (int k = 0; k < J; ++k) {
        const int g = li + L * k;
        if (g < G) store8(j, out_base + hh * j.out_hs + 8 * g, v[k]);
      }
    }
  }
}

__global__ void __launch_bounds__(kWarps * 32) k_head_transform(const __grid_constant__ HeadParams p) {
  extern __shared__ float4 smraw[];
  grid_dependency_wait();
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* base = reinterpret_cast<float*>(smraw) + (size_t)warp * (2 * p.cs_len + p.stage_len);
  float2* cs = reinterpret_cast<float2*>(base);
  float* stage = base + 2 * p.cs_len;
  for (long long item = (long long)blockIdx.x * kWarps + warp; item < p.items;
       item += (long long)gridDim.x * kWarps) {
    int n = 0;
    while (n + 1 < p.n_jobs && item >= p.job[n + 1].first) ++n;
    const HeadJob& j = p.job[n];
    const int at = (int)item - j.first;
    const int t = at / j.groups, grp = at - t * j.groups;
    const int h0 = grp * j.group, h1 = min(j.heads, h0 + j.group);
    // position of the token, and the pool row of a paged destination
    const int b = p.seq ? __ldg(&p.seq[t]) : t;
    int pos = 0;
    if (p.pos)
      pos = __ldg(&p.pos[t]);
    else if (b < p.lay.batch)
      pos = __ldg(&p.lay.seq_lens[b]) - 1;
    long long out_base = t * j.out_ts;
    if (j.paged) {
      long long row = -1;
      if (b >= 0 && b < p.lay.batch && pos >= 0)
        row = phys_row(p.lay.bt, p.lay.maxb, p.lay.bs, p.lay.nb, b, pos);
      if (row < 0) {
        if (lane == 0) flag_status(p.status, DSA_STATUS_BAD_BLOCK);
        continue;
      }
      out_base = row * j.out_ts;
    }
    if (j.rope_dim) {
      __syncwarp();
      for (int i = lane; i < (j.rope_dim >> 1); i += 32) cs[i] = rotation(__ldg(&j.inv_freq[i]), pos);
      __syncwarp();
    }
    const int G = j.dim >> 3;
    if (G <= 8)
      transform<8, 1>(j, t, h0, h1, out_base, cs, stage);
    else if (G <= 16)
      transform<16, 1>(j, t, h0, h1, out_base, cs, stage);
    else if (G <= 32)
      transform<32, 1>(j, t, h0, h1, out_base, cs, stage);
    else if (G <= 96)
      transform<32, 3>(j, t, h0, h1, out_base, cs, stage);
    else
      transform<32, 4>(j, t, h0, h1, out_base, cs, stage);
  }
}

bool aligned(const void* q, unsigned a) { return ((uintptr_t)q & (a - 1)) == 0; }

bool stride_ok(int64_t v) { return v >= 0 && v <= (1LL << 31); }

int rows_per_warp(int dim) { return dim <= 64 ? 4 : dim <= 128 ? 2 : 1; }

int check_part(const dsa_head_part& a, int N, bool paged, HeadJob* j) {
  if (N > 0 && (!a.in || !a.out))  // empty tensors have no address
    return set_error(DSA_ERR_INVALID, "head part: NULL tensor pointer");
  if (a.heads < 1 || a.dim < 8 || a.dim % 8 || a.dim > kMaxDim)
    return set_error(DSA_ERR_UNSUPPORTED,
                     "head part: heads >= 1, dim a multiple of 8 in 8..1024");
  if (a.out_dtype != DSA_BF16 && a.out_dtype != DSA_FP8_E4M3)
    return set_error(DSA_ERR_UNSUPPORTED, "head part: out_dtype BF16 or FP8_E4M3");
  const bool fp8 = a.out_dtype == DSA_FP8_E4M3;
  if (!aligned(a.in, 16) || !aligned(a.out, fp8 ? 8 : 16))
    return set_error(DSA_ERR_INVALID,
                     "head part: in and a bf16 out must be 16-byte aligned, an FP8 out 8-byte");
  if (a.in_token_stride % 8 || a.in_head_stride % 8 || a.out_token_stride % 8 ||
      a.out_head_stride % 8 || !stride_ok(a.in_token_stride) || !stride_ok(a.in_head_stride) ||
      !stride_ok(a.out_token_stride) || !stride_ok(a.out_head_stride))
    return set_error(DSA_ERR_INVALID, "head part: strides must be multiples of 8 in 0..2^31");
  const long long span = (a.heads - 1) * a.out_head_stride + a.dim;
  const bool heads_apart = a.heads == 1 || a.out_head_stride >= a.dim;
  const bool token_major = heads_apart && a.out_token_stride >= span;
  const bool head_major = a.out_token_stride >= a.dim &&
                          a.out_head_stride >= (long long)(N - 1) * a.out_token_stride + a.dim;
  if (!(token_major || (!paged && (head_major || (N <= 1 && heads_apart)))))
    return set_error(DSA_ERR_INVALID, "head part: the out strides make heads overlap");
  if (a.norm != DSA_NORM_NONE && a.norm != DSA_NORM_RMS && a.norm != DSA_NORM_LAYER)
    return set_error(DSA_ERR_UNSUPPORTED, "head part: norm must be NONE, RMS or LAYER");
  if (a.norm != DSA_NORM_NONE &&
      (a.norm_dim < 1 || a.norm_dim > a.dim || !(a.eps >= 0.0f) || a.eps > 3.4e38f))
    return set_error(DSA_ERR_INVALID, "head part: norm_dim in 1..dim and a finite eps >= 0");
  if (a.norm != DSA_NORM_NONE && (!aligned(a.weight, 16) || !aligned(a.bias, 16)))
    return set_error(DSA_ERR_INVALID, "head part: weight and bias must be 16-byte aligned");
  if (a.rope_dim < 0 || a.rope_dim % 2 || a.rope_offset < 0 || a.rope_offset % 2 ||
      (long long)a.rope_offset + a.rope_dim > a.dim)
    return set_error(DSA_ERR_INVALID,
                     "head part: rope_offset and rope_dim even, inside the head");
  if (a.rope_dim && (!a.inv_freq || !aligned(a.inv_freq, 4)))
    return set_error(DSA_ERR_INVALID, "head part: rope_dim needs inv_freq");
  j->in = reinterpret_cast<const __nv_bfloat16*>(a.in);
  j->in_ts = a.in_token_stride;
  j->in_hs = a.in_head_stride;
  j->out = a.out;
  j->out_ts = a.out_token_stride;
  j->out_hs = a.out_head_stride;
  j->weight = a.weight;
  j->bias = a.bias;
  j->inv_freq = a.inv_freq;
  j->eps = a.eps;
  j->heads = a.heads;
  j->dim = a.dim;
  j->norm = a.norm;
  j->norm_dim = a.norm_dim;
  j->rope_off = a.rope_offset;
  j->rope_dim = a.rope_dim;
  j->interleaved = a.interleaved ? 1 : 0;
  j->fp8 = fp8;
  j->paged = paged;
  return DSA_OK;
}

}  // namespace

int head_transform(const LayoutDev* lay, const int32_t* seq, const int32_t* pos, int N,
                   const dsa_head_part* cache, int n_cache, const dsa_head_part* heads,
                   int n_heads, int* status, cudaStream_t s) {
  HeadParams p{};
  if (lay) p.lay = *lay;
  p.seq = seq;
  p.pos = pos;
  p.N = N;
  p.status = status;
  p.n_jobs = n_cache + n_heads;
  long long items = 0;
  for (int i = 0; i < p.n_jobs; ++i) {
    HeadJob& j = p.job[i];
    const bool paged = i < n_cache;
    const int rc = check_part(paged ? cache[i] : heads[i - n_cache], N, paged, &j);
    if (rc) return rc;
    const int rpw = rows_per_warp(j.dim);
    j.group = rpw;
    j.groups = (j.heads + j.group - 1) / j.group;
    j.first = (int)items;
    items += (long long)N * j.groups;
    if (items > 0x7fffffffLL)
      return set_error(DSA_ERR_UNSUPPORTED, "head parts: tokens x heads beyond 2^31 - 1");
    if (j.rope_dim / 2 > p.cs_len) p.cs_len = j.rope_dim / 2;
    if (!j.interleaved && rpw * j.rope_dim > p.stage_len) p.stage_len = rpw * j.rope_dim;
  }
  if (N == 0) return DSA_OK;
  p.items = (int)items;
  p.cs_len = (p.cs_len + 1) & ~1;
  p.stage_len = (p.stage_len + 3) & ~3;
  const size_t smem = sizeof(float) * kWarps * (2 * (size_t)p.cs_len + p.stage_len);
  long long grid = (items + kWarps - 1) / kWarps;
  const long long cap = 16LL * sm_count();
  if (grid > cap) grid = cap;
  const cudaError_t e =
      launch_pdl(k_head_transform, dim3((unsigned)grid), dim3(kWarps * 32), smem, s, p);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("head_transform");
}

}  // namespace dsa
