// cache4.cu -- rows of a K/V cache held in 4 bits: written, and read back.
//
// The pool is [num_blocks][heads][block_size][row bytes]: the pages of the
// block table ("Day-0 Adaptation of Trillion-Parameter MoE Models on Domestic
// GPUs", section 3 (2)), inside a page one key head after the other, so that a
// head's positions of a page are one contiguous piece.  A row is the codes of
// K, those of V, the group scales of K, those of V (cache4.cuh).
//
// Quantisation of a group of 16 elements y = x / head scale:
//   s = E4M3(min(max |y| / 6, 448)),  code = the E2M1 value nearest to y / s.
// The nearest code is decided on |y| against (midpoint between two codes) * s,
// a product of at most 7 significant bits that fp32 holds exactly, so no
// division rounds an element over a midpoint; ties go to the even code.
//
// Both kernels take a group per thread: 32 bytes of bf16, 8 bytes of codes and
// one scale.  They are bound by those bytes; see the launchers for figures.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <string>

#include "cache4.cuh"
#include "device_common.cuh"
#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;

struct Geo {
  Cache4RowsParams a;
  int gk, groups;  // groups of 16 elements: of K, of K and V
  long long units;  // N * Hk * groups
};

// Row of the pool that token n's head h belongs to, -1 without one.
__device__ __forceinline__ long long token_row(const Cache4RowsParams& a, long long n, int h) {
  const int b = a.seq ? __ldg(&a.seq[n]) : (int)n;
  if (b < 0 || b >= a.lay.batch) return -1;
  const long long pos = a.pos ? __ldg(&a.pos[n]) : (long long)__ldg(&a.lay.seq_lens[b]) - 1;
  if (pos < 0) return -1;
  const long long slot = pos / a.lay.bs;
  if (slot >= a.lay.maxb) return -1;
  const int page = __ldg(&a.lay.bt[(long long)b * a.lay.maxb + slot]);
  if (page < 0 || page >= a.lay.nb) return -1;
  return ((long long)page * a.Hk + h) * a.lay.bs + (pos - slot * a.lay.bs);
}

struct Unit {
  long long n;
  int h, group, j;  // j: group of K or of V
  bool is_v;
};

__device__ __forceinline__ Unit unit_of(const Geo& g, long long u) {
  Unit x;
  long long row;
  if (u >> 32) {
    row = u / g.groups;
    x.n = row / g.a.Hk;
  } else {
    row = (uint32_t)u / (uint32_t)g.groups;
    x.n = (uint32_t)row / (uint32_t)g.a.Hk;
  }
  x.group = (int)(u - row * g.groups);
  x.h = (int)(row - x.n * g.a.Hk);
  x.is_v = x.group >= g.gk;
  x.j = x.is_v ? x.group - g.gk : x.group;
  return x;
}

// Byte offsets of a group's codes and scale within a row.
__device__ __forceinline__ int codes_at(const Geo& g, int group) { return 8 * group; }
__device__ __forceinline__ int scale_at(const Geo& g, int group) { return 8 * g.groups + group; }

// The 16 values of a group: code * group scale (exact in fp16 and so in fp32)
// * head scale, rounded once to bf16.
__device__ __forceinline__ void kept_values(uint2 codes, uint32_t s8, float hs, uint4 (&o)[2]) {
  const __half_raw sr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3);
  const float f = __half2float(__half(sr));
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = (i < 4 ? codes.x : codes.y) >> (8 * (i & 3));
    const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c & 0xffu), __NV_E2M1);
    const float2 v = __half22float2(__half2(hr));
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f * hs, v.y * f * hs);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  o[0] = make_uint4(w[0], w[1], w[2], w[3]);
  o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__global__ void __launch_bounds__(kThreads) k_cache4_write(const __grid_constant__ Geo g) {
  const Cache4RowsParams& a = g.a;
  grid_dependency_wait();
  launch_dependents();
  const long long step = (long long)gridDim.x * kThreads;
  for (long long u = (long long)blockIdx.x * kThreads + threadIdx.x; u < g.units; u += step) {
    const Unit x = unit_of(g, u);
    const __nv_bfloat16* src = x.is_v ? a.v + x.n * a.v_ts + x.h * a.v_hs : a.k + x.n * a.k_ts + x.h * a.k_hs;
    const uint4* p = reinterpret_cast<const uint4*>(src + 16 * x.j);
    const uint4 in[2] = {__ldg(p), __ldg(p + 1)};
    const float* hp = x.is_v ? a.v_scale : a.k_scale;
    const float hs = hp ? __ldg(&hp[x.h]) : 1.0f;
    const long long row = token_row(a, x.n, x.h);
    float y[16];
    const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = __uint_as_float(w[i] << 16);
      y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    if (hp) {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(y[i], hs);
    }
    // the largest magnitude by its bits, so that a NaN is the largest of all
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
    const uint32_t s8 = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(top), 6.0f), __NV_SATFINITE,
                                              __NV_E4M3);
    const __half_raw sr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3);
    const float t = __half2float(__half(sr));
    uint2 codes = make_uint2(0, 0);
    if (t > 0.0f) {  // none where the scale is 0 or NaN
      const float t0 = 0.25f * t, t1 = 0.75f * t, t2 = 1.25f * t, t3 = 1.75f * t, t4 = 2.5f * t,
                  t5 = 3.5f * t, t6 = 5.0f * t;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float m = fabsf(y[i]);
        uint32_t c = (m > t0) + (m >= t1) + (m > t2) + (m >= t3) + (m > t4) + (m >= t5) + (m > t6);
        c |= (__float_as_uint(y[i]) >> 28) & 8u;
        if (i < 8)
          codes.x |= c << (4 * i);
        else
          codes.y |= c << (4 * (i - 8));
      }
    }
    if (row >= 0) {
      uint8_t* dst = a.pool + row * a.row_bytes;
      *reinterpret_cast<uint2*>(dst + codes_at(g, x.group)) = codes;
      dst[scale_at(g, x.group)] = (uint8_t)s8;
      if (x.group == g.groups - 1)
        for (int i = 9 * g.groups; i < a.row_bytes; ++i) dst[i] = 0;
    } else if (x.group == 0) {
      flag_status(a.status, DSA_STATUS_BAD_BLOCK);
    }
    __nv_bfloat16* out = x.is_v ? a.v_out : a.k_out;
    if (out) {
      uint4 o[2];
      kept_values(codes, s8, hs, o);
      const int D = x.is_v ? a.Dv : a.Dk;
      uint4* q = reinterpret_cast<uint4*>(out + (x.n * a.Hk + x.h) * D + 16 * x.j);
      q[0] = o[0];
      q[1] = o[1];
    }
  }
}

__global__ void __launch_bounds__(kThreads) k_cache4_read(const __grid_constant__ Geo g) {
  const Cache4RowsParams& a = g.a;
  grid_dependency_wait();
  launch_dependents();
  const long long step = (long long)gridDim.x * kThreads;
  for (long long u = (long long)blockIdx.x * kThreads + threadIdx.x; u < g.units; u += step) {
    const Unit x = unit_of(g, u);
    const float* hp = x.is_v ? a.v_scale : a.k_scale;
    const float hs = hp ? __ldg(&hp[x.h]) : 1.0f;
    const long long row = token_row(a, x.n, x.h);
    uint4 o[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (row >= 0) {
      const uint8_t* src = a.pool + row * a.row_bytes;
      kept_values(__ldg(reinterpret_cast<const uint2*>(src + codes_at(g, x.group))),
                  __ldg(src + scale_at(g, x.group)), hs, o);
    } else if (x.group == 0) {
      flag_status(a.status, DSA_STATUS_BAD_BLOCK);
    }
    __nv_bfloat16* out = x.is_v ? a.v_out : a.k_out;
    const int D = x.is_v ? a.Dv : a.Dk;
    uint4* q = reinterpret_cast<uint4*>(out + (x.n * a.Hk + x.h) * D + 16 * x.j);
    q[0] = o[0];
    q[1] = o[1];
  }
}

}  // namespace

int launch_cache4_rows(const Cache4RowsParams& p, bool write, cudaStream_t s) {
  Geo g{};
  g.a = p;
  g.gk = p.Dk / 16;
  g.groups = (p.Dk + p.Dv) / 16;
  g.units = (long long)p.N * p.Hk * g.groups;
  if (g.units == 0) return DSA_OK;
  const long long blocks = (g.units + kThreads - 1) / kThreads;
  const long long most = 16LL * sm_count();
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  const cudaError_t e = launch_pdl(write ? k_cache4_write : k_cache4_read, dim3(grid), dim3(kThreads), 0, s, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch(write ? "cache4_write" : "cache4_read");
}

}  // namespace dsa
