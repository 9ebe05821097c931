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
// y is x / head scale rounded to fp32, and the nearest code is that of y / s itself,
// ties to the even one: y / s is divided in fp32, correctly rounded, and a quotient
// that arrives at a midpoint between two codes goes to the side that its exact
// remainder says.
//
// Both kernels take half a group per thread, so that a warp's accesses of 16 bytes
// of bf16 and of 4 bytes of codes lie side by side (with a group per thread the
// two accesses of 16 bytes, or one of 32, took 1.3 times as long).  A thread keeps
// its place in a token's row (key head, group) and goes from token to token, so that
// no division is left in the loop, the tokens' places in the pool having been looked
// up once per block.
//
// Measured: 32,768 tokens of 8 heads of 128 / 128 read in 35 us (172 MB, 72 % of the
// copy rate); 16,384 written, with head scales and the values back, in 48 us (153 MB,
// 47 %): an element costs ~9 instructions, most for dividing it exactly twice, which
// keep 68 % of the issue slots and 54 % of the ALU (the fullest pipe) busy; most
// stalls are waits for a turn, for a fixed latency and for the pipe.  The bound of five
// blocks an SM spills 32 bytes a thread in both writing kernels.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "cache4.cuh"
#include "device_common.cuh"
#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 64;

struct Geo {
  Cache4RowsParams a;
  int gk, groups;  // groups of 16 elements of a row: of K, of K and V
  int units;       // half groups of a token: 2 * Hk * groups
  int tokens;      // tokens of a block at a time (0: one, its units in turn)
  int chunk;       // tokens of a block, at most kChunk
};

// A thread's place in a token: key head, group of the row, half of the group.
struct Place {
  int h, group, j, half;  // j: group of K or of V
  bool is_v;
  __device__ __forceinline__ Place(const Geo& g, int unit) {
    half = unit & 1;
    h = (unit >> 1) / g.groups;
    group = (unit >> 1) - h * g.groups;
    is_v = group >= g.gk;
    j = is_v ? group - g.gk : group;
  }
};

// Page of token n and its offset in it, -1 without one.
__device__ __forceinline__ int token_page(const Cache4RowsParams& a, int n, int* off) {
  const int b = a.seq ? __ldg(&a.seq[n]) : n;
  if (b < 0 || b >= a.lay.batch) return -1;
  const int pos = a.pos ? __ldg(&a.pos[n]) : __ldg(&a.lay.seq_lens[b]) - 1;
  if (pos < 0) return -1;
  const int slot = pos / a.lay.bs;
  if (slot >= a.lay.maxb) return -1;
  *off = pos - slot * a.lay.bs;
  const int page = __ldg(&a.lay.bt[(long long)b * a.lay.maxb + slot]);
  return page >= 0 && page < a.lay.nb ? page : -1;
}

// The eight values of half a group: code * group scale (exact in fp16 and so in
// fp32), which is rounded to bf16 once; times a head scale to fp32 first.
__device__ __forceinline__ uint4 kept_values(uint32_t codes, uint32_t s8, float hs) {
  const __half_raw sr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3);
  const __half2 f = __half2half2(__half(sr));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(codes >> (8 * i) & 0xffu), __NV_E2M1);
    const float2 v = __half22float2(__hmul2(__half2(hr), f));
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * hs, v.y * hs);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float scale_value(uint32_t s8) {
  const __half_raw sr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3);
  return __half2float(__half(sr));
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split2(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// x / d by a reciprocal r of d (neg: -d), correctly rounded for quotients well
// inside fp32's range: the rounded product, its exact remainder, and one correction
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).
__device__ __forceinline__ uint64_t quotients(uint64_t x, uint64_t neg, uint64_t r) {
  const uint64_t q = mul2(x, r);
  return fma2(fma2(q, neg, x), r, q);
}

// Half a group of bf16 elements (the other half is the neighbour lane's): the
// group's scale and the codes.
template <bool scaled>
__device__ __forceinline__ uint32_t quantise(uint4 in, float hs, uint32_t* codes) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  // the largest magnitude by its bits, so that a NaN is the largest of all
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] << 16 & 0x7fff0000u, w[i] & 0x7fff0000u));
  top = max(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
  float most = __uint_as_float(top);
  if (scaled) most = __fdiv_rn(most, hs);
  const uint32_t s8 = __nv_cvt_float_to_fp8(__fdiv_rn(most, 6.0f), __NV_SATFINITE, __NV_E4M3);
  const float s = scale_value(s8);
  *codes = 0;
  if (!(s > 0.0f)) return s8;  // codes 0 where the scale is 0 or NaN
  uint64_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = pair2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  // The short division holds for quotients inside fp32's range: what lies below
  // it has code 0 either way.
  if (most < 1e30f && hs > 1e-20f && hs < 1e20f) {
    if (scaled) {
      const float rh = __frcp_rn(hs);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = quotients(y[i], pair2(-hs, -hs), pair2(rh, rh));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 v = split2(y[i]);
      if (scaled) v = make_float2(__fdiv_rn(v.x, hs), __fdiv_rn(v.y, hs));
      // (1e30: far beyond 6 s <= 2688)
      y[i] = pair2(fminf(fmaxf(v.x, -1e30f), 1e30f), fminf(fmaxf(v.y, -1e30f), 1e30f));
    }
  }
  // The nearest E2M1 value of y / s rounded to fp32 is that of y / s itself, unless
  // the rounding arrives at a midpoint between two codes.  (Elements that were not
  // divided have 8 significant bits and s has 4: their quotient is a midpoint or
  // 2^-12 away from it.)
  const float r = __frcp_rn(s);
  const uint64_t neg = pair2(-s, -s), rr = pair2(r, r);
  uint32_t q[8], low = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = split2(quotients(y[i], neg, rr));
    q[2 * i] = __float_as_uint(t.x);
    q[2 * i + 1] = __float_as_uint(t.y);
    if (scaled) low = min(low, min(q[2 * i] & 0xfffff, q[2 * i + 1] & 0xfffff));
  }
  if (scaled && low == 0) {
    // A midpoint (they have 3 significant bits) among them: the remainder says on
    // which side of it the quotient lies, and moves it there.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = split2(y[i]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float t = __uint_as_float(q[2 * i + e]), x = e ? v.y : v.x;
        const float rest = fmaf(-t, s, x) * t;  // > 0: further from zero
        if ((q[2 * i + e] & 0xfffff) == 0) q[2 * i + e] += (rest > 0.0f) - (rest < 0.0f);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (the sign is the element's own, also a zero's)
    const float2 v = make_float2(__uint_as_float((q[2 * i] & 0x7fffffffu) | (w[i] << 16 & 0x80000000u)),
                                 __uint_as_float((q[2 * i + 1] & 0x7fffffffu) | (w[i] & 0x80000000u)));
    *codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return s8;
}

// A thread's half group of the block's tokens t, t + step, ...; rows: where each
// token's row of head 0 begins in the pool, or -1.
template <bool kWrite, bool kScaled>
__device__ __forceinline__ void rows_of_unit(const Geo& g, int unit, const long long* rows, long long n0, int t,
                                             int step, int n) {
  constexpr int kBatch = kWrite ? 2 : 4;  // tokens in flight (a writer's registers are worth more warps)
  const Cache4RowsParams& a = g.a;
  const Place x(g, unit);
  const float* hp = x.is_v ? a.v_scale : a.k_scale;
  const float hs = hp ? __ldg(&hp[x.h]) : 1.0f;
  const int D = x.is_v ? a.Dv : a.Dk, d = 16 * x.j + 8 * x.half;
  const long long ts = x.is_v ? a.v_ts : a.k_ts;
  const __nv_bfloat16* src =
      kWrite ? (x.is_v ? a.v + x.h * a.v_hs : a.k + x.h * a.k_hs) + n0 * ts + d : nullptr;
  const long long out_step = (long long)a.Hk * D;
  __nv_bfloat16* out = x.is_v ? a.v_out : a.k_out;
  if (out) out += n0 * out_step + (long long)x.h * D + d;
  uint8_t* pool = a.pool + (long long)x.h * a.lay.bs * a.row_bytes;
  const int at = 8 * x.group + 4 * x.half, scale_at = 8 * g.groups + x.group;  // in a row
  for (int m0 = t; m0 < n; m0 += kBatch * step) {
    uint4 in[kBatch];
    uint32_t codes[kBatch], s8[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int m = m0 + i * step;
      if (m >= n) break;
      if (kWrite) {
        in[i] = __ldg(reinterpret_cast<const uint4*>(src + m * ts));
      } else {
        codes[i] = s8[i] = 0;
        if (rows[m] >= 0) {
          codes[i] = __ldg(reinterpret_cast<const uint32_t*>(pool + rows[m] + at));
          s8[i] = __ldg(pool + rows[m] + scale_at);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int m = m0 + i * step;
      if (m >= n) break;
      if (kWrite) {
        s8[i] = quantise<kScaled>(in[i], hs, &codes[i]);
        if (rows[m] >= 0) {
          uint8_t* p = pool + rows[m];
          *reinterpret_cast<uint32_t*>(p + at) = codes[i];
          if (x.half == 0) p[scale_at] = (uint8_t)s8[i];
          if (x.group == g.groups - 1 && x.half)
            for (int e = 9 * g.groups; e < a.row_bytes; ++e) p[e] = 0;
        }
      }
      if (out) *reinterpret_cast<uint4*>(out + m * out_step) = kept_values(codes[i], s8[i], hs);
    }
  }
}

template <bool kWrite, bool kScaled>
__global__ void __launch_bounds__(kThreads, kWrite ? 5 : 1) k_cache4_rows(const __grid_constant__ Geo g) {
  __shared__ long long rows[kChunk];
  const Cache4RowsParams& a = g.a;
  grid_dependency_wait();
  launch_dependents();
  const long long n0 = (long long)blockIdx.x * g.chunk;
  const int n = (int)min((long long)g.chunk, a.N - n0);
  if ((int)threadIdx.x < n) {
    int off = 0;
    const int page = token_page(a, (int)n0 + threadIdx.x, &off);
    if (page < 0) flag_status(a.status, DSA_STATUS_BAD_BLOCK);
    rows[threadIdx.x] = page < 0 ? -1 : ((long long)page * a.Hk * a.lay.bs + off) * a.row_bytes;
  }
  __syncthreads();
  if (g.tokens > 0) {
    const int t = threadIdx.x / g.units, unit = threadIdx.x - t * g.units;
    if (t < g.tokens) rows_of_unit<kWrite, kScaled>(g, unit, rows, n0, t, g.tokens, n);
  } else {
    for (int unit = threadIdx.x; unit < g.units; unit += kThreads) rows_of_unit<kWrite, kScaled>(g, unit, rows, n0, 0, 1, n);
  }
}

}  // namespace

int launch_cache4_rows(const Cache4RowsParams& p, bool write, cudaStream_t s) {
  Geo g{};
  g.a = p;
  g.gk = p.Dk / 16;
  g.groups = (p.Dk + p.Dv) / 16;
  if (p.N == 0) return DSA_OK;
  g.units = 2 * p.Hk * g.groups;
  g.tokens = kThreads / g.units;
  // as few tokens a block as fill the GPU, in whole passes of the block
  const int pass = std::max(g.tokens, 1), want = (int)((p.N + 8LL * sm_count() - 1) / (8LL * sm_count()));
  g.chunk = std::min(kChunk, (want + pass - 1) / pass * pass);
  const unsigned grid = (unsigned)((p.N + (long long)g.chunk - 1) / g.chunk);
  const cudaError_t e = launch_pdl(!write                      ? k_cache4_rows<false, false>
                             : p.k_scale || p.v_scale ? k_cache4_rows<true, true>
                                                      : k_cache4_rows<true, false>,
                             dim3(grid), dim3(kThreads), 0, s, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch(write ? "cache4_write" : "cache4_read");
}

}  // namespace dsa
