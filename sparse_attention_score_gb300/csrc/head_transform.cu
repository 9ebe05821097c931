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
// millions, where an fp32 product is off by whole fractions of a turn.  A
// frequency becomes a 64-bit fixed-point fraction of a turn (its mantissa times
// 2^64 / 2 pi, an integer product), and pos times that, modulo 2^64, wraps
// where the angle does: for inv_freq <= 1 the error is below pos * 2^-63
// turns.  Its upper 32 bits go through sincospif.
//
// One warp per item.  A head takes 8, 16 or 32 lanes (8 elements, 16 bytes per
// lane; heads beyond 256 elements three times that per lane), so a warp holds
// four, two or one heads at a time.  An item is a group of heads of one token,
// or, for parts of one head per token (cache rows), several tokens.  The
// warp forms the item's sines and cosines once; each lane folds them with the
// weights into
//   y_i = r (x_i A_i + partner_i B_i) + C_i,    r = 1 / rms (or deviation),
// so a head of 128 costs ~45 instructions of a warp whatever the norm and
// rotation, with the products two at a time (packed fp32).  Heads are loaded
// four at a time per lane.  Where a rotation begins or ends inside 8 elements
// (or its halves do), each element has a partner of its own and the heads go
// through shared memory as they were read, for the partners to be picked out
// of (8192 tokens, 40 heads of 128 rotated in 104: 44 us; in 96, by shuffles,
// 34).  A norm that ends inside 8 elements, a rotated pair on both sides of
// the norm's end, heads beyond 768 elements, and beyond 256 with such a
// rotation, take a plain path (195 us for the same heads).
//
// Measured on GB300: 16384 tokens, 64 rotated heads of 64 to bf16 and 64 heads
// of 128 to E4M3 (671 MB): 118 us, 5.7 TB/s, 84 % of the copy rate; 84 million
// warp instructions keep 56 % of the issue slots busy.  16384 cache rows of
// 576 with their indexer keys (44 MB): 21.6 us, where a third of the stalls
// are for instructions (each warp runs long code for a few rows).  One decode
// step of 32 tokens: 3 us, the launch.  Tried and left out: inputs requested
// before the position and page are known (15 % slower, registers), and a
// rolled loop over a wide head that reads it again from L1 (25-30 us for the
// cache rows).
#include <cuda_runtime.h>

#include <string>

#include "device_common.cuh"
#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxJobs = 2 * DSA_MAX_HEAD_PARTS;
constexpr int kMaxDim = 1024;
constexpr int kFlight = 4;  // 16-byte loads in flight per lane
constexpr int kWide = 3;    // granules per lane of a folded head beyond 256 elements

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
  int by_token;  // items: one head of several tokens, instead of heads of one token
  int groups;    // by_token 0: head groups per token; 1: heads
  int group;     // by_token 0: heads per group; 1: tokens per item
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

// Fraction of a turn per position, in units of 2^-64 turns: |f| / 2 pi =
// mantissa * 2^(e - 150) / 2 pi, with 2^64 / 2 pi as an integer.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  constexpr unsigned long long kTurn = 0x28BE60DB9391054Aull;  // 2^64 / 2 pi
  const uint32_t bits = __float_as_uint(f);
  int e = (int)(bits >> 23 & 0xffu);
  uint32_t m = bits & 0x7fffffu;
  if (e)
    m |= 0x800000u;
  else
    e = 1;
  const unsigned long long lo = kTurn * m, hi = __umul64hi(kTurn, m);
  const int s = 150 - e;  // the product times 2^-s
  unsigned long long u;
  if (s <= 0)
    u = s > -64 ? lo << -s : 0;
  else if (s < 64)
    u = (hi << (64 - s)) | (lo >> s);
  else
    u = s < 128 ? hi >> (s - 64) : 0;
  return (int)bits < 0 ? 0ull - u : u;
}

// (cos, sin) of pos * f, f as turns_of(f).
__device__ __forceinline__ float2 rotation(unsigned long long turns, int pos) {
  const unsigned long long u = turns * (unsigned long long)(long long)pos;
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

// Pairs of fp32 in one 64-bit register: Blackwell multiplies and adds two at a
// time (PTX mul / fma .f32x2), which the instruction-bound path here needs.
typedef unsigned long long f2;

__device__ __forceinline__ f2 pair2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& r, f2 (&v)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pair2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  f2 p[4];
  unpack8(r, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = split2(p[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void store8(const HeadJob& j, long long off, const f2 (&v)[4]) {
  if (j.fp8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(split2(v[2 * i]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(split2(v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(j.out) + off) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = split2(v[i]);
      const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(j.out) + off) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void store8(const HeadJob& j, long long off, const float (&v)[8]) {
  f2 p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair2(v[2 * i], v[2 * i + 1]);
  store8(j, off, p);
}

// What a lane knows of its head: the sub-warp's token and where it goes.
struct Where {
  long long tok;       // its token, -1: none
  long long out_base;  // element offset of the token's heads, -1: not stored
  int h0, h1;          // by_token 0: heads h0 .. h1 - 1; 1: the one head h0
  const float2* cs;    // cosines and sines of its token
};

// Plain path.  L lanes per head, J granules of 8 elements per lane.
template <int L, int J>
__device__ __noinline__ void transform_plain(const HeadJob& j, const Where w, float* stage) {
  const int lane = threadIdx.x & 31;
  const int sub = lane / L, li = lane % L;
  constexpr int kRows = 32 / L;
  const int G = j.dim >> 3;
  const int half = j.rope_dim >> 1;
  const int step = j.by_token ? j.heads : kRows;  // by_token: one round
  for (int h = w.h0; h < w.h1; h += step) {
    const int hh = j.by_token ? h : h + sub;
    const bool live = hh < w.h1 && w.tok >= 0;
    float v[J][8];
#pragma unroll
    for (int k = 0; k < J; ++k) {
      const int g = li + L * k;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (live && g < G)
        raw = *reinterpret_cast<const uint4*>(j.in + w.tok * j.in_ts + hh * j.in_hs + 8 * g);
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
              const float2 c = w.cs[e >> 1];
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
              const float2 c = w.cs[first ? e : e - half];
              const float p = st[first ? e + half : e - half];
              v[k][i] = first ? v[k][i] * c.x - p * c.y : v[k][i] * c.x + p * c.y;
            }
          }
        __syncwarp();
      }
    }
    if (live && w.out_base >= 0) {
#pragma unroll
      for (int k = 0; k < J; ++k) {
        const int g = li + L * k;
        if (g < G) store8(j, w.out_base + hh * j.out_hs + 8 * g, v[k]);
      }
    }
  }
}

// The folded form, one instantiation per kind of norm and rotation.
enum { kNoNorm = 0, kScale = 1, kFull = 2 };  // none; RMS without a bias; mean and / or bias
enum { kNoTurn = 0, kNeighbours = 1, kHalves = 2, kAny = 3 };  // kAny: either, from any even element
template <int n>
struct Int {
  static constexpr int value = n;
};
template <int n, int t>
struct Form {
  static constexpr int norm = n, turn = t;
};

// A lane's coefficients for granule g: y_i = r (x_i A_i + partner_i B_i) + C_i.
template <int kNorm, int kTurn>
struct Coef {
  f2 A[4], B[kTurn ? 4 : 1], C[kNorm == kFull ? 4 : 1];
  bool turned;   // the granule is rotated
  bool normed;
  int plane;     // lane that holds the partner granule (kHalves)
  int at[kTurn == kAny ? 8 : 1];  // kAny: byte of each partner among the staged heads
  unsigned pairs;                 // kAny: which pairs of the granule are rotated
};

// kAny: the heads of a warp's round in shared memory, as read (bf16).  Word w of
// lane l's granule is word 32 w + l: a lane's partners are a fixed distance
// away, so neither the writes nor the reads meet in a bank.
constexpr int kStaged = 512;  // bytes of a round

__device__ __forceinline__ void stage8(uint8_t* round, int lane, const uint4& raw) {
  uint32_t* d = reinterpret_cast<uint32_t*>(round) + lane;
  d[0] = raw.x;
  d[32] = raw.y;
  d[64] = raw.z;
  d[96] = raw.w;
}

// Coefficients of a granule whose elements each have a partner of their own.
// `first` is the lane of the head's first granule.
template <int kNorm>
__device__ __forceinline__ void coefs_any(const HeadJob& j, int g, int first, const float2* cs,
                                          Coef<kNorm, kAny>& c) {
  const int half = j.rope_dim >> 1;
  c.normed = kNorm != kNoNorm && 8 * g < j.norm_dim;
  c.pairs = 0;
  float A[8], B[8], C[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 8 * g + i, rel = e - j.rope_off;
    int pe = e;
    A[i] = 1.0f;
    B[i] = C[i] = 0.0f;
    if (8 * g < j.dim && rel >= 0 && rel < j.rope_dim) {
      const bool minus = j.interleaved ? (i & 1) == 0 : rel < half;
      pe = j.interleaved ? e ^ 1 : minus ? e + half : e - half;
      const float2 t = cs[j.interleaved ? rel >> 1 : minus ? rel : rel - half];
      A[i] = t.x;
      B[i] = minus ? -t.y : t.y;
      c.pairs |= 1u << (i >> 1);
    }
    c.at[i] = 4 * (32 * (pe >> 1 & 3) + first + (pe >> 3)) + 2 * (pe & 1);
    if (kNorm != kNoNorm && c.normed) {  // then the partner is normed too
      if (kNorm == kFull && j.bias) C[i] = __ldg(&j.bias[e]) * A[i] + __ldg(&j.bias[pe]) * B[i];
      if (j.weight) {
        A[i] *= __ldg(&j.weight[e]);
        B[i] *= __ldg(&j.weight[pe]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.A[i] = pair2(A[2 * i], A[2 * i + 1]);
    c.B[i] = pair2(B[2 * i], B[2 * i + 1]);
    if (kNorm == kFull) c.C[i] = pair2(C[2 * i], C[2 * i + 1]);
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ f2 swap2(f2 v) {
  const float2 f = split2(v);
  return pair2(f.y, f.x);
}

template <int kNorm, int kTurn>
__device__ __forceinline__ void coefs(const HeadJob& j, int g, int lane, const float2* cs,
                                      Coef<kNorm, kTurn>& c) {
  const int rel = 8 * g - j.rope_off;
  c.turned = kTurn != kNoTurn && 8 * g < j.dim && rel >= 0 && rel < j.rope_dim;
  c.normed = kNorm != kNoNorm && 8 * g < j.norm_dim;
  c.plane = lane;
  int gp = g;  // partner granule of the split halves
  float A[8], B[8], C[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    A[i] = 1.0f;
    B[i] = C[i] = 0.0f;
  }
  if (kTurn != kNoTurn && c.turned) {
    if (kTurn == kNeighbours) {
      const float4* t = reinterpret_cast<const float4*>(cs + (rel >> 1));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = t[i];
        A[4 * i] = A[4 * i + 1] = v.x;
        B[4 * i] = -v.y;
        B[4 * i + 1] = v.y;
        A[4 * i + 2] = A[4 * i + 3] = v.z;
        B[4 * i + 2] = -v.w;
        B[4 * i + 3] = v.w;
      }
    } else {
      const int half = j.rope_dim >> 1;
      const bool first = rel < half;
      const int d = first ? half >> 3 : -(half >> 3);
      gp = g + d;
      c.plane = lane + d;
      const float sgn = first ? -1.0f : 1.0f;
      const float4* t = reinterpret_cast<const float4*>(cs + (first ? rel : rel - half));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = t[i];
        A[2 * i] = v.x;
        B[2 * i] = sgn * v.y;
        A[2 * i + 1] = v.z;
        B[2 * i + 1] = sgn * v.w;
      }
    }
  }
  if (kNorm != kNoNorm && c.normed) {
    float q[8], qp[8];  // of the element, of its partner
    if (kNorm == kFull && j.bias) {
      load8(j.bias + 8 * g, q);
      if (kTurn == kHalves) load8(j.bias + 8 * gp, qp);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        C[i] = kTurn == kNoTurn ? q[i] : q[i] * A[i] + (kTurn == kHalves ? qp[i] : q[i ^ 1]) * B[i];
    }
    if (j.weight) {
      load8(j.weight + 8 * g, q);
      if (kTurn == kHalves) load8(j.weight + 8 * gp, qp);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        A[i] = kTurn == kNoTurn ? q[i] : A[i] * q[i];
        if (kTurn != kNoTurn) B[i] *= kTurn == kHalves ? qp[i] : q[i ^ 1];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.A[i] = pair2(A[2 * i], A[2 * i + 1]);
    if (kTurn != kNoTurn) c.B[i] = pair2(B[2 * i], B[2 * i + 1]);
    if (kNorm == kFull) c.C[i] = pair2(C[2 * i], C[2 * i + 1]);
  }
}

// 1 / rms or 1 / deviation of a head, from the sums over its normed elements;
// kFull also takes the mean off the values (and returns it).
template <int L, int J, int kNorm>
__device__ __forceinline__ float normalise(const HeadJob& j, f2 (&v)[J][4], int li, float* mean_out) {
  *mean_out = 0.0f;
  if (kNorm == kNoNorm) return 1.0f;
  const float inv = 1.0f / (float)j.norm_dim;
  if (kNorm == kFull && j.norm == DSA_NORM_LAYER) {
    f2 s = pair2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < J; ++k)
      if (8 * (li + L * k) < j.norm_dim) s = add2(s, add2(add2(v[k][0], v[k][1]), add2(v[k][2], v[k][3])));
    const float2 t = split2(s);
    const float mean = row_sum<L>(t.x + t.y) * inv;
    *mean_out = mean;
    const f2 off = pair2(-mean, -mean);
#pragma unroll
    for (int k = 0; k < J; ++k)
      if (8 * (li + L * k) < j.norm_dim) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = add2(v[k][i], off);
      }
  }
  f2 q = pair2(0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < J; ++k)
    if (8 * (li + L * k) < j.norm_dim) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(v[k][i], v[k][i], q);
    }
  const float2 t = split2(q);
  return rsqrtf(row_sum<L>(t.x + t.y) * inv + j.eps);
}

template <int kNorm, int kTurn>
__device__ __forceinline__ void finish8(const HeadJob& j, const Coef<kNorm, kTurn>& c,
                                        const f2 (&v)[4], float r, long long off, bool put,
                                        float mean = 0.0f, const uint8_t* round = nullptr) {
  f2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = mul2(v[i], c.A[i]);
  if (kTurn == kNeighbours) {
    if (c.turned) {  // elsewhere a neighbour's NaN must not meet a B of 0
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fma2(swap2(v[i]), c.B[i], y[i]);
    }
  } else if (kTurn == kAny) {
    const float off2 = kNorm == kFull && c.normed ? mean : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = *reinterpret_cast<const uint16_t*>(round + c.at[2 * i]);
      const uint32_t b = *reinterpret_cast<const uint16_t*>(round + c.at[2 * i + 1]);
      f2 p = pair2(__uint_as_float(a << 16), __uint_as_float(b << 16));
      if (kNorm == kFull) p = add2(p, pair2(-off2, -off2));
      if (c.pairs >> i & 1) y[i] = fma2(p, c.B[i], y[i]);
    }
  } else if (kTurn == kHalves) {
    f2 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xffffffffu, v[i], c.plane);
    if (c.turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fma2(p[i], c.B[i], y[i]);
    }
  }
  if (kNorm != kNoNorm) {
    const float rr = c.normed ? r : 1.0f;
    const f2 r2 = pair2(rr, rr);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = kNorm == kFull ? fma2(r2, y[i], c.C[i]) : mul2(r2, y[i]);
  }
  if (put) store8(j, off, y);
}

// Heads of at most 8 L elements: coefficients in registers, up to four heads
// in flight per lane.
template <int L, int kNorm, int kTurn>
__device__ __forceinline__ void transform_narrow(const HeadJob& j, const Where& w, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  const int sub = lane / L, li = lane % L;
  constexpr int kRows = 32 / L;
  Coef<kNorm, kTurn> c;
  if constexpr (kTurn == kAny)
    coefs_any(j, li, lane - li, w.cs, c);
  else
    coefs(j, li, lane, w.cs, c);
  const bool mine = 8 * li < j.dim && w.tok >= 0;
  constexpr int step = kRows;
  const int h0 = w.h0 + sub;
  const __nv_bfloat16* in = j.in + w.tok * j.in_ts + h0 * j.in_hs + 8 * li;
  long long off = w.out_base + h0 * j.out_hs + 8 * li;
  const long long in_step = step * j.in_hs, out_step = step * j.out_hs;
  const bool put = mine && w.out_base >= 0;
  const int rounds = (w.h1 - w.h0 + step - 1) / step;
  const int left = w.h1 - h0;  // of this sub-warp
  for (int r0 = 0; r0 < rounds; r0 += kFlight) {
    uint4 raw[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      raw[q] = make_uint4(0, 0, 0, 0);
      if (mine && (r0 + q) * step < left) raw[q] = *reinterpret_cast<const uint4*>(in + q * in_step);
    }
    if (kTurn == kAny) {
      __syncwarp();  // the rounds before are read
#pragma unroll
      for (int q = 0; q < kFlight; ++q) stage8(stage + kStaged * q, lane, raw[q]);
      __syncwarp();
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      if (r0 + q >= rounds) break;
      f2 v[1][4];
      unpack8(raw[q], v[0]);
      float mean;
      const float r = normalise<L, 1, kNorm>(j, v, li, &mean);
      finish8(j, c, v[0], r, off + q * out_step, put && (r0 + q) * step < left, mean,
              stage + kStaged * q);
    }
    in += kFlight * in_step;
    off += kFlight * out_step;
  }
}

// Heads beyond 256 elements: a warp per head, J granules per lane.  raw: head
// w.h0.
template <int J, int kNorm, int kTurn>
__device__ __forceinline__ void transform_wide(const HeadJob& j, const Where& w, uint4 (&raw)[J]) {
  const int lane = threadIdx.x & 31;
  for (int h = w.h0; h < w.h1; ++h) {
    f2 v[J][4];
#pragma unroll
    for (int k = 0; k < J; ++k) unpack8(raw[k], v[k]);
    if (h + 1 < w.h1) {
      const uint4* in = reinterpret_cast<const uint4*>(j.in + w.tok * j.in_ts + (h + 1) * j.in_hs);
#pragma unroll
      for (int k = 0; k < J; ++k)
        if (8 * (lane + 32 * k) < j.dim) raw[k] = in[lane + 32 * k];
    }
    float mean;
    const float r = normalise<32, J, kNorm>(j, v, lane, &mean);
#pragma unroll
    for (int k = 0; k < J; ++k) {
      const int g = lane + 32 * k;
      Coef<kNorm, kTurn> c;
      coefs(j, g, lane, w.cs, c);
      finish8(j, c, v[k], r, w.out_base + h * j.out_hs + 8 * g, 8 * g < j.dim && w.out_base >= 0);
    }
  }
}

// The instantiation for the part's norm and rotation.  kFull is right for every
// norm; only heads in groups, where the rounds are many, have kScale too (each
// form costs compile time and instruction cache).
template <bool kScaleToo, bool kAnyTurns, typename F>
__device__ __forceinline__ void by_form(const HeadJob& j, F f) {
  auto turn = [&](auto norm) {
    constexpr int n = decltype(norm)::value;
    if (j.rope_dim == 0)
      f(Form<n, kNoTurn>());
    else if constexpr (kAnyTurns)
      f(Form<n, kAny>());
    else if (j.interleaved)
      f(Form<n, kNeighbours>());
    else
      f(Form<n, kHalves>());
  };
  if (j.norm == DSA_NORM_NONE)
    turn(Int<kNoNorm>());
  else if (kScaleToo && j.norm == DSA_NORM_RMS && !j.bias)
    turn(Int<kScale>());
  else
    turn(Int<kFull>());
}

// The position of token t, and where its heads go (w.tok, h0, h1 are set).
__device__ __forceinline__ int locate(const HeadParams& p, const HeadJob& j, int t, bool flag,
                                      Where& w) {
  const bool there = w.tok >= 0;
  const int b = !there ? -1 : p.seq ? __ldg(&p.seq[t]) : t;
  int pos = 0;
  if (there && p.pos)
    pos = __ldg(&p.pos[t]);
  else if (b >= 0 && b < p.lay.batch)
    pos = __ldg(&p.lay.seq_lens[b]) - 1;
  w.out_base = there ? t * j.out_ts : -1;
  if (j.paged && there) {
    long long row = -1;
    if (b >= 0 && b < p.lay.batch && pos >= 0) {
      const unsigned slot = (unsigned)pos / (unsigned)p.lay.bs;
      if (slot < (unsigned)p.lay.maxb) {
        const int page = __ldg(&p.lay.bt[(long long)b * p.lay.maxb + slot]);
        if (page >= 0 && page < p.lay.nb)
          row = (long long)page * p.lay.bs + (pos - (int)(slot * (unsigned)p.lay.bs));
      }
    }
    if (row < 0 && flag) flag_status(p.status, DSA_STATUS_BAD_BLOCK);
    w.out_base = row < 0 ? -1 : row * j.out_ts;
  }
  return pos;
}

__device__ __forceinline__ void wide_item(const HeadParams& p, const HeadJob& j, int t, Where& w,
                                          float2* cs) {
  const int lane = threadIdx.x & 31;
  constexpr int J = kWide;
  // the first head is on its way while position and page are looked up
  const uint4* in = reinterpret_cast<const uint4*>(j.in + t * j.in_ts + w.h0 * j.in_hs);
  uint4 raw[J];
#pragma unroll
  for (int k = 0; k < J; ++k) {
    raw[k] = make_uint4(0, 0, 0, 0);
    if (8 * (lane + 32 * k) < j.dim) raw[k] = in[lane + 32 * k];
  }
  const int pos = locate(p, j, t, lane == 0, w);
  const int half = j.rope_dim >> 1;
  w.cs = cs;
  for (int i = lane; i < half; i += 32) cs[i] = rotation(turns_of(__ldg(&j.inv_freq[i])), pos);
  __syncwarp();
  by_form<false, false>(j, [&](auto f) { transform_wide<J, f.norm, f.turn>(j, w, raw); });
}

// One head of tokens t0, t0 + 1, .. t1 - 1, 32 / L at a time (parts with fewer
// heads than a warp holds: cache rows).  The frequencies' turns stay in
// registers, the next tokens' rows and positions are on their way while these
// are worked on.
template <int L, int J, int kNorm, int kTurn>
__device__ __forceinline__ void transform_tokens(const HeadParams& p, const HeadJob& j, int t0, int t1,
                                                 int h, float2* cs, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  const int sub = lane / L, li = lane % L;
  constexpr int kRows = 32 / L;
  const int half = kTurn == kNoTurn ? 0 : j.rope_dim >> 1;
  float2* mine = cs + sub * ((half + 1) & ~1);
  unsigned long long u[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (li + L * i < half) u[i] = turns_of(__ldg(&j.inv_freq[li + L * i]));
  const __nv_bfloat16* in = j.in + h * j.in_hs + 8 * li;
  Where w;
  w.h0 = h;
  w.h1 = h + 1;
  w.cs = mine;
  uint4 raw[J];
  auto fetch = [&](int t) {
#pragma unroll
    for (int k = 0; k < J; ++k) {
      raw[k] = make_uint4(0, 0, 0, 0);
      if (t < t1 && 8 * (li + L * k) < j.dim)
        raw[k] = *reinterpret_cast<const uint4*>(in + t * j.in_ts + 8 * L * k);
    }
  };
  fetch(t0 + sub);
  w.tok = t0 + sub < t1 ? t0 + sub : -1;
  int pos = locate(p, j, t0 + sub, li == 0, w);
  for (int base = t0; base < t1; base += kRows) {
    const int t = base + sub;
    if (kTurn != kNoTurn) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (li + L * i < half) mine[li + L * i] = rotation(u[i], pos);
      for (int i = li + 2 * L; i < half; i += L)
        mine[i] = rotation(turns_of(__ldg(&j.inv_freq[i])), pos);
      if (kTurn == kAny) stage8(stage, lane, raw[0]);
      __syncwarp();
    }
    f2 v[J][4];
#pragma unroll
    for (int k = 0; k < J; ++k) unpack8(raw[k], v[k]);
    const long long out = w.out_base + h * j.out_hs + 8 * li;
    const bool put = w.tok >= 0 && w.out_base >= 0;
    if (base + kRows < t1) {
      fetch(t + kRows);
      w.tok = t + kRows < t1 ? t + kRows : -1;
      pos = locate(p, j, t + kRows, li == 0, w);
    }
    float mean;
    const float r = normalise<L, J, kNorm>(j, v, li, &mean);
    if constexpr (kTurn == kAny) {
      static_assert(J == 1, "staged heads have a granule per lane");
      Coef<kNorm, kAny> c;
      coefs_any(j, li, lane - li, mine, c);
      finish8(j, c, v[0], r, out, put && 8 * li < j.dim, mean, stage);
      continue;
    } else {
#pragma unroll
    for (int k = 0; k < J; ++k) {
      const int g = li + L * k;
      const bool live = put && 8 * g < j.dim;
      // granules L k .. L k + L - 1: all outside the rotation, for every lane?
      if (kTurn != kNoTurn && (J == 1 || (8 * L * k < j.rope_off + j.rope_dim && 8 * L * (k + 1) > j.rope_off))) {
        Coef<kNorm, kTurn> c;
        coefs(j, g, lane, mine, c);
        finish8(j, c, v[k], r, out + 8 * L * k, live);
      } else {
        Coef<kNorm, kNoTurn> c;
        coefs(j, g, lane, mine, c);
        finish8(j, c, v[k], r, out + 8 * L * k, live);
      }
    }
    }
  }
}

// What the parts of a launch need: folded heads of up to 256 elements, up to
// 768 elements, of up to 256 with rotations that begin or end inside 8
// elements, or the plain path (then for all of its parts).
enum { kNarrowOnly = 0, kWithWide = 1, kAnyTurn = 2, kPlain = 3 };

template <int kKind>
__global__ void __launch_bounds__(kWarps * 32, kKind == kNarrowOnly ? 8 : 6)
    k_head_transform(const __grid_constant__ HeadParams p) {
  extern __shared__ float4 smraw[];
  grid_dependency_wait();
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* base = reinterpret_cast<float*>(smraw) + (size_t)warp * (2 * p.cs_len + p.stage_len);
  float2* cs = reinterpret_cast<float2*>(base);
  float* stage = base + 2 * p.cs_len;
  uint8_t* staged = reinterpret_cast<uint8_t*>(stage);
  const int item = blockIdx.x * kWarps + warp;
  if (item >= p.items) return;
  int n = 0;
  while (n + 1 < p.n_jobs && item >= p.job[n + 1].first) ++n;
  const HeadJob& j = p.job[n];
  const int at = item - j.first;
  const int G = j.dim >> 3;
  const int L = G <= 8 ? 8 : G <= 16 ? 16 : 32;
  const int sub = lane / L, li = lane % L;
  const int hi = at / j.groups, lo = at - hi * j.groups;
  if (kKind != kPlain && j.by_token) {
    const int t0 = hi * j.group, t1 = min(p.N, t0 + j.group);
    by_form<false, kKind == kAnyTurn>(j, [&](auto f) {
      if (G <= 16)
        transform_tokens<16, 1, f.norm, f.turn>(p, j, t0, t1, lo, cs, staged);
      else if (kKind != kWithWide || G <= 32)
        transform_tokens<32, 1, f.norm, f.turn>(p, j, t0, t1, lo, cs, staged);
      else if constexpr (kKind == kWithWide)
        transform_tokens<32, kWide, f.norm, f.turn>(p, j, t0, t1, lo, cs, staged);
    });
    return;
  }
  int t;
  Where w;
  if (kKind == kPlain && j.by_token) {  // one round of tokens
    t = hi * j.group + sub;
    w.h0 = lo;
    w.h1 = lo + 1;
  } else {
    t = hi;
    w.h0 = lo * j.group;
    w.h1 = min(j.heads, w.h0 + j.group);
  }
  w.tok = t < p.N ? t : -1;
  if (kKind == kWithWide && G > 32) {
    wide_item(p, j, t, w, cs);
    return;
  }
  const int pos = locate(p, j, t, li == 0, w);
  const int half = j.rope_dim >> 1;
  w.cs = cs;
  if (half) {
    if (kKind == kPlain && j.by_token) {
      float2* mine = cs + sub * ((half + 1) & ~1);
      for (int i = li; i < half; i += L) mine[i] = rotation(turns_of(__ldg(&j.inv_freq[i])), pos);
      w.cs = mine;
    } else {
      for (int i = lane; i < half; i += 32) cs[i] = rotation(turns_of(__ldg(&j.inv_freq[i])), pos);
    }
    __syncwarp();
  }
  if (kKind == kPlain) {
    if (L == 8)
      transform_plain<8, 1>(j, w, stage);
    else if (L == 16)
      transform_plain<16, 1>(j, w, stage);
    else if (G <= 32)
      transform_plain<32, 1>(j, w, stage);
    else
      transform_plain<32, 4>(j, w, stage);
    return;
  }
  by_form<true, kKind == kAnyTurn>(j, [&](auto f) {
    if (L == 8)
      transform_narrow<8, f.norm, f.turn>(j, w, staged);
    else if (L == 16)
      transform_narrow<16, f.norm, f.turn>(j, w, staged);
    else
      transform_narrow<32, f.norm, f.turn>(j, w, staged);
  });
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
  bool plain = false, any = false, wide = false;
  for (int i = 0; i < p.n_jobs; ++i) {
    HeadJob& j = p.job[i];
    const bool paged = i < n_cache;
    const int rc = check_part(paged ? cache[i] : heads[i - n_cache], N, paged, &j);
    if (rc) return rc;
    j.by_token = j.heads == 1;
    // the folded forms: the norm ends at a whole granule, and a rotated element
    // and its partner are both normed or both not ...
    const int r0 = j.rope_off, r1 = j.rope_off + j.rope_dim;
    const bool folds = j.dim <= 256 * kWide && (j.norm == DSA_NORM_NONE || j.norm_dim % 8 == 0) &&
                       (j.rope_dim == 0 || j.norm == DSA_NORM_NONE || r1 <= j.norm_dim ||
                        r0 >= j.norm_dim);
    // ... and partners in whole granules, the same register of two lanes; else
    // they go through shared memory
    const bool whole = j.rope_dim == 0 ||
                       (r0 % 8 == 0 && r1 % 8 == 0 &&
                        (j.interleaved || (j.rope_dim % 16 == 0 &&
                                           (j.dim <= 256 || r0 / 256 == (r1 - 1) / 256))));
    plain |= !folds;
    any |= !whole;
    wide |= j.dim > 256;
  }
  const int kind = plain || (any && wide) ? kPlain : any ? kAnyTurn : wide ? kWithWide : kNarrowOnly;
  for (int i = 0; i < p.n_jobs; ++i) {
    HeadJob& j = p.job[i];
    const int rpw = rows_per_warp(j.dim);
    const int pairs = ((j.rope_dim / 2 + 1) & ~1) * (j.by_token ? rpw : 1);
    if (pairs > p.cs_len) p.cs_len = pairs;
    if (kind == kPlain && !j.interleaved && rpw * j.rope_dim > p.stage_len)
      p.stage_len = rpw * j.rope_dim;
  }
  p.stage_len = (p.stage_len + 3) & ~3;
  if (kind == kAnyTurn) p.stage_len = kFlight * kStaged / 4;
  long long rows = 0;  // parts of at most 2^31 heads each: no overflow
  for (int i = 0; i < p.n_jobs; ++i) rows += (long long)N * p.job[i].heads;
  if (rows > 0x7fffffffLL - 63)  // room for the last block's idle warps in 32 bits
    return set_error(DSA_ERR_UNSUPPORTED, "head parts: tokens x heads beyond 2^31 - 64");
  // Heads per item: as many rounds of the warp as still leave 12 items per SM
  // (the sines, cosines and coefficients are the item's), 32 with 16 rounds and
  // where all parts are rows of tokens, one round where there are few tokens
  // and latency counts.  Measured with 12 and with 32 items: 200 tokens of 33 +
  // 8 heads of 224 6.1 and 10.1 us, 777 tokens of 24 + 4 heads of 80 4.8 and
  // 6.5; but 2000 tokens of 16 + 32 heads, with 16 rounds, 11.1 and 9.1, and
  // 8112 rows of K, V and indexer keys 12.7 and 10.7.
  bool rows_only = true;
  for (int i = 0; i < p.n_jobs; ++i) rows_only &= p.job[i].by_token != 0;
  long long items = 0;
  for (int rounds = 16; rounds >= 1; rounds /= 2) {
    items = 0;
    for (int i = 0; i < p.n_jobs; ++i) {
      HeadJob& j = p.job[i];
      const int rpw = rows_per_warp(j.dim);
      j.first = (int)items;
      if (j.by_token) {
        // the folded token loop takes 16 lanes for a head of up to 128
        j.group = kind == kPlain ? rpw : (j.dim <= 128 ? 2 : 1) * (rounds < 4 ? rounds : 4);
        j.groups = j.heads;
        items += ((long long)N + j.group - 1) / j.group * j.heads;
      } else {
        j.group = rounds * rpw < j.heads ? rounds * rpw : j.heads;
        j.groups = (j.heads + j.group - 1) / j.group;
        const int even = (j.heads + j.groups - 1) / j.groups;  // no group much shorter
        j.group = (even + rpw - 1) / rpw * rpw;
        items += (long long)N * j.groups;
      }
    }
    if (items >= (rounds > 8 || rows_only ? 32LL : 12LL) * sm_count()) break;
  }
  if (N == 0) return DSA_OK;
  p.items = (int)items;
  const size_t smem = sizeof(float) * kWarps * (2 * (size_t)p.cs_len + p.stage_len);
  const long long grid = (items + kWarps - 1) / kWarps;
  const cudaError_t e =
      launch_pdl(kind == kNarrowOnly ? k_head_transform<kNarrowOnly>
                 : kind == kWithWide ? k_head_transform<kWithWide>
                 : kind == kAnyTurn  ? k_head_transform<kAnyTurn>
                                     : k_head_transform<kPlain>,
                 dim3((unsigned)grid), dim3(kWarps * 32), smem, s, p);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("head_transform");
}

}  // namespace dsa
