// cache4_attn.cu -- decode attention over the 4-bit cache (cache4.cuh), one
// query per sequence, grouped heads.
//
// The exact softmax over every cached position of a sequence ("Day-0
// Adaptation of Trillion-Parameter MoE Models on Domestic GPUs", section 3
// (2)-(3), with every position selected) on the values that the codes stand
// for.  Per key head the G = Hq / Hk query heads of its group form the columns
// of two products:
//   S^T [positions x heads] = K Q^T,   O^T [dims x heads] += V^T P^T.
//
// What bounds it: the cache's bytes, 9/16 of a byte per element, and next to
// them the instructions that turn codes into operands.  At the copy rate an SM
// takes in ~24 bytes, 42 elements, per cycle, so all work on an element has to
// fit in three lane-instructions.  The codes therefore never pass through
// shared memory in a wider form (84 bytes per cycle to write and again to read
// it for a tensor-core operand): a warp reads codes from its ring, widens them in
// registers to fp16 fragments and multiplies with mma.sync m16n8k16.
//   K: dims may be taken in any order that Q follows, so a lane takes whole
//      groups of 16 dims of a position (8 bytes, one scale): a byte of codes
//      becomes a pair by one conversion and one multiplication with the scale.
//   V: the product runs over positions, so pairs need the same dim of two
//      positions: their words are interleaved by nibble (a shift and a LOP3 per
//      word) before the same conversion.
// code x group scale has at most 6 significant bits and lies in 2^-10..2688:
// fp16 holds it exactly.  Q is brought into fp16's range by a power of two per
// head (what is lost is below 2^-24 of the head's largest element, what fp32
// sums lose too).  Weights enter the second product as fp16 (each off by at
// most 2^-11 of itself), 2^7 above their own size so that small weights of long
// sequences stay clear of its underflow; sums and statistics are fp32.
//
// Work is counted in units of 256 (dims up to 64: 512) positions of one (sequence,
// key head, block of heads); all units, item after item, are split evenly over the
// CTAs.  A warp takes 32 (64) positions of a unit, with its own ring of bulk copies
// (one per run of positions inside a page) and its own softmax; an item's warps are
// joined through shared memory, its CTAs by k_cache4_merge in a fixed order.
// Lengths are read on the device, so a captured call follows them.
//
// Measured: 32 sequences of 8 to 32 thousand positions, 64 heads over 8 of 128: 159
// us for 746 MB (4.7 TB/s, 70 % of the copy rate); 4 of 65 to 262 thousand, 32 heads
// over 4 of 64: 59 us (3.7 TB/s; rows of 72 bytes are kept in 80).  An element takes
// 2.9 lane-instructions of the three that the copy rate leaves; at 61 % of the issue
// slots and 49 % of the ALU (conversions and logic run at half rate) no unit is full:
// 16 warps an SM wait for their own chains (fixed latencies first, then a turn and the
// math pipes; little for memory).  On the way, for the
// first of these: 228 us with the dims read from the arguments, 187 with a row's
// layout known at compile time, 170 with what a unit is told by its stage instead of
// found again, 158 without spills and with the scales of unusable positions zeroed in
// place (for 8,192 positions a sequence a single spilled value made 77 us 120: shared
// memory leaves the L1 no room).  A warp of its own to fill one ring for all would
// leave 96 registers, which spill.  Tiles of 64 positions gain only where rows are
// short.  One sequence of 4,096: 12.8 us, the chain from the lengths over one tile a
// warp to the join.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "cache4.cuh"
#include "device_common.cuh"
#include "dsa_internal.cuh"
#include "sm100.cuh"

namespace dsa {

namespace {

using namespace sm100;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 320;               // partial slots are laid out for these
constexpr int kMaxStages = 8;
constexpr float kLift = 7.0f;               // weights are 2^7 times their size
constexpr float kRescaleLog2 = 8.0f;        // the maximum may lag by 2^8: weights stay below 2^15
// A weight is 2^(z cs + r) in one fma, exact but for the rounding of r and of zt, which
// grow with the maximum: an eighth of a power of two each at 2^20, whole ones that pass
// fp16's range beyond.  From there on z cs is rounded before r is added to it, and
// the maximum does not lag.  (Such a column's zt is NaN, so that every tile looks for
// its maximum.)
constexpr float kFar = 1048576.0f;

struct Geo {
  Cache4AttnParams a;
  int G, HB, HH;     // query heads per key head, blocks of them, items per sequence
  int gk, gv;        // groups of 16 dims
  int stages;
  int unit, lgunit;  // positions of a unit
  int lgbs;          // log2 of the page size, or -1
  int one;           // every warp's tile lies in one page
  int* off;          // [B + 1] first unit of each sequence, then the total
  float2* ml;        // [2 slots per CTA][rows]
  float* po;         // [2 slots per CTA][rows][Dv]
};

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ int seq_len(const Cache4AttnParams& a, int b) {
  const int L = __ldg(&a.lay.seq_lens[b]);
  return L < 0 ? 0 : min(L, a.lay.max_len);  // the bound that the host counted with
}
__device__ __forceinline__ int units_of(const Geo& g, int L) {  // (L may be 2^31 - 1)
  return (int)(((unsigned)L + (unsigned)g.unit - 1u) >> g.lgunit);
}

__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The units of one CTA, item by item.
struct Walk {
  int b, L, n;      // sequence, its positions, units of an item
  int hh, unit;     // item of the sequence, unit of the item
  int left;         // units of this CTA from here on, this one included
  __device__ __forceinline__ void load(const Geo& g) {
    L = uniform(seq_len(g.a, b));
    n = units_of(g, L);
  }
  // to the next unit; sequences without positions have none
  __device__ __forceinline__ void next(const Geo& g) {
    if (--left <= 0) return;
    if (++unit < n) return;
    unit = 0;
    if (++hh < g.HH) return;
    hh = 0;
    do {
      ++b;
      load(g);
    } while (n == 0);
  }
};

// CTA c of G takes units [T c / G, T (c + 1) / G).
__device__ __forceinline__ int first_unit(int T, int G, int c) {
  return (int)((long long)T * c / G);
}
__device__ __forceinline__ int owner(int T, int G, int x) {
  return (int)((((long long)x + 1) * G - 1) / T);
}

__device__ __forceinline__ int total_units(const Geo& g, int lane) {
  int sum = 0;
  for (int b = lane; b < g.a.lay.batch; b += 32) sum += units_of(g, seq_len(g.a, b));
  return uniform(__reduce_add_sync(0xffffffffu, sum)) * g.HH;
}

__device__ __forceinline__ Walk start_at(const Geo& g, int lo, int n, int lane) {
  Walk w{};
  w.left = n;
  if (n <= 0) return w;
  int at = 0;
  for (int b0 = 0; b0 < g.a.lay.batch; b0 += 32) {
    const int b = b0 + lane;
    const int u = b < g.a.lay.batch ? units_of(g, seq_len(g.a, b)) * g.HH : 0;
    const int end = at + warp_scan(u, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, end > lo);
    if (hit) {
      const int l = __ffs(hit) - 1;
      w.b = b0 + l;
      const int r = lo - __shfl_sync(0xffffffffu, end - u, l);
      w.load(g);
      w.hh = r / w.n;
      w.unit = r - w.hh * w.n;
      return w;
    }
    at = __shfl_sync(0xffffffffu, end, 31);
  }
  w.left = 0;
  return w;
}

// Two E2M1 codes a byte -> four pairs of fp16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two E4M3 scales (low byte first) -> a pair of fp16.
__device__ __forceinline__ uint32_t widen_scales(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

// Shared memory: barriers, what a stage holds, the warps' (maximum, sum), the
// join's buffers (half of the warps' O), then the warps' rings.
template <int NC, int NT>
struct Shared {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kO = kHeads * 64 * NC;  // floats of a warp's O
  static constexpr int kBars = 0;
  static constexpr int kMeta = kBars + 8 * kWarps * kMaxStages;
  static constexpr int kMl = kMeta + 16 * kWarps * kMaxStages;
  static constexpr int kAbort = kMl + 8 * kWarps * kHeads;
  static constexpr int kJoin = (kAbort + 4 + 127) / 128 * 128;
  static constexpr int kRing = kJoin + 4 * kO * (kWarps / 2);
};

// Flags of a unit, of its item's part in this CTA.
constexpr uint32_t kFirst = 1, kLast = 2, kFromStart = 4, kToEnd = 8;
constexpr uint32_t kEnd = 1u << 31;  // beside the sequence: the CTA's last unit

// A load that stays where it is written, a unit ahead of its use.
__device__ __forceinline__ int ld_early(const int32_t* p) {
  int r;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ float power_of_two(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

constexpr int per_sm(int NC, int NT, int RW) { return NC * NT * (RW / 32) <= 2 ? 2 : 1; }

// RW: positions of a warp's tile.  kFull: Dk = Dv = 64 NC, where a row's layout is
// known at compile time (its loads are one instruction each) and no group of 16 dims
// is missing: 32 x 8,192, 64 heads over 8 of 128 in 72 us, without it 85; 131,072 x
// 4, 32 over 4 of 64: 44 and 49; 8,192 x 16, 32 over 4 of 256: 45 and 58.
template <int NC, int NT, int RW, bool kFull>
__global__ void __launch_bounds__(kThreads, per_sm(NC, NT, RW))
    k_cache4_attn(const __grid_constant__ Geo g) {
  using Sh = Shared<NC, NT>;
  constexpr int kHeads = Sh::kHeads;
  constexpr int kRowsW = RW, kUnit = RW * kWarps, kHalves = RW / 32, kMt = RW / 16;
  extern __shared__ __align__(128) uint8_t sm[];
  const Cache4AttnParams& a = g.a;
  const int lane = threadIdx.x & 31, warp = uniform(threadIdx.x >> 5);
  const int gq = lane >> 2, t = lane & 3;  // row and column groups of a fragment
  launch_dependents();
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::kBars) + warp * kMaxStages;
  uint4* meta = reinterpret_cast<uint4*>(sm + Sh::kMeta) + warp * kMaxStages;
  float2* ml = reinterpret_cast<float2*>(sm + Sh::kMl);
  int* abort = reinterpret_cast<int*>(sm + Sh::kAbort);
  float* join = reinterpret_cast<float*>(sm + Sh::kJoin);
  if (lane == 0)
    for (int i = 0; i < g.stages; ++i) mbar_init(&bars[i], 1);
  if (threadIdx.x == 0) *abort = 0;
  fence_mbar_init();
  __syncthreads();
  grid_dependency_wait();

  const int T = total_units(g, lane);
  if (blockIdx.x == 0 && warp == 0) {  // for the join: first unit of every sequence
    int at = 0;
    for (int b0 = 0; b0 < a.lay.batch; b0 += 32) {
      const int b = b0 + lane;
      int u = 0;
      if (b < a.lay.batch) {
        const int L = seq_len(a, b);
        u = units_of(g, L) * g.HH;
        if (__ldg(&a.lay.seq_lens[b]) > L) flag_status(a.status, DSA_STATUS_BAD_LENGTH);
      }
      const int end = at + warp_scan(u, lane);
      if (b < a.lay.batch) g.off[b] = end - u;
      at = __shfl_sync(0xffffffffu, end, 31);
    }
    if (lane == 0) g.off[a.lay.batch] = T;
  }
  const int G = min(T, (int)gridDim.x);
  if ((int)blockIdx.x >= G) return;
  const int lo = first_unit(T, G, blockIdx.x);
  const int mine = first_unit(T, G, blockIdx.x + 1) - lo;

  const int RB = kFull ? (72 * NC + 15) / 16 * 16 : a.row_bytes;
  const int Dk = kFull ? 64 * NC : a.Dk, Dv = kFull ? 64 * NC : a.Dv;
  const int gk = kFull ? 4 * NC : g.gk, gv = kFull ? 4 * NC : g.gv;
  const uint32_t stage_bytes = kRowsW * RB;
  const uint32_t ring = smem_u32(sm + Sh::kRing) + warp * g.stages * stage_bytes;
  const int stages = g.stages;

  // ---- requests, a unit at a time: this warp's 32 positions of it (none at an
  // item's end), and what the unit is.  The pages are looked up a unit ahead.
  Walk w = start_at(g, lo, mine, lane);
  int rs = 0, us = 0;           // stage to fill, stage to read
  uint32_t uphase = 0;
  int page[kHalves], poff[kHalves];
  uint32_t flags = kFirst | (w.unit == 0 ? kFromStart : 0);
  bool ok = true;               // no wait of this CTA's ran out
  auto locate = [&] {  // page and row of this lane's positions of the unit
    const int p0 = w.unit * kUnit + warp * kRowsW;
    const int rows = min(w.L - p0, kRowsW);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int i = g.one ? 0 : 32 * h + lane;  // (one page holds the whole tile)
      if (i < rows && (h == 0 || !g.one)) {
        const unsigned p = (unsigned)(p0 + i);
        const unsigned s = g.lgbs >= 0 ? p >> g.lgbs : p / (unsigned)a.lay.bs;
        poff[h] = (int)(p - s * (unsigned)a.lay.bs);
        page[h] = ld_early(&a.lay.bt[(long long)w.b * a.lay.maxb + s]);
      }
    }
  };
  auto request = [&] {
    if (w.left <= 0) return;
    const int rows = min(w.L - (w.unit * kUnit + warp * kRowsW), kRowsW);
    uint32_t valid[2] = {0, 0};
    bool good[kHalves];
    if (g.one) {
      good[0] = rows > 0 && page[0] >= 0 && page[0] < a.lay.nb;
      if (rows > 0 && !good[0]) flag_status(a.status, DSA_STATUS_BAD_BLOCK);
      if (good[0]) {
        valid[0] = rows >= 32 ? 0xffffffffu : (1u << rows) - 1u;
        if (kHalves > 1) valid[1] = rows >= 64 ? 0xffffffffu : rows > 32 ? (1u << (rows - 32)) - 1u : 0u;
      }
    } else {
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const bool have = 32 * h + lane < rows;
        good[h] = have && page[h] >= 0 && page[h] < a.lay.nb;
        if (have && !good[h]) flag_status(a.status, DSA_STATUS_BAD_BLOCK);
        valid[h] = __ballot_sync(0xffffffffu, good[h]);
      }
    }
    if (!ok) valid[0] = valid[1] = 0;  // the units go by all the same: the warps meet at an item's end
    if (w.unit + 1 == w.n) flags |= kLast | kToEnd;
    if (w.left == 1) flags |= kLast;
    if (lane == 0) {
      meta[rs] = make_uint4(valid[0], valid[1], (uint32_t)w.b | (w.left == 1 ? kEnd : 0u), (uint32_t)w.hh << 4 | flags);
      if (ok) mbar_arrive_expect_tx(&bars[rs], (uint32_t)(__popc(valid[0]) + __popc(valid[1])) * RB);
    }
    __syncwarp();
    const uint8_t* head = a.pool + (long long)(w.hh / g.HB) * a.lay.bs * RB;
    const long long step = (long long)a.Hk * a.lay.bs * RB;  // to the next page
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int i = g.one ? 0 : 32 * h + lane;
      if (ok && (h == 0 || !g.one) && good[h] && (g.one ? lane == 0 : lane == 0 || poff[h] == 0)) {
        const int run = g.one ? rows : min(a.lay.bs - poff[h], min(rows - i, 32 - lane));
        bulk_copy(ring + rs * stage_bytes + i * RB, head + page[h] * step + (long long)poff[h] * RB,
                  (uint32_t)(run * RB), smem_u32(&bars[rs]));
      }
    }
    if (++rs == stages) rs = 0;
    flags = (flags & kLast) ? kFirst | kFromStart : flags & kFromStart;
    w.next(g);
    if (w.left > 0) locate();
  };
  locate();
  for (int i = 0; i < stages; ++i) request();

  // ---- the products
  const int nck = (gk + 3) >> 2, ncv = (gv + 3) >> 2;
  const int sk = (Dk + Dv) / 2, sv = sk + gk;  // scales of K and V within a row
  uint32_t qf[NC][4][NT][2];
  float cs[NT][2];              // score factor of this lane's two columns
  float o[NT][NC * 4][4];
  float l[NT][2];               // sum of the lane's weights
  float zt[NT][2];              // the product that passes the running maximum by 2^8; -inf: none yet
  float r[NT][2];               // kLift - the running maximum (log2)
  for (bool more = mine > 0; more;) {
    const uint4 what = meta[us];
    const uint32_t part = what.w & 15u;
    const uint32_t base = ring + us * stage_bytes;
    const int b = (int)(what.z & ~kEnd);
    more = (what.z & kEnd) == 0;
    // key head, first query head of the block, heads of the block
    auto heads_of_item = [&](int* hk, int* h0, int* heads) {
      const int hh = (int)(what.w >> 4);
      *hk = hh / g.HB;
      const int hb = hh - *hk * g.HB;
      *h0 = *hk * g.G + hb * kHeads;
      *heads = min(kHeads, g.G - hb * kHeads);
    };
    if (part & kFirst) {
      int hk, h0, heads;
      heads_of_item(&hk, &h0, &heads);
      const float ks = a.k_scale ? __ldg(&a.k_scale[hk]) : 1.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = 8 * nt + gq;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((size_t)b * a.Hq + h0 + h) * Dk);
        uint4 x[NC][2];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          x[c][0] = x[c][1] = make_uint4(0, 0, 0, 0);
          const int j = 4 * c + t;
          if (h < heads && j < gk) {
            x[c][0] = __ldg(&src[2 * j]);
            x[c][1] = __ldg(&src[2 * j + 1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {x[c][i].x, x[c][i].y, x[c][i].z, x[c][i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max((w[k] << 16) & 0x7fff0000u, w[k] & 0x7fff0000u));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // The head's largest element to [1, 2) or, of a subnormal one, below; in
        // two factors, as 2^-e itself may pass fp32's range.  0, infinity and NaN
        // stay what they are.
        const int e = top < 0x7f800000u ? max((int)(top >> 23), 1) - 127 : 0;
        const float down = power_of_two(-(e >> 1)), down2 = power_of_two((e >> 1) - e);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // step k of the chunk: dims 4 k .. 4 k + 3 of the lane's group
            const uint4 v = x[c][k >> 1];
            const uint32_t w0 = (k & 1) ? v.z : v.x, w1 = (k & 1) ? v.w : v.y;
            qf[c][k][nt][0] = pack_half2(__uint_as_float(w0 << 16) * down * down2,
                                         __uint_as_float(w0 & 0xffff0000u) * down * down2);
            qf[c][k][nt][1] = pack_half2(__uint_as_float(w1 << 16) * down * down2,
                                         __uint_as_float(w1 & 0xffff0000u) * down * down2);
          }
        // columns 2 t and 2 t + 1 are heads of lanes 8 t and 8 t + 4
        // (a factor of 0 would make NaN of the -inf of hidden positions; products of at
        // most 2^21 times the smallest normal number are scores of 0 all the same)
        const float f0 = a.scale_log2 * ks * power_of_two(e >> 1) * power_of_two(e - (e >> 1));
        const float f = f0 < power_of_two(-126) ? power_of_two(-126) : f0;
        cs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
        cs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        l[nt][0] = l[nt][1] = 0.0f;
        zt[nt][0] = zt[nt][1] = -INFINITY;
        r[nt][0] = r[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < NC * 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.0f;
      }
    }
    // (the queries came in while the item's first rows were on their way)
    if (ok && !pair_wait(smem_u32(&bars[us]), uphase, abort)) {
      ok = false;
      if (lane == 0) {
        *abort = 1;
        flag_status(a.status, DSA_STATUS_TIMEOUT);
      }
      // this warp's copies still on their way have a moment to land (a stage that
      // holds none is waited for in vain)
      int never = 0, s = us;
      uint32_t ph = uphase;
      for (int i = 0; i < stages; ++i) {
        pair_wait(smem_u32(&bars[s]), ph, &never, 10000000ull);
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (++us == stages) {
      us = 0;
      uphase ^= 1;
    }
    const uint32_t valid[2] = {ok ? what.x : 0u, ok ? what.y : 0u};
    if ((valid[0] | valid[1]) != 0) {
      const bool whole = (valid[0] & (kHalves > 1 ? valid[1] : 0xffffffffu)) == 0xffffffffu;
      float z[kMt][NT][4];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[mt][nt][k] = 0.0f;
        const uint32_t r0 = base + (16 * mt + gq) * RB, r1 = r0 + 8 * RB;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (!kFull && NC > 1 && c >= nck) break;
          const int j = 4 * c + t;
          uint2 w0 = make_uint2(0, 0), w1 = make_uint2(0, 0);
          uint32_t s0 = 0, s1 = 0;
          if (kFull || j < gk) {
            w0 = lds64(r0 + 8 * j);
            w1 = lds64(r1 + 8 * j);
            s0 = lds8(r0 + sk + j);
            s1 = lds8(r1 + sk + j);
          }
          s0 = widen_scales(s0 * 0x101u);
          s1 = widen_scales(s1 * 0x101u);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t x0[4], x1[4];
            widen(half ? w0.y : w0.x, x0);
            widen(half ? w1.y : w1.x, x1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a0 = mul2(x0[2 * k], s0), a2 = mul2(x0[2 * k + 1], s0);
              const uint32_t a1 = mul2(x1[2 * k], s1), a3 = mul2(x1[2 * k + 1], s1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(z[mt][nt], a0, a1, a2, a3, qf[c][2 * half + k][nt][0], qf[c][2 * half + k][nt][1]);
            }
          }
        }
      }
      if (!whole) {
        // The scales of V of unusable positions become 0: their weight is 0, but
        // what the row holds there may be NaN.  (The fence orders these stores before
        // the bulk copy that refills the stage: only it orders the two proxies.)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          if (!((valid[h] >> lane) & 1u))
#pragma unroll 1
            for (int j = 0; j < gv; ++j) sts8(base + (32 * h + lane) * RB + sv + j, 0);
        fence_proxy_async_smem();
        __syncwarp();
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!((valid[mt >> 1] >> (16 * (mt & 1) + gq + 8 * (k >> 1))) & 1u))
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) z[mt][nt][k] = -INFINITY;
      }
      // The lane's own scores first: the maximum of a column is only needed where
      // one passes the running one by 2^8 (in the products' own scale: zt).
      auto top_of = [&](int nt, int e) {
        float y = fmaxf(z[0][nt][e], z[0][nt][e + 2]);
#pragma unroll
        for (int mt = 1; mt < kMt; ++mt) y = max3(y, z[mt][nt][e], z[mt][nt][e + 2]);
        return y;
      };
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          up |= !(top_of(nt, e) <= zt[nt][e]);
      bool far = false;
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = top_of(nt, e);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
            f[e] = 1.0f;
            const float top = __fmul_rn(y, cs[nt][e]), old = kLift - r[nt][e];  // (cs > 0; rounded before it meets others)
            if (y > zt[nt][e] || (isnan(zt[nt][e]) && top > old)) {
              f[e] = zt[nt][e] == -INFINITY ? 0.0f : ex2_approx(old - top);
              r[nt][e] = kLift - top;
              zt[nt][e] = fabsf(top) > kFar ? NAN : y + kRescaleLog2 / cs[nt][e];
            }
            far |= isnan(zt[nt][e]);
          }
          l[nt][0] *= f[0];
          l[nt][1] *= f[1];
#pragma unroll
          for (int i = 0; i < NC * 4; ++i) {
            o[nt][i][0] *= f[0];
            o[nt][i][1] *= f[1];
            o[nt][i][2] *= f[0];
            o[nt][i][3] *= f[1];
          }
        }
        far = __any_sync(0xffffffffu, far);
      }
      uint32_t pf[kMt][NT][2];
      auto weigh = [&](auto apart) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint64_t c2 = pair2(cs[nt][0], cs[nt][1]), r2 = pair2(r[nt][0], r[nt][1]);
          uint64_t sum = pair2(l[nt][0], l[nt][1]);
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float z0 = z[mt][nt][2 * k], z1 = z[mt][nt][2 * k + 1];
              float2 y;
              if (decltype(apart)::value)
                y = make_float2(__fadd_rn(__fmul_rn(z0, cs[nt][0]), r[nt][0]), __fadd_rn(__fmul_rn(z1, cs[nt][1]), r[nt][1]));
              else
                y = split2(fma2(pair2(z0, z1), c2, r2));
              const float e0 = ex2_approx(y.x), e1 = ex2_approx(y.y);
              sum = add2(sum, pair2(e0, e1));
              pf[mt][nt][k] = transpose8(pack_half2(e0, e1));
            }
          const float2 l2 = split2(sum);
          l[nt][0] = l2.x;
          l[nt][1] = l2.y;
        }
      };
      if (far)
        weigh(std::true_type{});
      else
        weigh(std::false_type{});
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        // positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of the 16
        const uint32_t ra = base + (16 * mt + 2 * t) * RB;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (!kFull && NC > 1 && c >= ncv) break;
          const int j = 4 * c + (gq >> 1);  // the lane's 8 dims are half of group j
          uint32_t wa = 0, wb = 0, wc = 0, wd = 0, sab = 0, scd = 0;
          if (kFull || j < gv) {
            const uint32_t at = ra + Dk / 2 + 32 * c + 4 * gq, st = ra + sv + j;
            wa = lds32(at);
            wb = lds32(at + RB);
            wc = lds32(at + 8 * RB);
            wd = lds32(at + 9 * RB);
            sab = lds8(st) | (lds8(st + RB) << 8);
            scd = lds8(st + 8 * RB) | (lds8(st + 9 * RB) << 8);
          }
          sab = widen_scales(sab);
          scd = widen_scales(scd);
          // byte i: dim 2 i (2 i + 1) of both positions
          uint32_t e_ab[4], o_ab[4], e_cd[4], o_cd[4];
          widen((wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u), e_ab);
          widen(((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u), o_ab);
          widen((wc & 0x0f0f0f0fu) | ((wd << 4) & 0xf0f0f0f0u), e_cd);
          widen(((wc >> 4) & 0x0f0f0f0fu) | (wd & 0xf0f0f0f0u), o_cd);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = mul2(e_ab[i], sab), a1 = mul2(o_ab[i], sab);
            const uint32_t a2 = mul2(e_cd[i], scd), a3 = mul2(o_cd[i], scd);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[nt][4 * c + i], a0, a1, a2, a3, pf[mt][nt][0], pf[mt][nt][1]);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage and what it held
    request();
    if (part & kLast) {
      int hk, h0, heads;
      heads_of_item(&hk, &h0, &heads);
      // ---- join the warps: references and sums, then O in three rounds
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[nt][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          if (gq == 0) ml[warp * kHeads + 8 * nt + 2 * t + e] = make_float2(zt[nt][e] == -INFINITY ? -INFINITY : kLift - r[nt][e], x);
        }
      __syncthreads();
      float sum[NT][2], top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = -INFINITY, S = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kHeads + 8 * nt + 2 * t + e].x);
          const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w * kHeads + 8 * nt + 2 * t + e];
            S += x.y * ex2_approx(x.x - ref);
          }
          top[nt][e] = M;
          sum[nt][e] = S;
          const float f = zt[nt][e] == -INFINITY ? 0.0f : ex2_approx(kLift - r[nt][e] - ref);
#pragma unroll
          for (int i = 0; i < NC * 4; ++i) {
            o[nt][i][e] *= f;
            o[nt][i][e + 2] *= f;
          }
        }
#pragma unroll
      for (int r = kWarps / 2; r >= 1; r >>= 1) {
        if (warp >= r && warp < 2 * r) {
          // (from the second round on the buffer that this warp itself has read)
          float4* dst = reinterpret_cast<float4*>(join + (r == kWarps / 2 ? warp - r : warp) * Sh::kO) + lane;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < NC * 4; ++i)
              dst[32 * (nt * NC * 4 + i)] = make_float4(o[nt][i][0], o[nt][i][1], o[nt][i][2], o[nt][i][3]);
        }
        __syncthreads();
        if (warp < r) {
          const float4* src = reinterpret_cast<const float4*>(join + (r == kWarps / 2 ? warp : warp + r) * Sh::kO) + lane;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < NC * 4; ++i) {
              const float4 x = src[32 * (nt * NC * 4 + i)];
              o[nt][i][0] += x.x;
              o[nt][i][1] += x.y;
              o[nt][i][2] += x.z;
              o[nt][i][3] += x.w;
            }
        }
      }
      if (warp == 0) {
        // the lane's eight dims 64 c + 8 gq of columns 2 t and 2 t + 1
        const bool whole = (part & kFromStart) && (part & kToEnd);
        const int slot = 2 * blockIdx.x + ((part & kFromStart) ? 1 : 0);
        const float vs = a.v_scale ? __ldg(&a.v_scale[hk]) : 1.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = 8 * nt + 2 * t + e;
            if (h >= heads) continue;
            const size_t row = (size_t)b * a.Hq + h0 + h;
            const float f = whole ? (sum[nt][e] == 0.0f ? 0.0f : vs / sum[nt][e]) : 1.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int d = 64 * c + 8 * gq;
              if (d >= a.Dv) continue;
              float x[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[2 * i] = o[nt][4 * c + i][e] * f;
                x[2 * i + 1] = o[nt][4 * c + i][e + 2] * f;
              }
              if (whole) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                  w[i] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                *reinterpret_cast<uint4*>(a.out + row * a.Dv + d) = make_uint4(w[0], w[1], w[2], w[3]);
              } else {
                float4* dst = reinterpret_cast<float4*>(g.po + ((size_t)slot * kHeads + h) * a.Dv + d);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
              }
            }
            if (gq == 0) {
              if (!whole)
                g.ml[slot * kHeads + h] = make_float2(top[nt][e], sum[nt][e]);
              else if (a.lse)
                a.lse[row] = sum[nt][e] == 0.0f
                                 ? -INFINITY
                                 : (top[nt][e] - kLift + log2f(sum[nt][e])) * 0.6931471805599453f;
            }
          }
      }
    }
  }
}

// The join of an item's CTAs: a block per item that several CTAs share (and
// per sequence without positions), four columns a thread.
__global__ void __launch_bounds__(256) k_cache4_merge(const __grid_constant__ Geo g, int ctas, int kHeads) {
  constexpr int kBatch = 8;
  const Cache4AttnParams& a = g.a;
  const int b = blockIdx.x / g.HH, hh = blockIdx.x - b * g.HH;
  grid_dependency_wait();
  launch_dependents();
  const int T = __ldcg(&g.off[a.lay.batch]), u0 = __ldcg(&g.off[b]), n = (__ldcg(&g.off[b + 1]) - u0) / g.HH;
  const int G = min(T, ctas);
  const int hk = hh / g.HB, hb = hh - hk * g.HB;
  const int h0 = hk * g.G + hb * kHeads, heads = min(kHeads, g.G - hb * kHeads);
  int c0 = 0, parts = 0;
  if (n > 0) {
    c0 = owner(T, G, u0 + hh * n);
    parts = owner(T, G, u0 + hh * n + n - 1) - c0 + 1;
    if (parts == 1) return;  // written by its CTA
  }
  const float vs = a.v_scale ? __ldg(&a.v_scale[hk]) : 1.0f;
  const int quads = a.Dv / 4;
  for (int i = threadIdx.x; i < heads * quads; i += blockDim.x) {
    const int h = i / quads, x = i - h * quads;
    float M = -INFINITY, l = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += kBatch) {
      float2 st[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int p = p0 + q;
        // the first CTA holds the item's beginning in its second slot
        const int slot = 2 * (c0 + p) + (p == 0 ? 1 : 0);
        st[q] = make_float2(-INFINITY, 0.0f);
        v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < parts) {
          st[q] = __ldcg(&g.ml[slot * kHeads + h]);
          v[q] = __ldcg(reinterpret_cast<const float4*>(g.po + ((size_t)slot * kHeads + h) * a.Dv) + x);
        }
      }
      float Mn = M;
#pragma unroll
      for (int q = 0; q < kBatch; ++q) Mn = fmaxf(Mn, st[q].x);
      const float ref = Mn == -INFINITY ? 0.0f : Mn;
      const float f = ex2_approx(M - ref);
      l *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const float w = ex2_approx(st[q].x - ref);
        l = fmaf(st[q].y, w, l);
        acc.x = fmaf(v[q].x, w, acc.x);
        acc.y = fmaf(v[q].y, w, acc.y);
        acc.z = fmaf(v[q].z, w, acc.z);
        acc.w = fmaf(v[q].w, w, acc.w);
      }
      M = Mn;
    }
    const float f = l == 0.0f ? 0.0f : vs / l;
    const size_t row = (size_t)b * a.Hq + h0 + h;
    const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * f, acc.y * f);
    const __nv_bfloat162 hi2 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    *reinterpret_cast<uint2*>(a.out + row * a.Dv + 4 * x) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
    if (x == 0 && a.lse)
      a.lse[row] = l == 0.0f ? -INFINITY : (M - kLift + log2f(l)) * 0.6931471805599453f;
  }
}

// Chunks of 64 dims of the wider of K and V: 1, 2 or 4 (three take four), and
// heads in blocks of 16 where a group has more than 8 and registers allow it.
int chunks_of(int Dk, int Dv) {
  const int n = (std::max(Dk, Dv) + 63) / 64;
  return n > 2 ? 4 : n;
}
// Positions of a warp's tile: what a tile costs beside its rows weighs most where
// the rows are short (64 dims, 131,072 x 4 positions, at the time: 48 us with 64, 55 with 32;
// 128 dims, 8,192 x 32: 81 with 64, 80 with 32).
constexpr int rows_of(int nc, int heads) { return nc == 1 ? 64 : 32; }
// Heads of a block, the columns of both products: 16 read the rows of a larger group
// once (32 x 8,192, 128 heads over 8 of 128: 111 us, blocks of 8 133; 128 over 4 of
// 64: 63 and 74); in groups of up to 8 they would only carry zeros, and with more
// than 128 dims their accumulators do not fit the registers.
int heads_of(int Dk, int Dv, int G) { return G > 8 && chunks_of(Dk, Dv) <= 2 ? 16 : 8; }

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Layout {
  size_t off, ml, po, total;
};
Layout ws_layout(int B, int Dk, int Dv, int G) {
  Layout w;
  const size_t rows = (size_t)2 * kMaxCtas * heads_of(Dk, Dv, G);
  w.off = kWsHeader;
  w.ml = w.off + round256(sizeof(int) * ((size_t)B + 1));
  w.po = w.ml + round256(sizeof(float2) * rows);
  w.total = w.po + sizeof(float) * rows * Dv;
  return w;
}

template <int NC, int NT, int RW, bool kFull>
int launch(Geo& g, cudaStream_t s, long long bound, int* ctas_out) {
  using Sh = Shared<NC, NT>;
  constexpr int per = per_sm(NC, NT, RW);
  const int stage = RW * kWarps * g.a.row_bytes;  // of all warps
  const int room = 227 * 1024 / per - 1024 * (per - 1) - Sh::kRing;
  g.stages = std::min(kMaxStages, room / stage);
  const int smem = Sh::kRing + g.stages * stage;
  const void* k = (const void*)k_cache4_attn<NC, NT, RW, kFull>;
  int rc = ensure_dynamic_smem(k, smem, "cache4_attn_decode");
  if (rc) return rc;
  const int ctas = (int)std::min<long long>(std::min(kMaxCtas, per * sm_count()), std::max(1LL, bound));
  *ctas_out = ctas;
  const cudaError_t e = launch_pdl(k_cache4_attn<NC, NT, RW, kFull>, dim3((unsigned)ctas), dim3(kThreads), (size_t)smem, s, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("cache4_attn_decode");
}

}  // namespace

size_t cache4_attn_ws(int B, int Hq, int Hk, int Dk, int Dv) {
  return ws_layout(B, Dk, Dv, Hq / Hk).total;
}

int launch_cache4_attn(const Cache4AttnParams& p, void* ws, cudaStream_t s) {
  Geo g{};
  g.a = p;
  g.G = p.Hq / p.Hk;
  const int heads = heads_of(p.Dk, p.Dv, g.G), nc = chunks_of(p.Dk, p.Dv);
  g.HB = (g.G + heads - 1) / heads;
  g.HH = p.Hk * g.HB;
  g.gk = p.Dk / 16;
  g.gv = p.Dv / 16;
  g.lgbs = -1;
  for (int i = 0; i <= 10; ++i)
    if (p.lay.bs == 1 << i) g.lgbs = i;
  const Layout w = ws_layout(p.lay.batch, p.Dk, p.Dv, g.G);
  char* base = reinterpret_cast<char*>(ws);
  g.off = reinterpret_cast<int*>(base + w.off);
  g.ml = reinterpret_cast<float2*>(base + w.ml);
  g.po = reinterpret_cast<float*>(base + w.po);
  const long long items = (long long)p.lay.batch * g.HH;
  const int rw = rows_of(nc, heads);
  g.unit = rw * kWarps;
  g.lgunit = rw == 64 ? 9 : 8;
  const long long bound = items * (((long long)p.lay.max_len + g.unit - 1) / g.unit);
  if (bound > 0x7fffffffLL || items > 0x7fffffffLL)
    return set_error(DSA_ERR_UNSUPPORTED, "cache4_attn_decode: heads x positions beyond 2^31 units of 256");
  if (g.HH >= 1 << 27) return set_error(DSA_ERR_UNSUPPORTED, "cache4_attn_decode: 2^27 blocks of heads or more");
  g.one = p.lay.bs % rw == 0;
  const bool full = p.Dk == 64 * nc && p.Dv == 64 * nc;
  int ctas = 0, rc;
#define DSA_LAUNCH(NC, NT) \
  (full ? launch<NC, NT, rows_of(NC, 8 * NT), true>(g, s, bound, &ctas) \
        : launch<NC, NT, rows_of(NC, 8 * NT), false>(g, s, bound, &ctas))
  if (nc == 1)
    rc = heads == 8 ? DSA_LAUNCH(1, 1) : DSA_LAUNCH(1, 2);
  else if (nc == 2)
    rc = heads == 8 ? DSA_LAUNCH(2, 1) : DSA_LAUNCH(2, 2);
  else
    rc = DSA_LAUNCH(4, 1);
#undef DSA_LAUNCH
  if (rc) return rc;
  const cudaError_t e = launch_pdl(k_cache4_merge, dim3((unsigned)items), dim3(256), 0, s, g, ctas, heads);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("cache4_attn_decode merge");
}

}  // namespace dsa
