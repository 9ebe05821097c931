// prefix_attn.cu -- exact decode attention over every cached position, for a
// batch that shares a prefix, on the tensor cores of SM pairs.
//
// The gather through the block table and the exact softmax are those of the
// sparse attention ("Day-0 Adaptation of Trillion-Parameter MoE Models on
// Domestic GPUs", section 3 (2)-(3)) with every position selected.  The rows
// of all sequences (B x Hq) are laid end to end; over the shared prefix they
// form M = 128 row tiles whatever sequence they belong to, so each cached row
// of the prefix is read once per 128 rows instead of once per sequence.
// Behind the prefix each sequence's Hq rows go over its own positions.
//
// Lines and tiles.  A line is one row tile over the prefix, or one sequence
// over its own positions; it is cut in tiles of 256 positions.  All tiles,
// line after line, are split evenly over the CTA pairs; each pair leaves one
// unnormalised partial (O, m, l) per line it touches and k_prefix_merge joins
// a row's partials in a fixed order:
//   M = max m_s,  l = sum l_s 2^(m_s - M),  O = sum O_s 2^(m_s - M) / l.
// Lengths are read on the device, so a captured call follows them.
//
// One tile on a pair (tcgen05 cta_group::2, M = 128: 64 rows per CTA).  The
// accumulator of 64 rows x N columns fills all 128 TMEM lanes with N / 2
// columns (lanes 64..127 hold columns N / 2..N - 1), so O[64 x 512] and two
// S[64 x 256] buffers fill TMEM exactly, and each CTA stages only half of
// every B operand:
//   S   [128 x 256] = Q . K^T    9 chunks of 64 dims (576), N = 256; CTA r
//       stages positions 128 r .. 128 r + 127 of the tile;
//   softmax: 4 warps per CTA, a thread has one row's scores of one half of
//       the tile; the running maximum is raised only when a tile exceeds it
//       by more than 2^8, and O is rescaled in TMEM then;
//   O   [128 x Dv] += P . V      V as stored (MN-major), N = 256 columns per
//       instruction; CTA r stages half of the columns of all 256 positions.
// P is rounded to bf16 for the second product (each weight by at most 2^-8 of
// itself, like the output's own rounding), except in short sequences; sums and
// statistics are fp32.
//
// Short sequences.  Over a few positions the roundings of single weights do not
// average out: with two or three, an output of N(0, 1) rows was off by up to
// 1.1e-2.  Where a line's rows may have no more than 512 positions (the
// sequence has, or the prefix), P is therefore kept as bf16 hi + lo, off by
// 2^-16 of itself, as in the sparse attention.  Such a line's tiles are 128
// positions: S is [128 x 128] (N = 128, a half of the tile 64 columns), each
// half writes hi to the first and lo to the second of its two chunks of P, and
// both are multiplied with the same 64 positions of V.  In a graph, against one
// bf16 for every line: one sequence of one position 14.2 us, was 12.9; 32 of up
// to 512 21.9, was 20.7; that a line may be short costs the others 1 to 3 %.
// (Hi first, and lo once the half had read its scores again, with V staged
// twice: 32 of up to 512 25.1 us.)
//
// Warp roles (256 threads): 0-3 softmax and O out of TMEM; 4 fills the ring of
// K (and Q, and the usable positions of a tile), 5 issues S; 6 fills the ring
// of V, 7 issues O (5 and 7 in CTA 0 of the pair only).  Each ring has one
// filler and one reader, so a barrier's phase is never a lap off.  The weights
// are handed over in four chunks of 64 positions and their buffer is taken
// back in halves, so that S of the next tile, its softmax and O of this one
// run side by side.
//
// What bounds it.  A tile is 36 MMAs for S and 32 for O, 64 cycles each: 4,352
// cycles of the tensor cores for 71 MFLOP.  Per CTA it also takes 278 KB from
// L2 through 112 KB of rings: a stage comes round in ~1,450 cycles (copy 840,
// MMAs 256, barriers and issue the rest), which allows ~77 bytes a cycle and
// needs 64.  Measured on GB300 (in a graph, warm): ~5,800 cycles per tile; 64
// sequences of 64 heads behind a prefix of 65,536: 350 us, 1,670 TFLOP/s (87 %
// of the cuBLAS rate); 32 behind 16,384: 66 us, 1,170 TFLOP/s.  Short lines are
// bound by the chain from the lengths to the output (a tile a pair: 10.5 us,
// 3 of them until the first copy of K is issued, 1 to write O, 3 for the join).
//
// Boxes are R rows high, R the largest power of two (at most 64) that divides
// the page size: such a group of positions never crosses a page.  A sequence's
// own tiles begin at the group that the prefix ends in.  A group that a line
// begins or ends in is staged for V in boxes of powers of two rows, and rows
// that are not the line's, or behind a bad block id, come from outside the
// pool, which TMA fills with zeros: whatever the cache holds there (NaN
// included) never meets a weight of 0.  Pages below 64 rows take more boxes, and
// what a box costs is its issue: rows come out of a lane's register by shuffle,
// loops are short, and 16 or 32 rows of V take both 64-column blocks in one box.
// 32 sequences behind 16,384 positions, own parts of up to 512: 58 us with
// pages of 64, 64 with 32, 72 with 16, 92 with 8 (rows read from shared memory
// one by one: 56, 87, 126 and 203).
// Every wait is bounded (DSA_STATUS_TIMEOUT, then the pair winds down).
#include <algorithm>

#include "device_common.cuh"
#include "dsa_internal.cuh"
#include "sm100.cuh"

namespace dsa {

namespace {

using namespace sm100;

constexpr int kTile = 256;             // positions per tile
constexpr int kRows = 128;             // rows of a pair, 64 per CTA
constexpr int kMaxChunks = 9;          // 64-dim chunks of a query row
constexpr int kStagesK = 4, kStagesV = 3;
constexpr int kStageBytes = 16384;
constexpr int kThreads = 256;          // softmax 0-3, K 4 (producer) and 5 (MMA), V 6 and 7
constexpr int kMaxPairs = 80;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;          // two S buffers of 128 columns
constexpr uint32_t kColO = 256;        // O: 128 columns per 256 dims of V
constexpr float kRescaleLog2 = 8.0f;
constexpr int kTabs = 8;               // tiles whose mask is kept (see the K producer)
constexpr int kShort = 512;            // lines of rows with at most this many positions: P as hi + lo

struct __align__(1024) Smem {
  uint8_t ringk[kStagesK][kStageBytes];
  uint8_t ringv[kStagesV][kStageBytes];
  uint8_t q[kMaxChunks][64 * 128];
  uint8_t p[kTile / 64][64 * 128];
  int tab[2][kTile];                   // per producer: physical row of each group of R positions
  uint32_t mask[kTabs][kTile / 32];    // usable positions
  int whole[kTabs];                    // every position of the tile is usable
  uint64_t fullk[kStagesK], emptyk[kStagesK], fullv[kStagesV], emptyv[kStagesV], qfull, qempty;
  uint64_t sfull[2], sfree[2], oready[2], pfull[4], pdone[2], pvdone;
  uint64_t vfull[kTabs], smsync[2], done;
  float redm[2][2][64];
  int fills[3];  // stages of K and V, and Q: times filled, for the drain after a failure
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory of k_prefix_attn");

struct Maps {
  CUtensorMap q, k, v[7];  // v[i]: boxes of 2^i rows of 64 columns
  CUtensorMap v2;          // boxes of R rows of two 64-column blocks
};

struct Geo {
  PrefixAttnParams a;
  int R;            // rows per box
  int lgbs;         // log2 of the page size, or -1
  // V is staged [group of Rv positions][64-column block][position of the group];
  // where 16 <= R < 64, R itself, so that a box can hold both blocks (`wide`:
  // Dv a multiple of 256) and 16 positions, an MMA's, still lie in one group.
  // With R = 64 two boxes of 8 KB are ahead of one of 16: 345 against 350 us
  // for 64 sequences behind 65,536 positions.
  int Rv;
  int wide;
  int row_tiles;    // of 128 rows over B * Hq
  int prefix_tiles;
  int Rl;           // rows of a sequence's partial: 64 or 128
  int start;        // first position of the group that the prefix ends in
  int pool_rows;
  int* off;         // [B + 1] first unit of each sequence's line, then the total
  float* ml;        // [slot][128][2]
  float* po;        // prefix slots [Dv / 4][128][4], then sequence slots [Dv / 4][Rl][4]
  int slots_pre;
};

__device__ __forceinline__ int seq_len(const PrefixAttnParams& a, int b) {
  const int L = __ldg(&a.lay.seq_lens[b]);
  return L < 0 ? 0 : min(L, a.lay.max_len);  // the bound that the host counted with
}

// 1 where the rows of a line may have no more than kShort positions: its
// tiles are half as long, and P is kept as hi + lo.
__host__ __device__ __forceinline__ int is_short(int n) { return n <= kShort; }

// Tiles of n positions; of half the length in a short line.
__host__ __device__ __forceinline__ int tiles_of(int n, int brief) {
  return (int)(((unsigned)n + (kTile >> brief) - 1) >> (8 - brief));
}
static_assert(kTile == 256, "tiles_of");

// The split counts in units: kTileUnits for a tile and kLineUnits more ahead of
// a line's first, for starting and ending it (queries in, first scores, last
// products, O out).  A tile belongs to the pair that holds its first unit.
// Measured with a line weighing 0, 1/2, 1, 3/2 and 2 tiles more: 64 sequences
// behind 65,536 positions 508, 409, 343, 355 and 356 us; 32 behind 16,384 72,
// 68, 64, 62 and 62 us; 32 short ones 23.2, 23.1, 21.6, 22.1 and 21.9 us.
constexpr int kTileUnits = 2;
constexpr int kLineUnits = 2;

// Where the tiles of a sequence of L positions begin: behind the prefix, but at
// a whole group of R positions (the few of the prefix before are masked), so
// that the height of a box depends on the page size alone.  (With tiles that
// began at the prefix's end and boxes that divided both, 8 sequences of 64
// heads behind 9,285 positions took 280 us, now 26.)
__device__ __forceinline__ int own_start(const Geo& g, int L) {
  return L >= g.a.prefix ? g.start : 0;
}

__device__ __forceinline__ int own_units(const Geo& g, int L) {
  const int own = L >= g.a.prefix ? L - g.a.prefix : L;
  const int t = min(tiles_of(L - own_start(g, L), is_short(L)), own);  // none where own is 0
  return t > 0 ? kTileUnits * t + kLineUnits : 0;
}

__device__ __forceinline__ float* slot_po(const Geo& g, int slot, bool pre) {
  return pre ? g.po + (size_t)slot * kRows * g.a.Dv
             : g.po + (size_t)g.slots_pre * kRows * g.a.Dv +
                   (size_t)(slot - g.slots_pre) * g.Rl * g.a.Dv;
}

// Pairs that take part: each has kTileUnits units or more, so every pair
// between a line's first tile and its last has one of its tiles.
__device__ __forceinline__ int pairs_used(int total, int pairs) {
  const int most = total / kTileUnits;
  return most < pairs ? most : pairs;
}

// The split, computed by each warp for itself.  Units are counted in 32 bits
// (the host refuses more).
struct Plan {
  int src;             // first sequence that has the whole prefix
  int row_lines;       // lines over the prefix
  int pre, total;      // units over the prefix, of all lines
  int mine;            // units of this pair
  int line0, unit0;    // where they start
};

// a / b for a, b >= 0, in 32 bits where they fit (a 64-bit division is a long
// instruction sequence).
__device__ __forceinline__ long long quot(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// A value that every lane has, known to be so: what the compiler cannot prove
// warp-uniform (anything loaded) costs each issued copy and MMA a loop over
// lanes on its operands.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ Plan make_plan(const Geo& g, int pair, int pairs, int lane) {
  const PrefixAttnParams& a = g.a;
  constexpr int kKept = 4;  // sequences of the first 128 in registers
  Plan p;
  int kept[kKept], sum = 0, src = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int b = lane + 32 * i;
    kept[i] = b < a.lay.batch ? seq_len(a, b) : -1;
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int L = kept[i];
    kept[i] = L >= 0 ? own_units(g, L) : 0;
    sum += kept[i];
    if (L >= a.prefix && lane + 32 * i < src) src = lane + 32 * i;
  }
  for (int b = lane + 32 * kKept; b < a.lay.batch; b += 32) {
    const int L = seq_len(a, b);
    sum += own_units(g, L);
    if (L >= a.prefix && b < src) src = b;
  }
  sum = uniform(__reduce_add_sync(0xffffffffu, sum));
  p.src = uniform(__reduce_min_sync(0xffffffffu, src));
  p.row_lines = (a.prefix > 0 && p.src != 0x7fffffff) ? g.row_tiles : 0;
  const int per = kTileUnits * g.prefix_tiles + kLineUnits;
  p.pre = p.row_lines * per;
  p.total = p.pre + sum;
  const int G = pairs_used(p.total, pairs);
  int lo = 0;
  p.mine = 0;
  if (pair < G) {  // [total pair / G, total (pair + 1) / G)
    const int q = p.total / G, r = p.total - q * G;
    lo = pair * q + pair * r / G;
    p.mine = (pair + 1) * q + (pair + 1) * r / G - lo;
  }
  p.line0 = p.unit0 = 0;
  if (p.mine > 0) {
    if (lo < p.pre) {
      p.line0 = lo / per;
      p.unit0 = lo - p.line0 * per;
    } else {
      int at = p.pre;
      auto find = [&](int b0, int n) {
        const int end = at + warp_scan(n, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, end > lo);
        if (hit) {
          const int l = __ffs(hit) - 1;
          p.line0 = p.row_lines + b0 + l;
          p.unit0 = lo - __shfl_sync(0xffffffffu, end - n, l);
          return true;
        }
        at = __shfl_sync(0xffffffffu, end, 31);
        return false;
      };
      bool found = false;
#pragma unroll
      for (int i = 0; i < kKept; ++i)
        if (!found) found = find(32 * i, kept[i]);
      for (int b0 = 32 * kKept; b0 < a.lay.batch && !found; b0 += 32)
        found = find(b0, b0 + lane < a.lay.batch ? own_units(g, seq_len(a, b0 + lane)) : 0);
      p.line0 = uniform(p.line0);
      p.unit0 = uniform(p.unit0);
    }
  }
  return p;
}

// The tiles of one pair, line by line: t in [first_t, t1) of `line`.
struct Tiles {
  int line, t, t1, first_t;
  int row0, rows;    // rows of the line
  int trow;          // row of the block table
  int p0, p1;        // positions of the line
  int skip;          // the first of them are the prefix's
  int brief;         // is_short
  int left;          // units of this pair behind this line
  bool ok;

  // first tile that begins at unit v of a line or behind it
  static __device__ __forceinline__ int tile_at(int v) {
    return v > kLineUnits ? (v - kLineUnits + kTileUnits - 1) / kTileUnits : 0;
  }
  // units [v, ...) of the line; false if this pair has no tile of them
  __device__ bool load(const Geo& g, const Plan& p, int v) {
    if (line < p.row_lines) {
      row0 = line * kRows;
      const int n = g.a.lay.batch * g.a.Hq - row0;
      rows = n < kRows ? n : kRows;
      trow = p.src;
      p0 = skip = 0;
      p1 = g.a.prefix;  // (its rows have as many positions, or more)
    } else {
      trow = line - p.row_lines;
      row0 = trow * g.a.Hq;
      rows = g.a.Hq;
      p1 = uniform(seq_len(g.a, trow));
      p0 = own_start(g, p1);
      skip = p1 >= g.a.prefix ? g.a.prefix - p0 : 0;
    }
    brief = is_short(p1);
    const int T = min(tiles_of(p1 - p0, brief), p1 - p0 - skip);
    const int n = T > 0 ? kTileUnits * T + kLineUnits - v : 0;
    const int take = n < left ? n : left;
    left -= take;
    t = first_t = tile_at(v);
    t1 = tile_at(v + take);
    return t1 > t;
  }
  __device__ void next_line(const Geo& g, const Plan& p) {
    ok = false;
    while (left > 0 && !ok) {
      ++line;
      ok = load(g, p, 0);
    }
  }
  __device__ void init(const Geo& g, const Plan& p) {
    line = p.line0;
    left = p.mine;
    t = t1 = first_t = brief = 0;
    ok = left > 0 && load(g, p, p.unit0);
    if (!ok) next_line(g, p);
  }
  __device__ __forceinline__ void next(const Geo& g, const Plan& p) {
    if (++t >= t1) next_line(g, p);
  }
  __device__ __forceinline__ bool first() const { return t == first_t; }
  __device__ __forceinline__ bool last() const { return t + 1 == t1; }
  __device__ __forceinline__ bool pre(const Plan& p) const { return line < p.row_lines; }
  __device__ __forceinline__ int pos() const { return p0 + t * (kTile >> brief); }
  __device__ __forceinline__ int keys() const {
    const int n = p1 - pos();
    return min(n, kTile >> brief);
  }
  // positions of the tile ahead of the line's own (less than a group)
  __device__ __forceinline__ int ahead() const { return t == 0 ? skip : 0; }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}

// Address, in the cluster's shared memory, of CTA 0's copy of a local object.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}

// The issuing roles run as whole warps on warp-uniform values and one elected
// lane (always the same) issues: descriptors and coordinates then stay in
// uniform registers.  Issued from a single-lane branch each MMA cost ~140
// cycles of register moves, twice its time on the tensor cores.

// TMA box (of one 64-column block, of several) into this CTA's shared memory; its
// bytes count on `bar` of CTA 0.
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_pair3(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                          int y, int z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on this barrier of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}\n" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void expect_tx_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void fail(Smem& sm, int* status) {
  sm.abort = 1;
  flag_status(status, DSA_STATUS_TIMEOUT);
}

// Position in a ring of n stages.
template <int n>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++s == n) {
      s = 0;
      phase ^= 1;
    }
  }
};

// Physical row of group i of a tile: `none` (a row outside the pool, which
// loads as zeros) past the tile's end, -1 behind a bad block id.
__device__ __forceinline__ int group_row(const Geo& g, const Tiles& t, int i, int lgR) {
  if ((i << lgR) >= t.keys()) return g.pool_rows;
  const unsigned p = (unsigned)t.pos() + (unsigned)(i << lgR);
  const unsigned q = g.lgbs >= 0 ? p >> g.lgbs : p / (unsigned)g.a.lay.bs;
  const int page = __ldg(&g.a.lay.bt[(long long)t.trow * g.a.lay.maxb + q]);
  if (page < 0 || page >= g.a.lay.nb) return -1;
  return page * g.a.lay.bs + (int)(p - q * (unsigned)g.a.lay.bs);
}

__global__ void __launch_bounds__(kThreads, 1)
    k_prefix_attn(const __grid_constant__ Maps maps, const __grid_constant__ Geo g) {
  extern __shared__ uint8_t smraw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  const PrefixAttnParams& a = g.a;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // warp-uniform
  const int rank = (int)cluster_rank();
  launch_dependents();

  if (threadIdx.x == 0) {
    sm.abort = 0;
    sm.fills[0] = sm.fills[1] = sm.fills[2] = 0;
    for (int i = 0; i < kStagesK; ++i) {
      mbar_init(&sm.fullk[i], 1);
      mbar_init(&sm.emptyk[i], 1);
    }
    for (int i = 0; i < kStagesV; ++i) {
      mbar_init(&sm.fullv[i], 1);
      mbar_init(&sm.emptyv[i], 1);
    }
    mbar_init(&sm.qfull, 1);
    mbar_init(&sm.qempty, 1);
    mbar_init(&sm.sfull[0], 1);
    mbar_init(&sm.sfull[1], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.sfree[i], 8);   // one arrival per softmax warp of both CTAs
      mbar_init(&sm.oready[i], 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sm.pfull[i], 4);  // of the warps that write the chunk
    mbar_init(&sm.pdone[0], 1);
    mbar_init(&sm.pdone[1], 1);
    mbar_init(&sm.pvdone, 1);
    for (int i = 0; i < kTabs; ++i) mbar_init(&sm.vfull[i], 1);
    mbar_init(&sm.smsync[0], 2);
    mbar_init(&sm.smsync[1], 2);
    mbar_init(&sm.done, 2);
    fence_mbar_init();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v[31 - __clz(g.R)]);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
  grid_dependency_wait();  // everything below reads inputs of earlier kernels

  const int pair = blockIdx.x >> 1;
  const Plan plan = make_plan(g, pair, gridDim.x >> 1, lane);
  if (blockIdx.x == 1 && warp == 0) {
    // for the merge: first unit of every sequence's line
    int at = plan.pre;
    for (int b0 = 0; b0 < a.lay.batch; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < a.lay.batch) {
        const int L = seq_len(a, b);
        n = own_units(g, L);
        if (__ldg(&a.lay.seq_lens[b]) > L) flag_status(a.status, DSA_STATUS_BAD_LENGTH);
      }
      const int end = at + warp_scan(n, lane);
      if (b < a.lay.batch) g.off[b] = end - n;
      at = __shfl_sync(0xffffffffu, end, 31);
    }
    if (lane == 0) g.off[a.lay.batch] = plan.total;
  }
  const int Cq = (a.Dqk + 63) / 64;
  const int cols = (a.Dv + 127) / 128;     // 128-column halves of V instructions
  const int ninst = (cols + 1) / 2;        // instructions of 256 columns; the last may have 128

  const int R = g.R, per = kTile / R;  // groups per tile
  const int lgR = 31 - __clz(R);
  const int none = g.pool_rows;

  if (warp == 4) {
    // ---------------------------------------------------------- K producer --
    // Queries, keys, and which positions of each tile are usable.
    Tiles t;
    t.init(g, plan);
    Ring<kStagesK> r;
    int u = 0, nq = 0;
    bool ok = true;
    const uint32_t qbar = leader_addr(&sm.qfull), fbar = leader_addr(&sm.fullk[0]);
    const uint32_t ring = smem_u32(sm.ringk[0]);
    const uint32_t empty = smem_u32(&sm.emptyk[0]), full = smem_u32(&sm.fullk[0]);
    int* tab = sm.tab[0];
    int ahead = t.ok && lane < per ? group_row(g, t, lane, lgR) : none;  // of the next tile
    while (t.ok) {
      if (t.first()) {  // the line's queries, once the previous line's last S is done
        if (nq > 0 && !pair_wait(smem_u32(&sm.qempty), (nq - 1) & 1, &sm.abort)) { ok = false; break; }
        // (a line of at most 64 rows: both CTAs take the same rows)
        const int q0 = t.row0 + (t.rows > 64 ? 64 * rank : 0);
        if (rank == 0) expect_tx_elected(smem_u32(&sm.qfull), 2 * Cq * 64 * 128);
        for (int c = 0; c < Cq; ++c)
          tma_pair(smem_u32(sm.q[0]) + c * 8192, &maps.q, qbar, 64 * c, q0);
        ++nq;
        if (lane == 0) sm.fills[2] = nq;
      }
      bool bad = lane < per && ahead < 0;
      if (lane < per) tab[lane] = ahead;
      for (int i = lane + 32; i < per; i += 32) {
        const int row = group_row(g, t, i, lgR);
        bad |= row < 0;
        tab[i] = row;
      }
      if (bad) flag_status(a.status, DSA_STATUS_BAD_BLOCK);
      __syncwarp();
      const int keys = t.keys(), skip = t.ahead(), brief = t.brief;
      const int nb = 128 >> brief >> lgR;  // boxes per stage
      const uint32_t bytes = kStageBytes >> brief;
      const int* mytab = tab + rank * nb;
      {
        // Usable positions.  The slot was tile u - 8's: K of tile u - 5 at
        // the latest has left the ring of 4 stages, so S of it was issued, so
        // the softmax of tile u - 7 is done.
        const int slot = u % kTabs;
        uint32_t word = 0;
        if (lane < kTile / 32) {
          const int k0 = 32 * lane;
          if (R >= 32) {
            word = tab[k0 >> lgR] >= 0 ? 0xffffffffu : 0u;
          } else {
            for (int i = 0; i < 32; i += R)
              if (tab[(k0 + i) >> lgR] >= 0) word |= ((1u << R) - 1u) << i;
          }
          const int n = keys - k0;
          if (n < 32) word &= n <= 0 ? 0u : (1u << n) - 1u;
          const int no = skip - k0;
          if (no > 0) word &= no >= 32 ? 0u : ~0u << no;
          sm.mask[slot][lane] = word;
        }
        const bool whole = __all_sync(0xffffffffu, lane >= kTile / 32 >> brief || word == 0xffffffffu);
        __syncwarp();  // lane 0's arrival releases every lane's word (a vote orders no memory)
        if (lane == 0) {
          sm.whole[slot] = whole;
          mbar_arrive(&sm.vfull[slot]);
        }
      }
      t.next(g, plan);
      if (t.ok && lane < per) ahead = group_row(g, t, lane, lgR);
      const int krows = lane < nb && mytab[lane] >= 0 ? mytab[lane] : none;
      const int r0 = uniform(mytab[0] >= 0 ? mytab[0] : none);  // a stage of two boxes
      const int r1 = uniform(nb < 2 || mytab[1] < 0 ? none : mytab[1]);
      for (int c = 0; c < Cq; ++c) {
        if (!pair_wait(empty + 8 * r.s, r.phase ^ 1, &sm.abort)) { ok = false; break; }
        if (rank == 0) expect_tx_elected(full + 8 * r.s, 2 * bytes);
        const uint32_t dst = ring + r.s * kStageBytes, bar = fbar + 8 * r.s;
        if (nb == 2) {
          tma_pair(dst, &maps.k, bar, 64 * c, r0);
          tma_pair(dst + R * 128, &maps.k, bar, 64 * c, r1);
        } else {
          uint32_t to = dst;
          for (int i0 = 0; i0 < nb; i0 += 32) {
            int row = krows;
            if (i0 > 0) row = mytab[i0 + lane] >= 0 ? mytab[i0 + lane] : none;
            const int n = nb - i0 < 32 ? nb - i0 : 32;
#pragma unroll 4
            for (int i = 0; i < n; ++i, to += R * 128)
              tma_pair(to, &maps.k, bar, 64 * c, __shfl_sync(0xffffffffu, row, i));
          }
        }
        r.step();
        if (lane == 0) sm.fills[0] = u * Cq + c + 1;
      }
      if (!ok) break;
      ++u;
      __syncwarp();
    }
    if (!ok && lane == 0) fail(sm, a.status);
  } else if (warp == 6) {
    // ---------------------------------------------------------- V producer --
    Tiles t;
    t.init(g, plan);
    Ring<kStagesV> r;
    int n_fills = 0;
    bool ok = true;
    const uint32_t fbar = leader_addr(&sm.fullv[0]);
    const uint32_t ring = smem_u32(sm.ringv[0]);
    const uint32_t empty = smem_u32(&sm.emptyv[0]), full = smem_u32(&sm.fullv[0]);
    const int nb = 64 >> lgR;
    const CUtensorMap* vmap = &maps.v[lgR];
    const uint32_t bstep = g.Rv * 128;  // to the next block of a group
    int* tab = sm.tab[1];
    int ahead = t.ok && lane < per ? group_row(g, t, lane, lgR) : none;
    while (t.ok) {
      const int keys = t.keys(), skip = t.ahead(), brief = t.brief;
      const int nkk = (keys + 63) >> 6;
      // the tile's groups, a lane each (more than 32, in pages of odd sizes, in
      // shared memory), and those that the line begins or ends in
      unsigned cuts = 0xffffffffu;
      const int rows = ahead >= 0 ? ahead : none;
      if (per <= 32) {
        const int n = keys - (lane << lgR);
        cuts = __ballot_sync(0xffffffffu, lane < per && rows != none && (n < R || (lane == 0 && skip > 0)));
      } else {
        for (int i = lane; i < per; i += 32) {
          const int row = i < 32 ? ahead : group_row(g, t, i, lgR);
          tab[i] = row >= 0 ? row : none;
        }
        __syncwarp();
      }
      t.next(g, plan);
      if (t.ok && lane < per) ahead = group_row(g, t, lane, lgR);
      for (int j = 0; j < 4 && ok; ++j) {
        // the O issuer's order; in a short line 0 and 1
        const int kk = ((j >> 1) | ((j & 1) << 1)) >> brief;
        if (kk >= nkk || j >= 4 >> brief) continue;
        const int g0 = kk * nb;
        const bool cut = per > 32 || (cuts >> g0 & ((1u << nb) - 1u)) != 0;
        for (int i = 0; i < ninst; ++i) {
          const int blocks = (i < ninst - 1 || cols % 2 == 0) ? 2 : 1;  // 64-column blocks per CTA
          const int x0 = 256 * i + 64 * blocks * rank;
          if (!pair_wait(empty + 8 * r.s, r.phase ^ 1, &sm.abort)) { ok = false; break; }
          if (rank == 0) expect_tx_elected(full + 8 * r.s, 2 * blocks * 64 * 128);
          const uint32_t bar = fbar + 8 * r.s;
          uint32_t dst = ring + r.s * kStageBytes;
          const uint32_t gstep = R * 128 * (R >= 16 ? blocks : 1);
          if (!cut && g.wide) {
            const int z = x0 >> 6;
#pragma unroll 1
            for (int gi = 0; gi < nb; ++gi, dst += gstep)
              tma_pair3(dst, &maps.v2, bar, 0, __shfl_sync(0xffffffffu, rows, g0 + gi), z);
          } else if (!cut) {
#pragma unroll 1
            for (int gi = 0; gi < nb; ++gi, dst += gstep) {
              const int row = __shfl_sync(0xffffffffu, rows, g0 + gi);
              tma_pair(dst, vmap, bar, x0, row);
              if (blocks == 2) tma_pair(dst + bstep, vmap, bar, x0 + 64, row);
            }
          } else {
            for (int gi = 0; gi < nb; ++gi, dst += gstep) {
              const int row = per <= 32 ? __shfl_sync(0xffffffffu, rows, g0 + gi) : uniform(tab[g0 + gi]);
              const int k0 = (g0 + gi) << lgR, n = keys - k0;  // cached positions of the group
              const int n0 = k0 == 0 ? skip : 0, n1 = n < R ? n : R;
              for (int blk = 0; blk < blocks; ++blk) {
                const int x = x0 + 64 * blk;
                const uint32_t d = dst + bstep * blk;
                if (row == none || (n >= R && n0 == 0)) {
                  tma_pair(d, vmap, bar, x, row);
                  continue;
                }
                // zeros, the line's rows, zeros, in boxes of powers of two
                int at = 0;
                if (n0 > 0)
                  for (int e = lgR - 1; e >= 0; --e)
                    if (n0 >> e & 1) {
                      tma_pair(d + at * 128, &maps.v[e], bar, x, none);
                      at += 1 << e;
                    }
                for (int e = lgR - 1; e >= 0; --e)
                  if ((n1 - n0) >> e & 1) {
                    tma_pair(d + at * 128, &maps.v[e], bar, x, row + at);
                    at += 1 << e;
                  }
                for (int e = lgR - 1; e >= 0; --e)
                  if ((R - n1) >> e & 1) {
                    tma_pair(d + at * 128, &maps.v[e], bar, x, none);
                    at += 1 << e;
                  }
              }
            }
          }
          r.step();
          ++n_fills;
        }
      }
      if (lane == 0) sm.fills[1] = n_fills;
      if (!ok) break;
      __syncwarp();
    }
    if (!ok && lane == 0) fail(sm, a.status);
  } else if (warp == 5) {
    // ------------------------------------------------------------ S issuer --
    // (With one warp issuing S and O in turn a tile took 7,700 cycles; with
    // two and the weights handed over whole 6,800; with the chunks 5,700.)
    if (rank == 0) {
      Tiles t;
      t.init(g, plan);
      Ring<kStagesK> r;
      int u = 0, nq = 0;
      bool ok = true;
      const uint32_t empty = smem_u32(&sm.emptyk[0]), full = smem_u32(&sm.fullk[0]);
      // descriptors: the address field counts 16 bytes; a step of 16 dims or
      // positions is 32 bytes of a K-major operand, 2048 of V
      const uint64_t dq = smem_desc(smem_u32(sm.q[0]), 16, 1024, kSwizzle128B);
      const uint64_t dk = smem_desc(smem_u32(sm.ringk[0]), 16, 1024, kSwizzle128B);
      while (t.ok && ok) {
        if (t.first()) {
          if (!pair_wait(smem_u32(&sm.qfull), nq & 1, &sm.abort)) { ok = false; break; }
          ++nq;
        }
        // the softmax of tile u - 2 has read this S buffer
        if (u >= 2 && !pair_wait(smem_u32(&sm.sfree[u & 1]), ((u >> 1) & 1) ^ 1, &sm.abort)) {
          ok = false;
          break;
        }
        const uint32_t d = tbase + kColS + 128 * (u & 1);
        const uint32_t id = t.brief ? instr_desc(kRows, 128, 1, 1, 0, 0) : instr_desc(kRows, 256, 1, 1, 0, 0);
        uint64_t qa = dq;
        for (int c = 0; c < Cq; ++c, qa += 512) {
          if (!pair_wait(full + 8 * r.s, r.phase, &sm.abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t kb = dk + 1024 * r.s;
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_pair(d, qa + 2 * k, kb + 2 * k, id, c + k);
          commit_pair(empty + 8 * r.s);
          r.step();
        }
        if (!ok) break;
        commit_pair(smem_u32(&sm.sfull[u & 1]));
        if (t.last()) commit_pair(smem_u32(&sm.qempty));
        ++u;
        t.next(g, plan);
      }
      if (!ok && lane == 0) fail(sm, a.status);
      commit_pair(smem_u32(&sm.done));
    }
  } else if (warp == 7) {
    // ------------------------------------------------------------ O issuer --
    if (rank == 0) {
      Tiles t;
      t.init(g, plan);
      Ring<kStagesV> r;
      int u = 0;
      bool ok = true;
      const uint32_t empty = smem_u32(&sm.emptyv[0]), full = smem_u32(&sm.fullv[0]);
      const uint64_t dp = smem_desc(smem_u32(sm.p[0]), 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(smem_u32(sm.ringv[0]), g.Rv * 128, 1024, kSwizzle128B);
      // the second, third and fourth 16 positions of a chunk of two blocks
      const int lgs = 27 - __clz(g.Rv), in = (1 << lgs) - 1;
      const int o1 = (1 >> lgs) * 16 * g.Rv + (1 & in) * 128;
      const int o2 = (2 >> lgs) * 16 * g.Rv + (2 & in) * 128;
      const int o3 = (3 >> lgs) * 16 * g.Rv + (3 & in) * 128;
      while (t.ok && ok) {
        const int nkk = (t.keys() + 63) >> 6;
        const int add0 = t.first() ? 0 : 1, brief = t.brief;
        t.next(g, plan);
        // O is rescaled, or read out for the line before
        if (!pair_wait(smem_u32(&sm.oready[u & 1]), (u >> 1) & 1, &sm.abort)) { ok = false; break; }
        // the weights in chunks of 64 positions, the two halves' in turn, as
        // the softmax finishes them; a chunk is free for the next tile's
        // weights as soon as both products of it are done
        for (int j = 0; j < 4 && ok; ++j) {
          const int kk = (j >> 1) | ((j & 1) << 1);  // 0, 2, 1, 3
          if (!pair_wait(smem_u32(&sm.pfull[kk]), u & 1, &sm.abort)) { ok = false; break; }
          // a short line: chunk kk and what it leaves, chunk kk + 1, on the same V
          if (brief && !pair_wait(smem_u32(&sm.pfull[kk | 1]), u & 1, &sm.abort)) { ok = false; break; }
          if (kk >> brief < nkk && j < 4 >> brief) {
            const uint64_t pa = dp + 512 * kk;
            for (int i = 0; i < ninst; ++i) {
              const int blocks = (i < ninst - 1 || cols % 2 == 0) ? 2 : 1;
              const uint32_t id = instr_desc(kRows, 128 * blocks, 1, 1, 0, 1);
              const uint32_t d = tbase + kColO + 128 * i;
              if (!pair_wait(full + 8 * r.s, r.phase, &sm.abort)) { ok = false; break; }
              tc_fence_after();
              const uint64_t vb = dv + 1024 * r.s;
              const bool two = blocks == 2;
              mma_pair(d, pa, vb, id, add0 + j);
              mma_pair(d, pa + 2, vb + (two ? o1 : 128), id, 1);
              mma_pair(d, pa + 4, vb + (two ? o2 : 256), id, 1);
              mma_pair(d, pa + 6, vb + (two ? o3 : 384), id, 1);
              if (brief) {
                mma_pair(d, pa + 512, vb, id, 1);
                mma_pair(d, pa + 514, vb + (two ? o1 : 128), id, 1);
                mma_pair(d, pa + 516, vb + (two ? o2 : 256), id, 1);
                mma_pair(d, pa + 518, vb + (two ? o3 : 384), id, 1);
              }
              commit_pair(empty + 8 * r.s);
              r.step();
            }
            if (!ok) break;
          }
          if (j < 2) commit_pair(smem_u32(&sm.pdone[j]));
        }
        if (!ok) break;
        commit_pair(smem_u32(&sm.pvdone));
        ++u;
      }
      if (!ok && lane == 0) fail(sm, a.status);
      commit_pair(smem_u32(&sm.done));
    }
  } else {
    // -------------------------------------------------------------- softmax --
    const int row = (warp & 1) * 32 + lane;   // of this CTA's 64
    const int half = warp >> 1;               // half of the tile's positions, of O's columns
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float c = a.scale_log2;
    const uint32_t pbar = leader_addr(&sm.pfull[2 * half]), fbar = leader_addr(&sm.sfree[0]);
    const uint32_t obar = leader_addr(&sm.oready[0]);
    Tiles t;
    t.init(g, plan);
    int u = 0;
    uint32_t sp = 0;
    bool ok = true;
    float m = -INFINITY, l = 0.0f;
    while (t.ok && ok) {
      if (t.first()) {
        m = -INFINITY;
        l = 0.0f;
      }
      if (!pair_wait(smem_u32(&sm.sfull[u & 1]), (u >> 1) & 1, &sm.abort)) { ok = false; break; }
      tc_fence_after();
      // Two passes over S in TMEM, 32 columns at a time: the maximum while
      // the tensor cores work on O of the previous tile, then the weights
      // straight into P.  (One pass with the thread's 128 scores in
      // registers took 1 % longer, and 225 registers.)
      const uint32_t ta = tbase + lanes + kColS + 128 * (u & 1);
      if (!pair_wait(smem_u32(&sm.vfull[u % kTabs]), (u / kTabs) & 1, &sm.abort)) { ok = false; break; }
      const bool whole = sm.whole[u % kTabs] != 0;
      const int brief = t.brief, nq = 4 >> brief;  // 32 columns of S at a time
      const uint32_t* mask = &sm.mask[u % kTabs][nq * half];
      float mt = -INFINITY;
#pragma unroll 1
      for (int q = 0; q < nq; ++q) {
        uint32_t z[32];
        tmem_ld_32cols(ta + 32 * q, z);
        tmem_wait_ld();
        if (!whole) {
          const uint32_t w = mask[q];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((w >> i) & 1u)) z[i] = 0xff800000u;
        }
        float m4[4] = {mt, __uint_as_float(z[0]), __uint_as_float(z[1]), __uint_as_float(z[2])};
#pragma unroll
        for (int i = 3; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(z[i]));
        mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
      sm.redm[u & 1][half][row] = mt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.smsync[warp & 1]);
      if (!pair_wait(smem_u32(&sm.smsync[warp & 1]), sp, &sm.abort)) { ok = false; break; }
      sp ^= 1;
      mt = fmaxf(mt, sm.redm[u & 1][half ^ 1][row]) * c;
      float f = 1.0f;
      bool resc = false;
      if (mt > m + kRescaleLog2 || (m == -INFINITY && mt > -INFINITY)) {
        if (m > -INFINITY) {
          f = exp2f(m - mt);
          resc = true;
        }
        m = mt;
      }
      const float mm = m == -INFINITY ? 0.0f : m;
      if (!t.first() && __any_sync(0xffffffffu, resc)) {
        // O of the tiles before is complete (u > 0: not the first tile)
        if (!pair_wait(smem_u32(&sm.pvdone), (u - 1) & 1, &sm.abort)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < 2 * cols; ++q) {
          uint32_t v[32];
          tmem_ld_32cols(tbase + lanes + kColO + 32 * q, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
          tmem_st_32cols(tbase + lanes + kColO + 32 * q, v);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(obar + 8 * (u & 1));
      float ls[2] = {l * f, 0.0f};
      // 32 columns of scores, the unusable ones -inf
      auto scores = [&](int q, uint32_t (&z)[32]) {
        tmem_ld_32cols(ta + 32 * q, z);
        tmem_wait_ld();
        if (!whole) {
          const uint32_t w = mask[q];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((w >> i) & 1u)) z[i] = 0xff800000u;
        }
      };
      if (brief) {
        // A short line's half has 64 columns: their weights' bf16 part goes to
        // the half's first chunk of P, what that leaves to the second.
        if (u > 0 && !pair_wait(smem_u32(&sm.pvdone), (u - 1) & 1, &sm.abort)) { ok = false; break; }
        uint8_t* dst = sm.p[2 * half] + row * 128;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t z[32];
          scores(q, z);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e0 = ex2_approx(fmaf(__uint_as_float(z[8 * k + 2 * i]), c, -mm));
              const float e1 = ex2_approx(fmaf(__uint_as_float(z[8 * k + 2 * i + 1]), c, -mm));
              ls[0] += e0;
              ls[1] += e1;
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(e0, e1);
              const float2 h = __bfloat1622float2(h2);
              const __nv_bfloat162 l2 = __floats2bfloat162_rn(e0 - h.x, e1 - h.y);
              hi[i] = *reinterpret_cast<const uint32_t*>(&h2);
              lo[i] = *reinterpret_cast<const uint32_t*>(&l2);
            }
            uint8_t* to = dst + (((4 * q + k) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(to + sizeof(sm.p[0])) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_cluster(pbar);
          arrive_cluster(pbar + 8);
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t z[32];
          scores(q, z);
          // The previous tile's products have read this chunk of P: the
          // half's first chunk by its own barrier, the second by the whole
          // tile's, which every tile waits for here once (a phase of pvdone
          // left out would make a later wait test the wrong one).
          if ((q & 1) == 0 && u > 0 &&
              !pair_wait(q == 0 ? smem_u32(&sm.pdone[half]) : smem_u32(&sm.pvdone), (u - 1) & 1,
                         &sm.abort)) {
            ok = false;
            break;
          }
          uint8_t* dst = sm.p[2 * half + (q >> 1)] + row * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // eight weights, 16 bytes of the row's 128-byte line
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e0 = ex2_approx(fmaf(__uint_as_float(z[8 * k + 2 * i]), c, -mm));
              const float e1 = ex2_approx(fmaf(__uint_as_float(z[8 * k + 2 * i + 1]), c, -mm));
              ls[0] += e0;
              ls[1] += e1;
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
              pk[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            *reinterpret_cast<uint4*>(dst + (((4 * (q & 1) + k) ^ (row & 7)) << 4)) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          if (q & 1) {  // a chunk is written
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(pbar + 8 * (q >> 1));
          }
        }
      }
      if (!ok) break;
      l = ls[0] + ls[1];
      __syncwarp();
      if (lane == 0) arrive_cluster(fbar + 8 * (u & 1));
      if (t.last()) {
        // this pair's partial of the line: O out of TMEM, unnormalised
        if (!pair_wait(smem_u32(&sm.pvdone), u & 1, &sm.abort)) { ok = false; break; }
        tc_fence_after();
        const bool pre = t.pre(plan);
        const int slot = pre ? pair + t.line : g.slots_pre + pair + t.trow;
        const int Rw = pre ? kRows : g.Rl;
        // A line of at most 64 rows is in both CTAs: each writes half of its
        // columns (one SM stores ~30 bytes a cycle, 4,400 cycles for all).
        const bool twice = t.rows <= 64;
        const int r = twice ? row : 64 * rank + row;
        const int qb = twice ? rank * cols : 0, qe = twice ? qb + cols : 2 * cols;
        float4* po = reinterpret_cast<float4*>(slot_po(g, slot, pre)) + r;
#pragma unroll 1
        for (int q0 = qb; q0 < qe; q0 += 2) {
          uint32_t v[2][32];
          tmem_ld_32cols(tbase + lanes + kColO + 32 * q0, v[0]);
          if (q0 + 1 < qe) tmem_ld_32cols(tbase + lanes + kColO + 32 * q0 + 32, v[1]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int q = q0 + e, i = q >> 2;
            const int n2 = (i < ninst - 1 || cols % 2 == 0) ? 128 : 64;  // columns per half
            const int dv = 256 * i + n2 * half + 32 * (q & 3);
            float4* dst = po + (size_t)(dv / 4) * Rw;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (q < qe && dv + 4 * j < a.Dv)
                dst[j * Rw] = make_float4(__uint_as_float(v[e][4 * j]), __uint_as_float(v[e][4 * j + 1]),
                                          __uint_as_float(v[e][4 * j + 2]),
                                          __uint_as_float(v[e][4 * j + 3]));
          }
        }
        tc_fence_before();
        // the two halves' sums; the slot of redm is the next tile's, whose
        // own exchange comes after this one
        sm.redm[(u + 1) & 1][half][row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.smsync[warp & 1]);
        if (!pair_wait(smem_u32(&sm.smsync[warp & 1]), sp, &sm.abort)) { ok = false; break; }
        sp ^= 1;
        if (half == 0 && !(twice && rank == 1))
          reinterpret_cast<float2*>(g.ml)[(size_t)slot * kRows + r] =
              make_float2(m, l + sm.redm[(u + 1) & 1][1][row]);
        // nobody writes redm[(u + 1) & 1] again before this read is done
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.smsync[warp & 1]);
        if (!pair_wait(smem_u32(&sm.smsync[warp & 1]), sp, &sm.abort)) { ok = false; break; }
        sp ^= 1;
      }
      ++u;
      t.next(g, plan);
    }
    if (!ok && lane == 0) fail(sm, a.status);
  }

  __syncthreads();
  if (warp == 0) {
    int never = 0;
    // MMAs of the pair done; after a failure also the copies in flight
    pair_wait(smem_u32(&sm.done), 0, &never, 100000000ull);
    if (sm.abort && rank == 0) {
      for (int i = 0; i < kStagesK; ++i) {
        const int n = (sm.fills[0] - i + kStagesK - 1) / kStagesK;  // fills of this stage
        if (n > 0) pair_wait(smem_u32(&sm.fullk[i]), (n - 1) & 1, &never, 10000000ull);
      }
      for (int i = 0; i < kStagesV; ++i) {
        const int n = (sm.fills[1] - i + kStagesV - 1) / kStagesV;
        if (n > 0) pair_wait(smem_u32(&sm.fullv[i]), (n - 1) & 1, &never, 10000000ull);
      }
      if (sm.fills[2] > 0) pair_wait(smem_u32(&sm.qfull), (sm.fills[2] - 1) & 1, &never, 10000000ull);
    } else if (sm.abort) {
      // CTA 1's copies count on CTA 0's barriers; its own never completes, so
      // this gives them a millisecond
      pair_wait(smem_u32(&sm.qfull), 0, &never, 1000000ull);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no arrival is on its way to a CTA that has left
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// The join of each row's partials, in two shapes.  Both take a lane per row
// (partials are stored with rows innermost, so a warp reads 512 contiguous
// bytes), turn the finished block in shared memory and write it row by row.
constexpr int kMergeThreads = 256;

// Where the partials of row h of sequence b are: prefix slots p0 .. p0 + np - 1
// (row prow), sequence slots s0 .. s0 + ns - 1 (row h).
struct RowParts {
  int p0 = 0, np = 0, s0 = 0, ns = 0, prow = 0;
  __device__ RowParts(const Geo& g, int pairs, int b, int h) {
    const PrefixAttnParams& a = g.a;
    const long long total = __ldcg(&g.off[a.lay.batch]), o0 = __ldcg(&g.off[b]),
                    o1 = __ldcg(&g.off[b + 1]), pre = __ldcg(&g.off[0]);
    const int L = seq_len(a, b);
    const int G = pairs_used((int)total, pairs);
    if (h >= a.Hq) return;
    // unit x is pair ((x + 1) G - 1) / total's; a tile is its first unit's
    if (pre > 0 && L >= a.prefix) {
      const int r = b * a.Hq + h, line = r / kRows;
      prow = r - line * kRows;
      const long long x = (long long)line * (kTileUnits * g.prefix_tiles + kLineUnits) + kLineUnits;
      const int c0 = (int)quot((x + 1) * G - 1, total);
      const int c1 = (int)quot((x + kTileUnits * (g.prefix_tiles - 1) + 1) * G - 1, total);
      p0 = c0 + line;
      np = c1 - c0 + 1;
    }
    if (o1 > o0) {
      const int c0 = (int)quot((o0 + kLineUnits + 1) * G - 1, total);
      const int c1 = (int)quot((o1 - kTileUnits + 1) * G - 1, total);
      s0 = g.slots_pre + c0 + b;
      ns = c1 - c0 + 1;
    }
  }
  __device__ int count() const { return np + ns; }
  __device__ float2 stat(const Geo& g, int i, int h) const {
    const float2* ml = reinterpret_cast<const float2*>(g.ml);
    return i < np ? __ldcg(&ml[(size_t)(p0 + i) * kRows + prow])
                  : __ldcg(&ml[(size_t)(s0 + i - np) * kRows + h]);
  }
  // the partial's float4 of columns 0..3 of the row; `step` float4 to the next
  __device__ const float4* cols(const Geo& g, int i, int h, int* step) const {
    const bool pre = i < np;
    *step = pre ? kRows : g.Rl;
    return reinterpret_cast<const float4*>(slot_po(g, pre ? p0 + i : s0 + i - np, pre)) +
           (pre ? prow : h);
  }
};

// Running (M, l, acc) with a batch of partials folded in; an empty partial (no
// usable position: l = 0) is left out.
template <int J, int kBatch>
__device__ __forceinline__ void fold(float& M, float& l, float4 (&acc)[J],
                                     const float2 (&st)[kBatch], const float4 (&x)[kBatch][J]) {
  float Mn = M;
#pragma unroll
  for (int q = 0; q < kBatch; ++q)
    if (st[q].y != 0.0f) Mn = fmaxf(Mn, st[q].x);
  const float Ms = Mn == -INFINITY ? 0.0f : Mn;
  const float f = M == -INFINITY ? 1.0f : exp2f(M - Ms);
  l *= f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    acc[j].x *= f;
    acc[j].y *= f;
    acc[j].z *= f;
    acc[j].w *= f;
  }
#pragma unroll
  for (int q = 0; q < kBatch; ++q) {
    if (st[q].y != 0.0f) {
      const float w = exp2f(st[q].x - Ms);
      l = fmaf(st[q].y, w, l);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        acc[j].x = fmaf(w, x[q][j].x, acc[j].x);
        acc[j].y = fmaf(w, x[q][j].y, acc[j].y);
        acc[j].z = fmaf(w, x[q][j].z, acc[j].z);
        acc[j].w = fmaf(w, x[q][j].w, acc[j].w);
      }
    }
  }
  M = Mn;
}

__device__ __forceinline__ uint2 pack4(const float4& v, float f) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * f, v.w * f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__device__ __forceinline__ float lse_of(float M, float l) {
  return l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

// Many rows: grid (B, groups of 32 heads, groups of 128 columns); a warp takes
// 16 columns and all partials of its rows, four in flight (32 sequences of 64
// heads: 3 us; 6 us with blocks of 32 columns, each with its own look at the
// plan).
__global__ void __launch_bounds__(kMergeThreads) k_prefix_merge(const __grid_constant__ Geo g,
                                                                int pairs) {
  constexpr int kBatch = 4;
  __shared__ uint2 tile[32][33];  // four bf16 each, padded
  const PrefixAttnParams& a = g.a;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 32 + lane;
  const int x0 = blockIdx.z * 128;
  grid_dependency_wait();
  launch_dependents();
  const RowParts rp(g, pairs, b, h);
  const int n = rp.count();
  float M = -INFINITY, l = 0.0f;
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    float2 st[kBatch];
    float4 x[kBatch][4];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + q;
      st[q] = make_float2(-INFINITY, 0.0f);
      int step = 0;
      const float4* po = nullptr;
      if (i < n) {
        st[q] = rp.stat(g, i, h);
        po = rp.cols(g, i, h, &step);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int dv = x0 + 4 * (warp + 8 * j);
        x[q][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n && dv < a.Dv) x[q][j] = __ldcg(&po[(size_t)(dv / 4) * step]);
      }
    }
    fold(M, l, acc, st, x);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < 4; ++j) tile[lane][warp + 8 * j] = pack4(acc[j], inv);
  if (a.lse && blockIdx.z == 0 && warp == 0 && h < a.Hq) a.lse[(size_t)b * a.Hq + h] = lse_of(M, l);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = warp + 8 * i;  // row; a lane writes four columns
    const int hh = blockIdx.y * 32 + r, x = x0 + 4 * lane;
    if (hh < a.Hq && x < a.Dv)
      *reinterpret_cast<uint2*>(a.out + ((size_t)b * a.Hq + hh) * a.Dv + x) = tile[r][lane];
  }
}

// Few rows, each with about as many partials as there are pairs: grid (B,
// groups of 32 heads, groups of 32 columns); the eight warps share the
// partials, all of a row's first 24 in flight at once, and are joined in
// shared memory (7 sequences, 22 partials a row: 3.3 us against 5.5 us
// with a warp on four columns of all partials, eight in flight).
__global__ void __launch_bounds__(kMergeThreads)
    k_prefix_merge_deep(const __grid_constant__ Geo g, int pairs) {
  constexpr int kBatch = 3;
  __shared__ float4 part[8][8][32];  // [warp][four columns][row]
  __shared__ float2 stat[8][32];
  __shared__ uint2 tile[32][9];
  const PrefixAttnParams& a = g.a;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 32 + lane;
  const int x0 = blockIdx.z * 32;
  grid_dependency_wait();
  launch_dependents();
  const RowParts rp(g, pairs, b, h);
  const int n = rp.count();
  float M = -INFINITY, l = 0.0f;
  float4 acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < n; i0 += 8 * kBatch) {
    float2 st[kBatch];
    float4 x[kBatch][8];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + 8 * q;
      st[q] = make_float2(-INFINITY, 0.0f);
      int step = 0;
      const float4* po = nullptr;
      if (i < n) {
        st[q] = rp.stat(g, i, h);
        po = rp.cols(g, i, h, &step);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[q][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n && x0 + 4 * j < a.Dv) x[q][j] = __ldcg(&po[(size_t)(x0 / 4 + j) * step]);
      }
    }
    fold(M, l, acc, st, x);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[warp][j][lane] = acc[j];
  stat[warp][lane] = make_float2(M, l);
  __syncthreads();
  {
    // warp w joins the eight warps' sums of columns 4 w .. 4 w + 3
    float2 st[8];
    float4 x[8][1], sum[1] = {make_float4(0.f, 0.f, 0.f, 0.f)};
    float Mj = -INFINITY, lj = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      st[q] = stat[q][lane];
      x[q][0] = part[q][warp][lane];
    }
    fold(Mj, lj, sum, st, x);
    tile[lane][warp] = pack4(sum[0], lj == 0.0f ? 0.0f : 1.0f / lj);
    if (a.lse && blockIdx.z == 0 && warp == 0 && h < a.Hq)
      a.lse[(size_t)b * a.Hq + h] = lse_of(Mj, lj);
  }
  __syncthreads();
  const int r = threadIdx.x >> 3, k = threadIdx.x & 7;  // row, four columns
  const int hh = blockIdx.y * 32 + r, x = x0 + 4 * k;
  if (hh < a.Hq && x < a.Dv)
    *reinterpret_cast<uint2*>(a.out + ((size_t)b * a.Hq + hh) * a.Dv + x) = tile[r][k];
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Layout {
  size_t off, ml, po, total;
  int row_tiles, slots_pre, slots_seq, Rl;
};

Layout ws_layout(int B, int Hq, int Dv, int prefix) {
  Layout w;
  w.row_tiles = (int)(((long long)B * Hq + kRows - 1) / kRows);
  w.Rl = Hq <= 64 ? 64 : 128;
  // a pair's partial of a line is slot pair + line: lines and pairs both only
  // grow along the tiles, so no two partials share a slot
  w.slots_pre = prefix > 0 ? kMaxPairs + w.row_tiles : 0;
  w.slots_seq = kMaxPairs + B;
  w.off = kWsHeader;
  w.ml = w.off + round256(sizeof(int) * ((size_t)B + 1));
  w.po = w.ml + round256(sizeof(float) * 2 * kRows * ((size_t)w.slots_pre + w.slots_seq));
  w.total = w.po + sizeof(float) * (size_t)Dv *
                       ((size_t)w.slots_pre * kRows + (size_t)w.slots_seq * w.Rl);
  return w;
}

}  // namespace

size_t prefix_attn_ws(int B, int Hq, int Dqk, int Dv, int prefix) {
  (void)Dqk;
  return ws_layout(B, Hq, Dv, prefix).total;
}

int launch_prefix_attn(const PrefixAttnParams& p, void* ws, cudaStream_t s) {
  Geo g{};
  g.a = p;
  const Layout w = ws_layout(p.lay.batch, p.Hq, p.Dv, p.prefix);
  char* base = reinterpret_cast<char*>(ws);
  g.off = reinterpret_cast<int*>(base + w.off);
  g.ml = reinterpret_cast<float*>(base + w.ml);
  g.po = reinterpret_cast<float*>(base + w.po);
  g.slots_pre = w.slots_pre;
  g.row_tiles = w.row_tiles;
  g.Rl = w.Rl;
  g.prefix_tiles = tiles_of(p.prefix, is_short(p.prefix));
  g.pool_rows = (int)((long long)p.lay.nb * p.lay.bs);
  int R = 64;
  while (p.lay.bs % R) R >>= 1;
  g.R = R;
  g.start = p.prefix & -R;
  g.lgbs = -1;
  for (int i = 0; i <= 10; ++i)
    if (p.lay.bs == 1 << i) g.lgbs = i;
  Maps m{};
  int rc = make_tmap_2d(&m.q, p.q, false, p.Dqk, (uint64_t)p.lay.batch * p.Hq, (uint64_t)p.Dqk * 2,
                        64, 64);
  if (!rc)
    rc = make_tmap_2d(&m.k, p.kp, false, p.Dqk, (uint64_t)g.pool_rows, (uint64_t)p.ks * 2, 64, R);
  for (int i = 0; (1 << i) <= R && !rc; ++i)
    rc = make_tmap_2d(&m.v[i], p.vp, false, p.Dv, (uint64_t)g.pool_rows, (uint64_t)p.vs * 2, 64,
                      1u << i);
  g.Rv = R >= 16 ? R : 64;  // (smaller groups would cut an MMA's positions)
  g.wide = R >= 16 && R < 64 && p.Dv % 256 == 0;
  if (!rc && g.wide)
    rc = make_tmap_blocks(&m.v2, p.vp, p.Dv, (uint64_t)g.pool_rows, (uint64_t)p.vs * 2, R, 2);
  if (rc) return rc;
  const size_t smem = sizeof(Smem) + 1024;
  rc = ensure_dynamic_smem((const void*)k_prefix_attn, (int)smem, "prefix_attn_decode");
  if (rc) return rc;
  int pairs = max_active_clusters((const void*)k_prefix_attn, kThreads, smem, 2);
  if (pairs < 1) return set_error(DSA_ERR_CUDA, "prefix_attn_decode: no cluster of two CTAs fits");
  if (pairs > kMaxPairs) pairs = kMaxPairs;
  // most tiles of a sequence's own line: of the longest, or of the longest short one
  const long long own = std::max(tiles_of(p.lay.max_len, 0),
                                 tiles_of(std::min(p.lay.max_len, kShort), 1));
  const long long bound =
      (long long)g.row_tiles * (kTileUnits * (long long)g.prefix_tiles + kLineUnits) +
      (long long)p.lay.batch * (kTileUnits * own + kLineUnits);
  if (bound > 0x7fffffffLL)
    return set_error(DSA_ERR_UNSUPPORTED, "prefix_attn_decode: rows x positions beyond 2^30 tiles");
  if (pairs > bound / kTileUnits) pairs = (int)(bound / kTileUnits);
  cudaError_t e = launch_pdl_cluster(k_prefix_attn, dim3((unsigned)(2 * pairs)), dim3(kThreads),
                                     smem, 2, s, m, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  rc = check_launch("prefix_attn_decode");
  if (rc) return rc;
  const unsigned heads = (unsigned)((p.Hq + 31) / 32);
  const long long small = (long long)p.lay.batch * heads * ((p.Dv + 31) / 32);
  if (small <= 4LL * sm_count())
    e = launch_pdl(k_prefix_merge_deep,
                   dim3((unsigned)p.lay.batch, heads, (unsigned)((p.Dv + 31) / 32)),
                   dim3(kMergeThreads), 0, s, g, pairs);
  else
    e = launch_pdl(k_prefix_merge,
                   dim3((unsigned)p.lay.batch, heads, (unsigned)((p.Dv + 127) / 128)),
                   dim3(kMergeThreads), 0, s, g, pairs);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("prefix_attn_decode merge");
}

}  // namespace dsa
