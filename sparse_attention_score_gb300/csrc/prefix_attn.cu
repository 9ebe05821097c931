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
// P is rounded to bf16 for the second product (each weight off by 2^-9 on
// average, like the output's own rounding); sums and statistics are fp32.
//
// Warp roles (192 threads): 0-3 softmax and O out of TMEM; 4 producer: TMA
// boxes of whole 64-dim chunks into a ring of 16 KB stages, in the order the
// MMAs take them, and the tile's table of physical rows; 5 TMEM owner and,
// in CTA 0 of the pair, MMA issuer.  S of the next tile is issued before O of
// this one, so the softmax runs beside the tensor cores.
//
// Boxes are R rows high, R the largest power of two (at most 64) that divides
// the page size and the prefix length: such a group of positions never
// crosses a page.  A group that the sequence ends in is staged for V in boxes
// of 8 rows and 1 row, and rows past the end, or behind a bad block id, from
// outside the pool, which TMA fills with zeros: whatever the cache holds
// there (NaN included) never meets a weight of 0.
// Every wait is bounded (DSA_STATUS_TIMEOUT, then the pair winds down).
#include "device_common.cuh"
#include "dsa_internal.cuh"
#include "sm100.cuh"

namespace dsa {

namespace {

using namespace sm100;

constexpr int kTile = 256;             // positions per tile
constexpr int kRows = 128;             // rows of a pair, 64 per CTA
constexpr int kMaxChunks = 9;          // 64-dim chunks of a query row
constexpr int kStages = 7;
constexpr int kStageBytes = 16384;
constexpr int kThreads = 224;          // softmax 0-3, producers 4 and 6, MMA 5
constexpr int kMaxPairs = 80;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;          // two S buffers of 128 columns
constexpr uint32_t kColO = 256;        // O: 128 columns per 256 dims of V
constexpr float kRescaleLog2 = 8.0f;
constexpr int kTabs = 6;               // tiles whose mask is kept (see the producer)

struct __align__(1024) Smem {
  uint8_t ring[kStages][kStageBytes];
  uint8_t q[kMaxChunks][64 * 128];
  uint8_t p[kTile / 64][64 * 128];
  int tab[2][2][kTile];                // per producer, tiles u and u + 1: physical row
                                       // of each group of R positions
  uint32_t mask[kTabs][kTile / 32];    // usable positions
  int whole[kTabs];                    // every position of the tile is usable
  uint64_t full[kStages], empty[kStages], qfull, qempty, sfull[2], pfull, pvdone;
  uint64_t vfull[kTabs], smsync[2], done;
  float redm[2][2][64];
  int units;  // stages filled, for the drain after a failure
  unsigned long long sum;
  int src, line0, tile0;
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory of k_prefix_attn");

struct Maps {
  CUtensorMap q, k, v, v8, v1;
};

struct Geo {
  PrefixAttnParams a;
  int R;            // rows per box
  int row_tiles;    // of 128 rows over B * Hq
  int prefix_tiles;
  int Rl;           // rows of a sequence's partial: 64 or 128
  long long pool_rows;
  long long* off;   // [B + 1] first tile of each sequence's line, then the total
  float* ml;        // [slot][128][2]
  float* po;        // prefix slots [Dv / 4][128][4], then sequence slots [Dv / 4][Rl][4]
  int slots_pre;
};

__device__ __forceinline__ long long seq_len(const PrefixAttnParams& a, int b) {
  long long L = __ldg(&a.lay.seq_lens[b]);
  const long long cap = (long long)a.lay.maxb * a.lay.bs;
  if (L > cap) L = cap;
  return L < 0 ? 0 : L;
}

__device__ __forceinline__ int own_tiles(const PrefixAttnParams& a, long long L) {
  const long long n = L >= a.prefix ? L - a.prefix : L;
  return (int)((n + kTile - 1) / kTile);
}

__device__ __forceinline__ float* slot_po(const Geo& g, int slot, bool pre) {
  return pre ? g.po + (size_t)slot * kRows * g.a.Dv
             : g.po + (size_t)g.slots_pre * kRows * g.a.Dv +
                   (size_t)(slot - g.slots_pre) * g.Rl * g.a.Dv;
}

// The tiles [lo, hi) of one pair, line by line.
struct Walker {
  int line;          // row tiles first, then sequences
  int t, t1;         // this pair's tiles of the line: [t, t1)
  long long left;    // tiles left in this pair, this line's included
  bool pre;
  int rows;          // rows of the line
  int row0;          // first row of the line
  int trow;          // row of the block table
  long long p0, p1;  // positions of the line
  bool ok;

  __device__ void load(const Geo& g, int row_lines, int src) {
    if (line < row_lines) {
      pre = true;
      row0 = line * kRows;
      const int n = g.a.lay.batch * g.a.Hq - row0;
      rows = n < kRows ? n : kRows;
      trow = src;
      p0 = 0;
      p1 = g.a.prefix;
    } else {
      pre = false;
      const int b = line - row_lines;
      row0 = b * g.a.Hq;
      rows = g.a.Hq;
      trow = b;
      p1 = seq_len(g.a, b);
      p0 = p1 >= g.a.prefix ? g.a.prefix : 0;
    }
    const long long n = (p1 - p0 + kTile - 1) / kTile - t;
    t1 = t + (int)(n < left ? n : left);
  }
  __device__ void init(const Geo& g, int row_lines, int src, int line0, int tile0, long long n) {
    line = line0;
    t = tile0;
    left = n;
    ok = n > 0;
    if (ok) load(g, row_lines, src);
  }
  // the next line with tiles, once t has reached t1
  __device__ void next_line(const Geo& g, int row_lines, int src, long long used) {
    left -= used;
    ok = left > 0;
    t = 0;
    while (ok) {
      ++line;
      load(g, row_lines, src);
      if (t1 > 0) break;
    }
  }
};

// One tile after the other over the lines.
struct Tiles {
  Walker w;
  int first_t;
  bool ok, first, last;
  __device__ void set() {
    ok = w.ok;
    first = ok && w.t == first_t;
    last = ok && w.t == w.t1 - 1;
  }
  __device__ void init(const Geo& g, int rl, int src, int line0, int tile0, long long n) {
    w.init(g, rl, src, line0, tile0, n);
    first_t = w.t;
    set();
  }
  __device__ void next(const Geo& g, int rl, int src) {
    if (++w.t >= w.t1) {
      w.next_line(g, rl, src, w.t1 - first_t);
      first_t = 0;
    }
    set();
  }
  __device__ long long pos() const { return w.p0 + (long long)w.t * kTile; }
  __device__ int keys() const {
    const long long n = w.p1 - pos();
    return n < kTile ? (int)n : kTile;
  }
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

// mbar_wait of a whole warp on a barrier that the pair's other CTA may arrive
// on.  (Default semantics: what crosses CTAs is ordered by the async proxy's
// own completion, or was made visible to it by its writer's proxy fence.  With
// .acquire.cluster and .release.cluster the softmax spent 1,100 cycles more
// per tile.)
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns = 2000000000ull) {
  auto done = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0) != 0;
  };
  if (done()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (done()) return true;
    if ((it & 63u) == 0) {
      if (__any_sync(0xffffffffu, *abort != 0 || globaltimer_ns() - t0 > limit_ns)) return false;
    }
  }
}

// The issuing roles run as whole warps on warp-uniform values and one elected
// lane (always the same) issues: descriptors and coordinates then stay in
// uniform registers.  Issued from a single-lane branch each MMA cost ~140
// cycles of register moves, twice its time on the tensor cores.

// TMA box into this CTA's shared memory; its bytes count on `bar` of CTA 0.
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

// Ring position of the producer and of the MMA issuer.
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ void step() {
    if (++s == kStages) {
      s = 0;
      phase ^= 1;
    }
  }
};

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
    sm.sum = 0;
    sm.src = 0x7fffffff;
    sm.units = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.qfull, 1);
    mbar_init(&sm.qempty, 1);
    mbar_init(&sm.sfull[0], 1);
    mbar_init(&sm.sfull[1], 1);
    mbar_init(&sm.pfull, 8);  // one arrival per softmax warp of both CTAs
    mbar_init(&sm.pvdone, 1);
    for (int i = 0; i < kTabs; ++i) mbar_init(&sm.vfull[i], 1);
    mbar_init(&sm.smsync[0], 2);
    mbar_init(&sm.smsync[1], 2);
    mbar_init(&sm.done, 1);
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
    tma_prefetch_desc(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  grid_dependency_wait();  // everything below reads inputs of earlier kernels

  // total tiles, and the first sequence that has the whole prefix
  {
    unsigned long long n = 0;
    int src = 0x7fffffff;
    for (int b = threadIdx.x; b < a.lay.batch; b += kThreads) {
      const long long L = seq_len(a, b);
      n += own_tiles(a, L);
      if (L >= a.prefix && b < src) src = b;
      if (blockIdx.x == 0 && __ldg(&a.lay.seq_lens[b]) > L) flag_status(a.status, DSA_STATUS_BAD_LENGTH);
    }
    if (n) atomicAdd(&sm.sum, n);
    if (src != 0x7fffffff) atomicMin(&sm.src, src);
  }
  __syncthreads();
  const int src = sm.src;
  const int row_lines = (a.prefix > 0 && src != 0x7fffffff) ? g.row_tiles : 0;
  const long long pre_tiles = (long long)row_lines * g.prefix_tiles;
  const long long total = pre_tiles + (long long)sm.sum;
  int G = gridDim.x >> 1;
  if (G > total) G = (int)total;
  const int pair = blockIdx.x >> 1;
  const long long lo = pair < G ? total * pair / G : 0;
  const long long mine = pair < G ? total * (pair + 1) / G - lo : 0;
  if (warp == 4) {  // line and tile of `lo`
    int line0 = 0, tile0 = 0;
    if (mine > 0) {
      if (lo < pre_tiles) {
        line0 = (int)(lo / g.prefix_tiles);
        tile0 = (int)(lo - (long long)line0 * g.prefix_tiles);
      } else {
        long long at = pre_tiles;
        for (int b0 = 0; b0 < a.lay.batch; b0 += 32) {
          const int n = b0 + lane < a.lay.batch ? own_tiles(a, seq_len(a, b0 + lane)) : 0;
          long long inc = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, at + inc > lo);
          if (hit) {
            const int l = __ffs(hit) - 1;
            const long long end = at + __shfl_sync(0xffffffffu, inc, l);
            line0 = row_lines + b0 + l;
            tile0 = (int)(lo - (end - __shfl_sync(0xffffffffu, n, l)));
            break;
          }
          at += __shfl_sync(0xffffffffu, inc, 31);
        }
      }
    }
    if (lane == 0) {
      sm.line0 = line0;
      sm.tile0 = tile0;
    }
  }
  if (blockIdx.x == 1 && warp == 0) {  // first tile of every sequence, for the merge
    long long at = pre_tiles;
    for (int b0 = 0; b0 < a.lay.batch; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < a.lay.batch ? own_tiles(a, seq_len(a, b)) : 0;
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (b < a.lay.batch) g.off[b] = at + inc - n;
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) g.off[a.lay.batch] = total;
  }
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
  const int line0 = sm.line0, tile0 = sm.tile0;
  const int Cq = (a.Dqk + 63) / 64;
  const int cols = (a.Dv + 127) / 128;     // 128-column halves of V instructions
  const int ninst = (cols + 1) / 2;        // instructions of 256 columns; the last may have 128

  if (warp == 4 || warp == 6) {
    // ----------------------------------------------------------- producers --
    // Two warps fill the stages in turn (a stage takes one warp ~350 cycles of
    // waiting, table reads and issue; the MMAs empty one in 256).
    const int me = warp >> 1 & 1;  // warp 4: 0, even stages of the sequence; warp 6: 1
    Tiles tk, tv;
    tk.init(g, row_lines, src, line0, tile0, mine);
    tv = tk;
    Ring r;
    int uk = 0, uv = 0, nq = 0, unit = 0;
    bool ok = true;
    const int R = g.R, per = kTile / R;  // groups per tile
    const int lgR = 31 - __clz(R);
    const int none = (int)g.pool_rows;   // a row outside the pool: zeros
    const uint32_t qbar = leader_addr(&sm.qfull);
    const uint32_t fbar = leader_addr(&sm.full[0]);
    const uint32_t ring = smem_u32(sm.ring[0]);
    const uint32_t empty = smem_u32(&sm.empty[0]), full = smem_u32(&sm.full[0]);
    // physical row of the tile's group i: `none` past the line's end, -1 - none
    // behind a bad block id
    auto lookup = [&](const Tiles& t, int i) {
      const long long p = t.pos() + (long long)i * R;
      if (p >= t.w.p1) return none;
      const uint32_t q = (uint32_t)p / (uint32_t)a.lay.bs;
      const int page = __ldg(&a.lay.bt[(long long)t.w.trow * a.lay.maxb + q]);
      if (page < 0 || page >= a.lay.nb) return -1 - none;
      return page * a.lay.bs + (int)((uint32_t)p - q * (uint32_t)a.lay.bs);
    };
    int ahead = tk.ok && lane < per ? lookup(tk, lane) : none;  // of the next tile to stage
    while ((tk.ok || uv < uk) && ok) {
      if (tk.ok) {
        const int slot = uk % kTabs;
        const int keys = tk.keys();
        int* tab = sm.tab[me][uk & 1];
        bool bad = false;
        for (int i = lane; i < per; i += 32) {
          int row = i < 32 ? ahead : lookup(tk, i);
          if (row < 0) {
            bad = true;
            row = -1;
          }
          tab[i] = row;
        }
        if (bad) flag_status(a.status, DSA_STATUS_BAD_BLOCK);
        __syncwarp();
        Tiles tn = tk;
        tn.next(g, row_lines, src);
        if (tn.ok && lane < per) ahead = lookup(tn, lane);
        if (tk.first) {  // the line's queries, once the previous line's last S is done
          if (me == 0) {
            if (nq > 0 && !pair_wait(smem_u32(&sm.qempty), (nq - 1) & 1, &sm.abort)) {
              ok = false;
              break;
            }
            const bool both = tk.w.rows > 64;
            if (rank == 0) expect_tx_elected(smem_u32(&sm.qfull), (both ? 2 : 1) * Cq * 64 * 128);
            if (rank == 0 || both)
              for (int c = 0; c < Cq; ++c)
                tma_pair(smem_u32(sm.q[0]) + c * 8192, &maps.q, qbar, 64 * c,
                         tk.w.row0 + 64 * rank);
          }
          ++nq;
        }
        if (me == 1) {
          // usable positions of the tile.  The slot was tile uk - 6's: at most
          // the ring's 7 stages of the K and V issued before (at least one of
          // each per tile) are not yet read by the MMAs, so O of that tile has
          // begun and its softmax is past the mask.
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
            sm.mask[slot][lane] = word;
          }
          const bool whole = __all_sync(0xffffffffu, lane >= kTile / 32 || word == 0xffffffffu);
          if (lane == 0) {
            sm.whole[slot] = whole;
            mbar_arrive(&sm.vfull[slot]);
          }
        }
        const int nb = 128 >> lgR;  // boxes per stage
        const int* mytab = tab + rank * nb;
        const int row0 = mytab[0] >= 0 ? mytab[0] : none;  // stages of one or two boxes
        const int row1 = nb < 2 || mytab[1] < 0 ? none : mytab[1];
        for (int c = 0; c < Cq; ++c, ++unit) {
          if ((unit & 1) == me) {
            if (!pair_wait(empty + 8 * r.s, r.phase ^ 1, &sm.abort)) { ok = false; break; }
            if (rank == 0) expect_tx_elected(full + 8 * r.s, 2 * kStageBytes);
            const uint32_t dst = ring + r.s * kStageBytes, bar = fbar + 8 * r.s;
            if (nb == 2) {
              tma_pair(dst, &maps.k, bar, 64 * c, row0);
              tma_pair(dst + kStageBytes / 2, &maps.k, bar, 64 * c, row1);
            } else {
              for (int i = 0; i < nb; ++i)
                tma_pair(dst + i * R * 128, &maps.k, bar, 64 * c, mytab[i] >= 0 ? mytab[i] : none);
            }
          }
          r.step();
        }
        if (!ok) break;
        ++uk;
        tk = tn;
      }
      // V runs one tile behind K, as the MMAs do
      if ((uk - uv == 2 || !tk.ok) && uv < uk) {
        const int* tab = sm.tab[me][uv & 1];
        const int keys = tv.keys();
        const int nkk = (keys + 63) / 64;
        const int nb = 64 >> lgR;
        for (int i = 0; i < ninst && ok; ++i) {
          const int blocks = (i < ninst - 1 || cols % 2 == 0) ? 2 : 1;  // 64-column blocks per CTA
          const int x0 = 256 * i + 64 * blocks * rank;
          for (int kk = 0; kk < nkk; ++kk, ++unit) {
            if ((unit & 1) == me) {
              if (!pair_wait(empty + 8 * r.s, r.phase ^ 1, &sm.abort)) { ok = false; break; }
              if (rank == 0) expect_tx_elected(full + 8 * r.s, 2 * blocks * 64 * 128);
              const uint32_t bar = fbar + 8 * r.s;
              for (int gi = 0; gi < nb; ++gi) {
                const int k0 = 64 * kk + gi * R;  // first position of the group in the tile
                const int row = tab[k0 >> lgR];
                const int n = keys - k0;          // cached positions of the group
                uint32_t dst = ring + r.s * kStageBytes + gi * R * 128;
                if (row < 0 || n >= R || n <= 0) {
                  tma_pair(dst, &maps.v, bar, x0, row >= 0 ? row : none);
                  if (blocks == 2) tma_pair(dst + 8192, &maps.v, bar, x0 + 64, row >= 0 ? row : none);
                  continue;
                }
                // the line ends inside the group
                for (int blk = 0; blk < blocks; ++blk, dst += 8192) {
                  const int x = x0 + 64 * blk;
                  int j = 0;
                  for (; j + 8 <= R; j += 8)
                    if (j + 8 <= n || j >= n) {
                      tma_pair(dst + j * 128, &maps.v8, bar, x, j < n ? row + j : none);
                    } else {
                      for (int q = j; q < j + 8; ++q)
                        tma_pair(dst + q * 128, &maps.v1, bar, x, q < n ? row + q : none);
                    }
                  for (; j < R; ++j)
                    tma_pair(dst + j * 128, &maps.v1, bar, x, j < n ? row + j : none);
                }
              }
            }
            r.step();
          }
        }
        if (!ok) break;
        ++uv;
        tv.next(g, row_lines, src);
      }
    }
    if (lane == 0) atomicMax(&sm.units, unit);
    if (!ok && lane == 0) fail(sm, a.status);
  } else if (warp == 5) {
    // ---------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      Tiles ts, tv;
      ts.init(g, row_lines, src, line0, tile0, mine);
      tv = ts;
      Ring r;
      int us = 0, uv = 0, nq = 0;
      bool ok = true;
      const uint32_t idS = instr_desc(kRows, 256, 1, 1, 0, 0);
      const uint32_t empty = smem_u32(&sm.empty[0]), full = smem_u32(&sm.full[0]);
      // descriptors: the address field counts 16 bytes; a step of 16 dims or
      // positions is 32 bytes of a K-major operand, 2048 of V
      const uint64_t dq = smem_desc(smem_u32(sm.q[0]), 16, 1024, kSwizzle128B);
      const uint64_t dp = smem_desc(smem_u32(sm.p[0]), 16, 1024, kSwizzle128B);
      const uint64_t dk = smem_desc(smem_u32(sm.ring[0]), 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(smem_u32(sm.ring[0]), 8192, 1024, kSwizzle128B);
      while ((ts.ok || uv < us) && ok) {
        if (ts.ok) {
          if (ts.first) {
            if (!pair_wait(smem_u32(&sm.qfull), nq & 1, &sm.abort)) { ok = false; break; }
            ++nq;
          }
          // S buffer us % 2 was read before the weights of tile us - 2 were
          // announced, which O of that tile has waited for
          const uint32_t d = tbase + kColS + 128 * (us & 1);
          for (int c = 0; c < Cq; ++c) {
            if (!pair_wait(full + 8 * r.s, r.phase, &sm.abort)) { ok = false; break; }
            tc_fence_after();
            const uint64_t qa = dq + 512 * c, kb = dk + 1024 * r.s;
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_pair(d, qa + 2 * k, kb + 2 * k, idS, c + k);
            commit_pair(empty + 8 * r.s);
            r.step();
          }
          if (!ok) break;
          commit_pair(smem_u32(&sm.sfull[us & 1]));
          if (ts.last) commit_pair(smem_u32(&sm.qempty));
          ++us;
          ts.next(g, row_lines, src);
        }
        if ((us - uv == 2 || !ts.ok) && uv < us) {
          const int nkk = (tv.keys() + 63) / 64;
          if (!pair_wait(smem_u32(&sm.pfull), uv & 1, &sm.abort)) { ok = false; break; }
          for (int i = 0; i < ninst && ok; ++i) {
            const int blocks = (i < ninst - 1 || cols % 2 == 0) ? 2 : 1;
            const uint32_t id = instr_desc(kRows, 128 * blocks, 1, 1, 0, 1);
            const uint32_t d = tbase + kColO + 128 * i;
            for (int kk = 0; kk < nkk; ++kk) {
              if (!pair_wait(full + 8 * r.s, r.phase, &sm.abort)) { ok = false; break; }
              tc_fence_after();
              const uint64_t pa = dp + 512 * kk, vb = dv + 1024 * r.s;
              const int add = tv.first ? kk : 1;
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_pair(d, pa + 2 * k, vb + 128 * k, id, add + k);
              commit_pair(empty + 8 * r.s);
              r.step();
            }
          }
          if (!ok) break;
          commit_pair(smem_u32(&sm.pvdone));
          ++uv;
          tv.next(g, row_lines, src);
        }
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
    const uint32_t pbar = leader_addr(&sm.pfull);
    Tiles t;
    t.init(g, row_lines, src, line0, tile0, mine);
    int u = 0;
    uint32_t sp = 0;
    bool ok = true;
    float m = -INFINITY, l = 0.0f;
    while (t.ok && ok) {
      const bool live = t.w.rows > 64 * rank;  // else this CTA's rows are not of the line
      if (t.first) {
        m = -INFINITY;
        l = 0.0f;
      }
      if (!pair_wait(smem_u32(&sm.sfull[u & 1]), (u >> 1) & 1, &sm.abort)) { ok = false; break; }
      tc_fence_after();
      if (live) {
        uint32_t z[4][32];
        const uint32_t ta = tbase + lanes + kColS + 128 * (u & 1);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32cols(ta + 32 * q, z[q]);
        tmem_wait_ld();
        if (!pair_wait(smem_u32(&sm.vfull[u % kTabs]), (u / kTabs) & 1, &sm.abort)) { ok = false; break; }
        if (!sm.whole[u % kTabs]) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t w = sm.mask[u % kTabs][4 * half + q];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((w >> i) & 1u)) z[q][i] = 0xff800000u;
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 32; ++i) mx[q] = fmaxf(mx[q], __uint_as_float(z[q][i]));
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
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
        l *= f;
        float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t pk[64];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float e0 = ex2_approx(fmaf(__uint_as_float(z[q][i]), c, -mm));
            const float e1 = ex2_approx(fmaf(__uint_as_float(z[q][i + 1]), c, -mm));
            ls[q] += e0 + e1;
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
            pk[(32 * q + i) / 2] = *reinterpret_cast<const uint32_t*>(&b2);
          }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        // the previous O product has read P, and O may be rescaled
        if (u > 0 && !pair_wait(smem_u32(&sm.pvdone), (u - 1) & 1, &sm.abort)) { ok = false; break; }
        tc_fence_after();
        if (!t.first && __any_sync(0xffffffffu, resc)) {
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
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          uint8_t* dst = sm.p[2 * half + (k >> 3)] + row * 128 + (((k & 7) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) =
              make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
      } else if (u > 0 && !pair_wait(smem_u32(&sm.pvdone), (u - 1) & 1, &sm.abort)) {
        // a warp without rows keeps in step: two arrivals of it in one phase
        // of pfull would stand for a warp that has not written its weights
        ok = false;
        break;
      }
      __syncwarp();
      if (lane == 0) arrive_cluster(pbar);
      if (t.last) {
        // this pair's partial of the line: O out of TMEM, unnormalised
        if (!pair_wait(smem_u32(&sm.pvdone), u & 1, &sm.abort)) { ok = false; break; }
        tc_fence_after();
        if (live) {
          const int slot = t.w.pre ? pair + t.w.line
                                   : g.slots_pre + pair + (t.w.line - row_lines);
          const int Rw = t.w.pre ? kRows : g.Rl;
          float4* po = reinterpret_cast<float4*>(slot_po(g, slot, t.w.pre)) + 64 * rank + row;
#pragma unroll 1
          for (int q = 0; q < 2 * cols; ++q) {
            const int i = q >> 2;
            const int n2 = (i < ninst - 1 || cols % 2 == 0) ? 128 : 64;  // columns per half
            const int dv = 256 * i + n2 * half + 32 * (q & 3);
            uint32_t v[32];
            tmem_ld_32cols(tbase + lanes + kColO + 32 * q, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (dv + 4 * j < a.Dv)
                po[(size_t)(dv / 4 + j) * Rw] =
                    make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          }
          tc_fence_before();
          // the two halves' sums; the slot of redm is the next tile's, whose
          // own exchange comes after this one
          sm.redm[(u + 1) & 1][half][row] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.smsync[warp & 1]);
          if (!pair_wait(smem_u32(&sm.smsync[warp & 1]), sp, &sm.abort)) { ok = false; break; }
          sp ^= 1;
          if (half == 0)
            reinterpret_cast<float2*>(g.ml)[(size_t)slot * kRows + 64 * rank + row] =
                make_float2(m, l + sm.redm[(u + 1) & 1][1][row]);
          // nobody writes redm[(u + 1) & 1] again before this read is done
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.smsync[warp & 1]);
          if (!pair_wait(smem_u32(&sm.smsync[warp & 1]), sp, &sm.abort)) { ok = false; break; }
          sp ^= 1;
        }
      }
      ++u;
      t.next(g, row_lines, src);
    }
    if (!ok && lane == 0) fail(sm, a.status);
  }

  __syncthreads();
  if (warp == 0) {
    int never = 0;
    // MMAs of the pair done; after a failure also the copies in flight
    pair_wait(smem_u32(&sm.done), 0, &never, 100000000ull);
    if (sm.abort && rank == 0) {
      for (int i = 0; i < kStages; ++i) {
        const int n = (sm.units - i + kStages - 1) / kStages;  // fills of this stage
        if (n > 0) pair_wait(smem_u32(&sm.full[i]), (n - 1) & 1, &never, 10000000ull);
      }
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

// Join the partials of each row.  Grid (B, groups of 32 heads, quarters of
// 128 columns), 256 threads: a lane is a row (partials are stored with rows
// innermost, so a warp reads 512 contiguous bytes per float4 of columns), the
// warps take the columns in turn; the finished block is turned in shared
// memory and written row by row.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) k_prefix_merge(const __grid_constant__ Geo g,
                                                                int pairs) {
  __shared__ uint32_t tile[32][66];  // 128 bf16 per row, padded
  const PrefixAttnParams& a = g.a;
  grid_dependency_wait();
  launch_dependents();
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 32 + lane;
  const int x0 = blockIdx.z * 128;
  const long long total = g.off[a.lay.batch], o0 = g.off[b], o1 = g.off[b + 1];
  int G = pairs;
  if (G > total) G = (int)total;
  const bool mine = h < a.Hq;
  const long long L = seq_len(a, b);
  // partials: prefix slots p0 .. p0 + np - 1, sequence slots s0 .. s0 + ns - 1
  int p0 = 0, np = 0, s0 = 0, ns = 0, prow = 0;
  const long long first = g.off[0];
  if (first > 0 && L >= a.prefix && mine) {
    const int r = b * a.Hq + h, line = r / kRows;
    prow = r - line * kRows;
    const long long x = (long long)line * g.prefix_tiles;
    const int c0 = (int)(((x + 1) * G - 1) / total);
    const int c1 = (int)(((x + g.prefix_tiles) * G - 1) / total);
    p0 = c0 + line;
    np = c1 - c0 + 1;
  }
  if (o1 > o0 && mine) {
    const int c0 = (int)(((o0 + 1) * G - 1) / total);
    const int c1 = (int)((o1 * G - 1) / total);
    s0 = g.slots_pre + c0 + b;
    ns = c1 - c0 + 1;
  }
  const float2* ml = reinterpret_cast<const float2*>(g.ml);
  const int n = np + ns;
  auto stat = [&](int i) {
    return i < np ? __ldcg(&ml[(size_t)(p0 + i) * kRows + prow])
                  : __ldcg(&ml[(size_t)(s0 + i - np) * kRows + h]);
  };
  float M = -INFINITY;
  for (int i = 0; i < n; ++i) {
    const float2 v = stat(i);
    if (v.y != 0.0f) M = fmaxf(M, v.x);
  }
  const float Ms = M == -INFINITY ? 0.0f : M;
  float l = 0.0f;
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < n; ++i) {
    const float2 v = stat(i);
    const float w = v.y != 0.0f ? exp2f(v.x - Ms) : 0.0f;
    if (v.y != 0.0f) l = fmaf(v.y, w, l);
    const bool pre = i < np;
    const int Rw = pre ? kRows : g.Rl;
    const float4* po = reinterpret_cast<const float4*>(
                           slot_po(g, pre ? p0 + i : s0 + i - np, pre)) + (pre ? prow : h);
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int dv = x0 + 4 * (warp + 8 * j);
      x[j] = dv < a.Dv && v.y != 0.0f ? __ldcg(&po[(size_t)(dv / 4) * Rw])
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[j].x = fmaf(w, x[j].x, acc[j].x);
      acc[j].y = fmaf(w, x[j].y, acc[j].y);
      acc[j].z = fmaf(w, x[j].z, acc[j].z);
      acc[j].w = fmaf(w, x[j].w, acc[j].w);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[j].x * inv, acc[j].y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[j].z * inv, acc[j].w * inv);
    tile[lane][2 * (warp + 8 * j)] = *reinterpret_cast<const uint32_t*>(&lo);
    tile[lane][2 * (warp + 8 * j) + 1] = *reinterpret_cast<const uint32_t*>(&hi);
  }
  if (a.lse && blockIdx.z == 0 && warp == 0 && mine)
    a.lse[(size_t)b * a.Hq + h] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
  __syncthreads();
  const int w4 = min(128, a.Dv - x0) / 8;  // 16-byte pieces of a row's quarter
  for (int i = threadIdx.x; i < 32 * 16; i += kMergeThreads) {
    const int r = i >> 4, k = i & 15, hh = blockIdx.y * 32 + r;
    if (hh < a.Hq && k < w4)
      *reinterpret_cast<uint4*>(a.out + ((size_t)b * a.Hq + hh) * a.Dv + x0 + 8 * k) =
          make_uint4(tile[r][4 * k], tile[r][4 * k + 1], tile[r][4 * k + 2], tile[r][4 * k + 3]);
  }
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
  w.ml = w.off + round256(sizeof(long long) * ((size_t)B + 1));
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
  g.off = reinterpret_cast<long long*>(base + w.off);
  g.ml = reinterpret_cast<float*>(base + w.ml);
  g.po = reinterpret_cast<float*>(base + w.po);
  g.slots_pre = w.slots_pre;
  g.row_tiles = w.row_tiles;
  g.Rl = w.Rl;
  g.prefix_tiles = (p.prefix + kTile - 1) / kTile;
  g.pool_rows = (long long)p.lay.nb * p.lay.bs;
  int R = 64;
  while (p.lay.bs % R || p.prefix % R) R >>= 1;
  g.R = R;
  Maps m;
  int rc = make_tmap_2d(&m.q, p.q, false, p.Dqk, (uint64_t)p.lay.batch * p.Hq, (uint64_t)p.Dqk * 2,
                        64, 64);
  if (!rc)
    rc = make_tmap_2d(&m.k, p.kp, false, p.Dqk, (uint64_t)g.pool_rows, (uint64_t)p.ks * 2, 64, R);
  if (!rc)
    rc = make_tmap_2d(&m.v, p.vp, false, p.Dv, (uint64_t)g.pool_rows, (uint64_t)p.vs * 2, 64, R);
  if (!rc)
    rc = make_tmap_2d(&m.v8, p.vp, false, p.Dv, (uint64_t)g.pool_rows, (uint64_t)p.vs * 2, 64, 8);
  if (!rc)
    rc = make_tmap_2d(&m.v1, p.vp, false, p.Dv, (uint64_t)g.pool_rows, (uint64_t)p.vs * 2, 64, 1);
  if (rc) return rc;
  const size_t smem = sizeof(Smem) + 1024;
  rc = ensure_dynamic_smem((const void*)k_prefix_attn, (int)smem, "prefix_attn_decode");
  if (rc) return rc;
  int pairs = max_active_clusters((const void*)k_prefix_attn, kThreads, smem, 2);
  if (pairs < 1) return set_error(DSA_ERR_CUDA, "prefix_attn_decode: no cluster of two CTAs fits");
  if (pairs > kMaxPairs) pairs = kMaxPairs;
  const long long bound = (long long)g.row_tiles * g.prefix_tiles +
                          (long long)p.lay.batch * ((p.lay.max_len + kTile - 1) / kTile);
  if (pairs > bound) pairs = bound < 1 ? 1 : (int)bound;
  cudaError_t e = launch_pdl_cluster(k_prefix_attn, dim3((unsigned)(2 * pairs)), dim3(kThreads),
                                     smem, 2, s, m, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  rc = check_launch("prefix_attn_decode");
  if (rc) return rc;
  e = launch_pdl(k_prefix_merge,
                 dim3((unsigned)p.lay.batch, (unsigned)((p.Hq + 31) / 32),
                      (unsigned)((p.Dv + 127) / 128)),
                 dim3(kMergeThreads), 0, s, g, pairs);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("prefix_attn_decode merge");
}

}  // namespace dsa
