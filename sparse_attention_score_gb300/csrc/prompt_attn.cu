// prompt_attn.cu -- exact causal attention of whole prompts, several sequences
// packed end to end, grouped heads, on the tensor cores.
//
// The exact softmax of the sparse attention ("Day-0 Adaptation of
// Trillion-Parameter MoE Models on Domestic GPUs", section 3 (3): the
// compute-bound prefill) with every causal position selected, on keys and
// values that are still in hand as packed heads, so nothing is gathered.
//
// Rows and tiles.  A row is one (token, query head).  The heads that share a key
// head and the tokens of a sequence are laid together in tiles of 128 rows:
// gp heads (the largest power of two that divides the group) of 128 / gp
// tokens, which a TMA box brings in as such.  An item is two such tiles, A and
// B, one behind the other in the sequence, over all the keys that they see, in
// tiles of 128 keys.  CTAs (one per SM, persistent) take items off a counter,
// those of late tokens, which see most, first.
//
// One key tile (tcgen05, M = 128, one accumulator of 128 columns each):
//   S_X [128 x 128] = Q_X K^T       X = A, B; operands in shared memory;
//   softmax: a thread has a row of S_X; the running maximum is raised only when a
//       tile exceeds it by more than 2^8, and O_X rescaled then (an economy known
//       from published attention kernels);
//   P_X bf16 over S_X in TMEM;  O_X [128 x Dv] += P_X V, P_X from TMEM.
// The tensor cores alternate: while the softmax of A works on its scores, they
// do O and the next S of B.  TMEM: S_A, S_B, O_A, O_B, 128 columns each.  V of
// more than 128 columns is taken in two halves, each an item of its own that
// computes S again.
//
// P is rounded to bf16 once, each weight by at most 2^-8 of itself, which gives up
// exactness for speed: over values of mixed sign the output shrinks by the same root
// of the number of keys as the summed roundings, so they add about as much as the
// bf16 output's own rounding, however many keys there are (0.0023 of the output's
// norm instead of 0.0017 behind 6,000 keys).  hi + lo weights (2^-16, both multiplied
// with the same V) take that away for half as many products again: 16384 tokens of 64
// heads over 8 4,369 us, now 3,042, chunks behind 6,000 keys 875 and 670.  They are
// taken where that costs little: by an item whose first row sees no more than 512
// keys.  Statistics and sums are fp32.
//
// What no row may see.  Scores of hidden keys are set to -inf by the row's own
// limit.  V has no such place: a hidden row's weight is 0, but 0 times what an
// unrelated sequence, or a later token, has there may be NaN.  Two warps
// therefore look through V of the key tiles that some row sees in part (one or
// two per item; of every tile where weights are hi + lo, whose lo may be 0), before
// the product: rows that no row of the item sees become zeros, and so do
// infinities and NaN; an item with such values adds them to the rows that do see
// them when it writes its output.
//
// Few rows over many keys.  Items are cut along the keys where one would take more
// than twice an even share of the work, and where items of one size leave the last
// wave of CTAs mostly idle: a piece leaves its unnormalised (O, m, l) in the
// workspace, an item's first piece names the item there, and k_prompt_merge joins a
// row's pieces in a fixed order.  8 tokens of 24 heads over 6 behind 6,177 keys: 27
// us, uncut 104; ~3,000 tokens of 64 heads of 192 / 128 behind 6,000 keys (5.05 items
// per SM) 608 us when uncut ones took 656 (595 since).
//
// Warp roles (384 threads): 0-3 softmax of A, 4-7 of B, 8 fills the ring of K
// and V (chunks of 64 dims of 128 keys) and Q, 9 issues the products, 10 and 11
// look through V.  Every wait is bounded (DSA_STATUS_TIMEOUT, then the CTA winds
// down).
//
// What bounds it.  A key tile of an item is 2,048 cycles of MMAs (128 dims) and, by
// count, 256 KB through shared memory (scores read both operands there), as many
// cycles at 128 bytes each; the exponentials take 1,024 of the special-function units.
// 16384 tokens of 64 heads over 8 key heads of 128: 2,855 us, 1,540 TFLOP/s (81 % of
// the cuBLAS rate, 91 % of its rate under the power cap), the matrix unit 62 % busy;
// chunks of 64 heads of 192 / 128: 1,440 TFLOP/s, with keys and values of all heads
// read from memory 2.7 times (items go pair by pair, over all heads); 12 ragged prompts
// of up to 1,500 tokens, 24 heads over 4 of 80: 86 us, bound by the chain of a tile
// (scores, softmax, weights: ~1.9 us) and an item's setup and output (~4.6 us) where
// items have a handful of tiles.
// Measured on the way, for the first of these: MMAs whose operands the compiler
// cannot prove warp-uniform 4,317 us (each is then a loop over lanes; shuffles make
// them uniform now: 3,244 with the weights in one pass where the maximum holds); all
// 128 scores of a row in registers at once, spilled: 4,320; 16 softmax warps with half
// a row each: 3,226 where 8 took 3,030; less code per role, weights handed over in
// halves and chunks released by their own last product: 2,890.  A split of the
// registers between the roles (setmaxnreg 72 / 216) did not end; the cause is not
// known and it is left out.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "device_common.cuh"
#include "dsa_internal.cuh"
#include "prompt_attn.cuh"
#include "sm100.cuh"

namespace dsa {

namespace {

using namespace sm100;

constexpr int kTile = 128;              // rows of a tile, keys of a tile
constexpr int kChunk = 64;              // dims of a chunk
constexpr int kChunkBytes = kTile * kChunk * 2;
constexpr int kThreads = 384;
constexpr int kMaxRing = 12;            // chunks
constexpr int kSlots = 4;               // item descriptors in flight
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 X
constexpr float kRescaleLog2 = 8.0f;
// A weight is 2^(z c - m) in one fma, exact but for the rounding of the maximum m, which
// all weights of a row have in common and their sum takes out again.  From |m| = 2^24
// on that rounding is a power of two and more, and past 2^31 or so of infinity: there
// z c is rounded like m before m leaves it, and the largest weight is 1 again.
constexpr float kFar = 16777216.0f;
constexpr int kShort = 512;
// Key tiles after which O leaves TMEM for a sum of its own in the workspace.  The matrix
// unit cuts its sums off where an fp32 addition rounds, so that O shrinks by about 2^-27
// for every key: 0.7 % over 10^6, an eighth of bf16's half step over the 65,536 of this.
// Asking for it costs 2 % (16384 tokens of 64 heads over 8 2,900 us, without 2,853; 12
// ragged prompts 88 and 86), so it is an instantiation of its own for calls with more
// keys than 2^18, over which a sequence would lose half of bf16's half step.
constexpr int kFlush = 512;
constexpr int kLongKeys = 1 << 18;
constexpr int kMaxCtas = 160;
constexpr int kVWidth = 128;            // columns of V per item
constexpr int kReaders = 11;            // warps that read an item's descriptor

struct Item {
  int end;        // no more items
  int q0;         // tile A's first token in q
  int tok;        // ... and in its sequence
  int nq, nk, k0; // of the sequence
  int hk, h0;     // key head, first query head
  int v0, dv;     // columns of V
  int j0;         // the first key tile of the item
  int n[2];       // key tiles of A and B from there on
  int lim;        // keys that the first row sees
  int jm;         // the first key tile whose V is looked through
  int slot;       // of the partial result, -1: the item sees all its keys' tiles
};

struct Smem {
  uint64_t full[kMaxRing], empty[kMaxRing];
  uint64_t qfull[2], qempty[2], sfull[2], pfull[2][2], ofull[2];
  uint64_t ifull[kSlots], iempty[kSlots], done;
  Item item[kSlots];
  int odd[2][2 * kSlots];  // per reader of V: the item's V held infinities or NaN
  int vissued;       // V tiles to look through: whose copies were issued,
  int vclean[2];     // ... which each of the two warps is done with
  int fills, qfills[2];
  uint32_t tmem_base;
  int abort;
  float work[kThreads / 32];  // what each warp found of the sequences' work and pairs
  int pairs[kThreads / 32];
};

struct Maps {
  CUtensorMap q, k, v;
};

// Key tiles that a piece of a cut item has at least: it costs its setup, a partial
// result and its part of the join.  A token of 32 heads over 8 behind 4,096 keys takes
// 24.2 us with 3, 22.8 with 4, 26.3 with 6, 27.6 with 8 and 40.6 with 12; 8 tokens of
// 24 over 6 behind 6,177 keys 26.8, 26.5, 28.3, 31.1 and 36.4.
constexpr int kMinPiece = 4;
constexpr int kSlotRows = 2 * kTile;

// A cut item, for the join.
struct __align__(16) Join {
  int slot, used;  // its first partial result and how many there are
  int q0, left;    // tile A's first token in q; the sequence's tokens from there on
  int h0, v0;      // first query head, first column of V
  int pad[2];
};

struct Geo {
  PromptAttnParams a;
  int slots;          // partial results that the workspace holds, 0: no item is cut
  int ctas;
  int many;           // there may be more items than CTAs
  float2* ml;         // [slot][256] (maximum, sum)
  float* po;          // [slot][columns / 4][256][4]
  float* acc;         // [CTA][columns / 4][256][4]: O of an item's tiles but the last ones
  Join* join;         // [joins], at most one per slot
  int* joins;
  int* jleft;         // blocks of the join that are done
  int G, lgp, HB;     // query heads per key head, log2 of gp, G / gp
  int lgpair;         // log2 of a pair's tokens
  int VH;             // items per head over V's columns
  int HH;             // items per pair of tiles
  int nkc;            // chunks of Q and K
  int ring;           // chunks
  int* next;          // the next item
  int* left;          // CTAs that are done
};

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void expect_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from TMEM: a row per lane, two bf16 of a row per column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_8cols(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t pair2(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
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

// Scores of columns 32 q .. 32 q + 31 that lie at or behind `see` are hidden.
__device__ __forceinline__ void hide(uint32_t (&z)[32], int q, int see) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (32 * q + i >= see) z[i] = 0xff800000u;
}

// A warp that has nothing to do in an item waits as long as the others work on it (256
// rows take 12 ns a key: 26 s over 2^31 of them); whoever gives up sets *abort, which
// ends this wait too.  Every other wait is for one step of a neighbour.
constexpr uint64_t kStepNs = 2000000000ull, kItemNs = 60000000000ull;

// pair_wait with less code: the warps of a scheduler share an instruction cache
// that holds little more than the loops below.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit = kStepNs) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, ok != 0)) return true;
    if ((it & 63u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, *abort != 0 || now - t0 > limit)) return false;
    }
  }
}

// Wait of a whole warp until *count (in shared memory, only growing) is at
// least n; bounded like pair_wait.
__device__ __forceinline__ bool count_wait(const int* count, int n, volatile int* abort, uint64_t limit = kStepNs) {
  const uint32_t addr = smem_u32(count);
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    if (__all_sync(0xffffffffu, v >= n)) return true;
    if ((it & 63u) == 0 && __any_sync(0xffffffffu, *abort != 0 || globaltimer_ns() - t0 > limit)) return false;
  }
}

__device__ __forceinline__ void count_set(int* count, int n) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(count)), "r"(n) : "memory");
}

__device__ __forceinline__ void fail(Smem& sm, int* status) {
  sm.abort = 1;
  flag_status(status, DSA_STATUS_TIMEOUT);
}

// Tokens and keys of sequence b, empty if its offsets are not inside q and k.
__device__ __forceinline__ bool sequence(const PromptAttnParams& a, int b, int* q0, int* nq, int* k0, int* nk) {
  const int qa = a.cu_q ? __ldg(&a.cu_q[b]) : 0, qb = a.cu_q ? __ldg(&a.cu_q[b + 1]) : a.Nq;
  const int ka = a.cu_k ? __ldg(&a.cu_k[b]) : 0, kb = a.cu_k ? __ldg(&a.cu_k[b + 1]) : a.Nk;
  const bool good = qa >= 0 && qb >= qa && qb <= a.Nq && ka >= 0 && kb >= ka && kb <= a.Nk;
  *q0 = good ? qa : 0;
  *nq = good ? qb - qa : 0;
  *k0 = good ? ka : 0;
  *nk = good ? kb - ka : 0;
  return good;
}

__host__ __device__ __forceinline__ int visible(int tok, int nq, int nk) {  // keys that a token sees
  const long long v = (long long)tok + 1 + nk - nq;
  return v < 0 ? 0 : (int)(v > nk ? nk : v);
}

// Key tiles over n keys (which may be 2^31 - 1).
__host__ __device__ __forceinline__ int tiles_over(int n) { return (int)(((unsigned)n + kTile - 1u) / kTile); }

__device__ __forceinline__ int scan_add(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// One sequence's items.  Pairs of tiles are counted from the last token's on, so
// that the number of keys that they see falls.  (Counts fit 32 bits: the host
// refuses more items.)
struct Seq {
  int q0, nq, k0, nk;
  int pairs;       // pairs of tiles, of 2^lg tokens
  int most;        // key tiles of the first pair
  int cut, pieces; // the first `cut` pairs are cut in up to `pieces` pieces
  int tail, tpieces;  // the last `tail` pairs in up to `tpieces`
  __host__ __device__ __forceinline__ int tiles_of(int lg, int pair) const {
    const long long end = (long long)(pairs - pair) << lg;
    return tiles_over(visible((int)(end < nq ? end : nq) - 1, nq, nk));
  }
  __host__ __device__ __forceinline__ void shape(int lg) {
    pairs = (int)(((long long)nq + (1 << lg) - 1) >> lg);
    most = pairs > 0 ? tiles_of(lg, 0) : 0;
    cut = tail = 0;
    pieces = tpieces = 1;
  }
  // about the key tiles of all pairs: they fall evenly to the last pair that sees any
  __host__ __device__ __forceinline__ float work(int lg) const {
    if (pairs == 0) return 0.0f;
    const int least = tiles_of(lg, pairs - 1);
    const int some = least > 0 ? pairs : (nk >> lg) + 1;
    return 0.5f * (float)(some < pairs ? some : pairs) * (float)(most + least + 1);
  }
  // pieces of a cut pair of N key tiles
  __device__ __forceinline__ int used(int N, int pair, int c) const {
    return pair < cut ? N / c : max(min(tpieces, N / kMinPiece), 1);
  }
  // Pairs of N >= 2 c key tiles are cut in N / c pieces (c tiles and less than c
  // more, so that an even share stays one): those whose last token sees more than
  // (2 c - 1) * 128 keys.
  __device__ __forceinline__ void cut_at(int lg, int c) {
    if (c <= 0 || most < 2 * c) return;
    pieces = most / c;
    const long long first = (long long)(2 * c - 1) * kTile + nq - nk;  // the first such token
    const long long below = first <= 0 ? 0 : first >> lg;              // pairs that end before it
    cut = below < pairs ? pairs - (int)below : 0;
  }
};

// Key tiles of a piece: an even share of the work, but no less than pays for a
// partial result and the join; 0 where nothing is cut.
__host__ __device__ __forceinline__ int piece_of(float work, int HH, int ctas) {
  const float c = ceilf(work * (float)HH / (float)ctas);
  return c < (float)kMinPiece ? kMinPiece : c < 1e6f ? (int)c : 1000000;
}

// Where items of about one size leave the last wave of CTAs mostly idle, those of
// that wave are cut too: `rest` of `items` are over, of N key tiles each.
__host__ __device__ __forceinline__ bool cut_tail(long long items, int ctas, int rest, int N) {
  return items >= ctas && items < 12LL * ctas && rest > 0 && N >= 3 * kMinPiece &&
         (long long)(ctas - rest) * N >= 8LL * ctas;
}

// Read by every CTA from the same lengths, in the same order.
struct Cuts {
  int c;          // key tiles of a piece, 0: nothing is cut
  int items;      // uncut
};
// A warp's part: every twelfth group of 32 sequences (~1 us for each group; with one
// warp of every CTA, and again in the join, 608 sequences of 256 tokens behind as many
// took 129 us, 83 so).
__device__ __forceinline__ void add_up(const Geo& g, Smem& sm, int warp, int lane) {
  float sum = 0.0f;
  int pairs = 0;
  for (int b0 = 32 * warp; b0 < g.a.B; b0 += kThreads) {
    Seq s;
    s.nq = s.nk = 0;
    if (b0 + lane < g.a.B) sequence(g.a, b0 + lane, &s.q0, &s.nq, &s.k0, &s.nk);
    s.shape(g.lgpair);
    sum += s.work(g.lgpair);
    pairs += s.pairs;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  pairs = __reduce_add_sync(0xffffffffu, pairs);
  if (lane == 0) {
    sm.work[warp] = sum;
    sm.pairs[warp] = pairs;
  }
}
__device__ __forceinline__ Cuts find_cuts(const Geo& g, const Smem& sm) {
  if (g.slots == 0) return Cuts{0, 0};
  float sum = 0.0f;
  int pairs = 0;
#pragma unroll 1
  for (int i = 0; i < kThreads / 32; ++i) {
    sum += sm.work[i];
    pairs += sm.pairs[i];
  }
  return Cuts{piece_of(sum, g.HH, g.ctas), pairs * g.HH};
}

// Sequences in groups of 32, a lane each: items and slots of the partial results,
// counted up from group to group.
struct Group {
  int b0 = -32;
  int base = 0, end = 0, mine = 0;     // items: before the group, up to this lane's sequence, its own
  int sbase = 0, send = 0, smine = 0;  // slots
  Seq s;
  __device__ __forceinline__ bool next(const Geo& g, const Cuts& cuts, int lane) {
    b0 += 32;
    if (b0 >= g.a.B) return false;
    if (b0 > 0) {
      base = __shfl_sync(0xffffffffu, end, 31);
      sbase = __shfl_sync(0xffffffffu, send, 31);
    }
    s.q0 = s.nq = s.k0 = s.nk = 0;
    if (b0 + lane < g.a.B && !sequence(g.a, b0 + lane, &s.q0, &s.nq, &s.k0, &s.nk))
      flag_status(g.a.status, DSA_STATUS_BAD_LENGTH);
    s.shape(g.lgpair);
    s.cut_at(g.lgpair, cuts.c);
    // (an even share needs about two slots per SM; where that does not hold, what
    // has no slots is not cut)
    smine = min((long long)s.cut * s.pieces * g.HH, (long long)g.slots + 1);
    send = sbase + scan_add(smine, lane);
    if (send > g.slots) {
      s.cut = 0;
      s.pieces = 1;
      send = g.slots;  // (and nothing behind it is)
    }
    if (g.many && b0 + 32 >= g.a.B && cuts.c > 0) {
      // the last sequence's last pairs
      const unsigned some = __ballot_sync(0xffffffffu, s.pairs > 0);
      if (some && lane == 31 - __clz(some)) {
        const int rest = cuts.items % g.ctas, tail = min((rest + g.HH - 1) / g.HH, s.pairs - s.cut);
        if (tail > 0) {
          const int N = s.tiles_of(g.lgpair, s.pairs - tail);
          const int n = min(N / kMinPiece, (g.slots - send) / (tail * g.HH));
          if (n >= 2 && cut_tail(cuts.items, g.ctas, rest, N)) {
            s.tail = tail;
            s.tpieces = n;
            smine += tail * n * g.HH;
            send += tail * n * g.HH;
          }
        }
      }
    }
    mine = (s.pairs + s.cut * (s.pieces - 1) + s.tail * (s.tpieces - 1)) * g.HH;
    end = base + scan_add(mine, lane);
    return true;
  }
};

// The item `at`, found from the last one on.
struct Finder {
  Group grp;
  Cuts cuts{};
  int joined = 0;  // of an item's first piece: how many there are
  __device__ __forceinline__ void init(const Geo& g, const Smem& sm, int lane) {
    cuts = find_cuts(g, sm);
    grp.next(g, cuts, lane);
  }
  // 1: an item, 0: none are left, 2: an empty piece
  __device__ int find(const Geo& g, int at, int lane, Item* it) {
    for (;;) {
      const unsigned hit = __ballot_sync(0xffffffffu, grp.end > at);
      if (hit) {
        const int l = __ffs(hit) - 1;
        auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, l); };
        Seq s;
        s.q0 = of(grp.s.q0);
        s.nq = of(grp.s.nq);
        s.k0 = of(grp.s.k0);
        s.nk = of(grp.s.nk);
        s.pairs = of(grp.s.pairs);
        s.cut = of(grp.s.cut);
        s.pieces = of(grp.s.pieces);
        s.tail = of(grp.s.tail);
        s.tpieces = of(grp.s.tpieces);
        int r = at - of(grp.end - grp.mine);
        int slot0 = of(grp.send - grp.smine), pair0 = 0, pieces = s.pieces;
        const int in_cut = s.cut * s.pieces * g.HH, whole = (s.pairs - s.cut - s.tail) * g.HH;
        int pair, piece = 0, x;
        it->slot = -1;
        if (r >= in_cut + whole) {  // of the tail
          r -= in_cut + whole;
          slot0 += in_cut;
          pair0 = s.pairs - s.tail;
          pieces = s.tpieces;
        } else if (r >= in_cut) {
          r -= in_cut;
          pair0 = s.cut;
          pieces = 0;
        }
        if (pieces > 0) {
          const int each = pieces * g.HH;
          pair = r / each;
          const int y = r - pair * each;
          piece = y / g.HH;
          x = y - piece * g.HH;
          it->slot = slot0 + (pair * g.HH + x) * pieces + piece;
        } else {
          pair = r / g.HH;
          x = r - pair * g.HH;
        }
        pair += pair0;
        const int vh = g.VH == 2 ? x & 1 : 0;
        x >>= g.VH - 1;
        const int hb = x % g.HB;
        it->end = 0;
        it->hk = x / g.HB;
        it->h0 = it->hk * g.G + (hb << g.lgp);
        const int per = kTile >> g.lgp;
        it->tok = (s.pairs - 1 - pair) * 2 * per;
        it->q0 = s.q0 + it->tok;
        it->nq = s.nq;
        it->nk = s.nk;
        it->k0 = s.k0;
        it->v0 = vh * kVWidth;
        it->dv = min(g.a.Dv - it->v0, kVWidth);
        it->lim = visible(it->tok, s.nq, s.nk);
        // (lo of hi + lo may be 0: no infinity may meet it either)
        it->jm = it->lim <= kShort ? 0 : it->lim / kTile;
        int j1 = 1 << 30;
        it->j0 = 0;
        if (it->slot >= 0) {
          const int N = s.tiles_of(g.lgpair, pair), used = s.used(N, pair, cuts.c), width = (N + used - 1) / used;
          joined = piece == 0 ? used : 0;
          if (piece >= used) return 2;
          it->j0 = piece * width;
          j1 = it->j0 + width;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int first_tok = it->tok + t * per;
          const int last = first_tok + min(per, s.nq - first_tok) - 1;
          const int n = first_tok < s.nq ? tiles_over(visible(last, s.nq, s.nk)) : 0;
          it->n[t] = max(min(n, j1) - it->j0, 0);
        }
        return 1;
      }
      if (!grp.next(g, cuts, lane)) return 0;
    }
  }
};

// kLong: a sequence may have more than kLongKeys keys.
template <bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    k_prompt_attn(const __grid_constant__ Maps maps, const __grid_constant__ Geo g) {
  extern __shared__ uint8_t smraw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  const PromptAttnParams& a = g.a;
  const uint32_t qsm = (uint32_t)uniform((int)smem_u32(base));                              // [2][nkc] chunks
  const uint32_t rsm = qsm + 2 * g.nkc * kChunkBytes;               // [ring] chunks
  uint8_t* rptr = base + 2 * g.nkc * kChunkBytes;
  Smem& sm = *reinterpret_cast<Smem*>(rptr + g.ring * kChunkBytes);
  const int lane = threadIdx.x & 31;
  const int warp = uniform(threadIdx.x >> 5);
  launch_dependents();
  if (threadIdx.x == 0) {
    sm.abort = sm.vissued = sm.vclean[0] = sm.vclean[1] = 0;
    sm.fills = sm.qfills[0] = sm.qfills[1] = 0;
    for (int i = 0; i < g.ring; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qfull[i], 1);
      mbar_init(&sm.qempty[i], 1);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pfull[i][0], 4);
      mbar_init(&sm.pfull[i][1], 4);
      mbar_init(&sm.ofull[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.ifull[i], 1);
      mbar_init(&sm.iempty[i], kReaders);
    }
    for (int i = 0; i < 4 * kSlots; ++i) sm.odd[i / (2 * kSlots)][i % (2 * kSlots)] = 0;
    mbar_init(&sm.done, 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
  grid_dependency_wait();
  if (g.slots > 0) {
    add_up(g, sm, warp, lane);
    __syncthreads();
  }

  const int per = kTile >> g.lgp;  // tokens of a tile
  const int nkc = g.nkc;
  // The next item's descriptor, for every warp but the producer's: it may be
  // read until item_done().
  int islot = 0;
  uint32_t iphase = 0;
  auto wait_item = [&]() -> bool {
    if (!warp_wait(smem_u32(&sm.ifull[islot]), iphase, &sm.abort, kItemNs)) {
      if (lane == 0) fail(sm, a.status);
      return false;
    }
    return uniform(sm.item[islot].end) == 0;
  };
  auto item_done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.iempty[islot]);
    if (++islot == kSlots) {
      islot = 0;
      iphase ^= 1;
    }
  };
  // A copy of what the issuer and the readers of V need, known to be the same in
  // every lane: descriptors made from these stay in uniform registers, and an MMA
  // is one instruction (without it the 32 MMAs of a key tile took ~4,500 cycles).
  auto next_item = [&](Item& it) -> bool {
    if (!wait_item()) return false;
    const Item& x = sm.item[islot];
    it.tok = uniform(x.tok);
    it.nq = uniform(x.nq);
    it.nk = uniform(x.nk);
    it.dv = uniform(x.dv);
    it.n[0] = uniform(x.n[0]);
    it.n[1] = uniform(x.n[1]);
    it.lim = uniform(x.lim);
    it.jm = uniform(x.jm);
    it.j0 = uniform(x.j0);
    item_done();
    return true;
  };

  if (warp >= 8) {
    if (warp == 8) {
      // --------------------------------------------------------- producer --
      Finder f;
      f.init(g, sm, lane);
      int rs = 0;
      uint32_t rphase = 1;  // an empty ring's barriers have completed "phase 1"
      int nfill = 0, nv = 0, nq[2] = {0, 0};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        Item it;
        int found;
        do {
          int at = 0;
          if (lane == 0) at = atomicAdd(g.next, 1);
          found = f.find(g, uniform(at), lane, &it);
        } while (found == 2);
        const bool have = found == 1;
        it.end = have ? 0 : 1;
        const int s = k % kSlots;
        if (!warp_wait(smem_u32(&sm.iempty[s]), ((k / kSlots) & 1) ^ 1, &sm.abort)) { ok = false; break; }
        if (lane == 0) {
          sm.item[s] = it;
          mbar_arrive(&sm.ifull[s]);
          if (have && it.slot >= 0 && f.joined > 0) {
            const int i = atomicAdd(g.joins, 1);
            if (i < g.slots) g.join[i] = Join{it.slot, f.joined, it.q0, it.nq - it.tok, it.h0, it.v0, {0, 0}};
          }
        }
        __syncwarp();
        if (!have) break;
        const int N = max(it.n[0], it.n[1]);
        const int nvc = (it.dv + kChunk - 1) / kChunk;
        auto fill = [&](const CUtensorMap* map, int x, int y, int z) {
          if (!warp_wait(smem_u32(&sm.empty[rs]), rphase, &sm.abort)) return false;
          const uint32_t bar = smem_u32(&sm.full[rs]);
          expect_elected(bar, kChunkBytes);
          tma_3d(rsm + rs * kChunkBytes, map, bar, x, y, z);
          ++nfill;
          if (++rs == g.ring) {
            rs = 0;
            rphase ^= 1;
          }
          return true;
        };
        _Pragma("unroll")
          for (int t = 0; t < 2; ++t) {
            if (!ok) break;
          if (it.n[t] == 0) continue;
          if (!warp_wait(smem_u32(&sm.qempty[t]), (nq[t] & 1) ^ 1, &sm.abort)) { ok = false; break; }
          const uint32_t bar = smem_u32(&sm.qfull[t]);
          expect_elected(bar, nkc * kChunkBytes);
          for (int c = 0; c < nkc; ++c)
            tma_3d(qsm + (t * nkc + c) * kChunkBytes, &maps.q, bar, kChunk * c, it.h0, it.q0 + t * per);
          ++nq[t];
        }
        for (int j = 0; j < N && ok; ++j) {
          for (int c = 0; c < nkc && ok; ++c) ok = fill(&maps.k, kChunk * c, it.hk, it.k0 + kTile * (it.j0 + j));
          for (int c = 0; c < nvc && ok; ++c) ok = fill(&maps.v, it.v0 + kChunk * c, it.hk, it.k0 + kTile * (it.j0 + j));
          if (it.j0 + j >= it.jm) {
            ++nv;
            __syncwarp();
            if (lane == 0) count_set(&sm.vissued, nv);
          }
        }
      }
      if (lane == 0) {
        sm.fills = nfill;
        sm.qfills[0] = nq[0];
        sm.qfills[1] = nq[1];
        if (!ok) fail(sm, a.status);
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- issuer --
      const uint32_t id_s = instr_desc(128, 128, 1, 1, 0, 0);
      const uint64_t dq = smem_desc(qsm, 16, 1024, kSwizzle128B);
      const uint64_t dk = smem_desc(rsm, 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(rsm, kChunkBytes, 1024, kSwizzle128B);  // blocks of 64 columns, chunk after chunk
      constexpr int kStep = kChunkBytes / 16;  // a chunk, in descriptor units
      int rs = 0;          // the ring's next chunk
      uint32_t rphase = 0;
      auto advance = [&](int n) {
        rs += n;
        if (rs >= g.ring) {
          rs -= g.ring;
          rphase ^= 1;
        }
      };
      uint32_t qphase = 0, pphase = 0;  // bit X
      int nclean = 0;
      bool ok = true;
      Item it;
      while (ok && next_item(it)) {
        const int N = max(it.n[0], it.n[1]);
        const int nvc = (it.dv + kChunk - 1) / kChunk;
        const bool brief = it.lim <= kShort;
        const int jm = max(it.jm - it.j0, 0);  // from this tile on V is looked through
        int vs = 0;                     // first chunk of V of the tile before
        uint32_t vturn = 0;             // ... and its phase
        // waits for chunks s .. s + n - 1 of the ring, s being in phase `turn`
        auto landed = [&](int s, int n, uint32_t turn) {
          bool all = true;
#pragma unroll 1
          for (int c = 0; c < n && all; ++c, ++s) {
            if (s == g.ring) {
              s = 0;
              turn ^= 1;
            }
            all = warp_wait(smem_u32(&sm.full[s]), turn, &sm.abort);
          }
          return all;
        };
        auto release = [&](int s, int n) {
#pragma unroll 1
          for (int c = 0; c < n; ++c, ++s) {
            if (s == g.ring) s = 0;
            commit_elected(smem_u32(&sm.empty[s]));
          }
        };
#pragma unroll 1
        for (int j = 0; j <= N && ok; ++j) {
          // this tile's K is chunks rs .. rs + nkc - 1, its V the nvc behind
          if (j > 0) {
            ok = landed(vs, nvc, vturn);
            if (ok && j - 1 >= jm) {
              ++nclean;
              ok = count_wait(&sm.vclean[0], nclean, &sm.abort) && count_wait(&sm.vclean[1], nclean, &sm.abort);
            }
          }
          if (!ok) break;
          bool kready = false;
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int n = t ? it.n[1] : it.n[0];
            const uint32_t ts = tbase + kColS + 128 * t;
            if (j > 0 && j - 1 < n) {  // O_X += P_X V of the tile before
              const uint32_t d = tbase + kColO + 128 * t;
              const bool split = vs + nvc > g.ring;  // the two chunks lie at the ring's ends
              const uint32_t id = (uint32_t)uniform((int)instr_desc(128, split ? kChunk : kChunk * nvc, 1, 1, 0, 1));
#pragma unroll 1
              for (int h = 1; h >= 0; --h) {  // 64 keys at a time, as their weights are ready
                if (!warp_wait(smem_u32(&sm.pfull[t][h]), pphase >> t & 1, &sm.abort)) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int part = 0; part < (split ? 2 : 1); ++part) {
                  const uint64_t vb = dv + (uint64_t)(uint32_t)uniform(kStep * (part ? 0 : vs) + 512 * h);
                  const uint32_t p = ts + 64 * h;
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mma_ts(d + kChunk * part, p + 8 * k, vb + 128 * k, id, (j > 1 || h == 0 || k > 0) ? 1 : 0);
                  if (brief) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_ts(d + kChunk * part, p + 32 + 8 * k, vb + 128 * k, id, 1);
                  }
                }
              }
              if (!ok) break;
              pphase ^= 1u << t;
              if (j == n) commit_elected(smem_u32(&sm.ofull[t]));
              if (t == 1 || j - 1 >= it.n[1]) release(vs, nvc);  // V of the tile before is done with
            }
            if (j < n) {  // S_X of this tile
              if (j == 0) {
                if (!warp_wait(smem_u32(&sm.qfull[t]), qphase >> t & 1, &sm.abort)) { ok = false; break; }
                qphase ^= 1u << t;
              }
              int s = rs;
#pragma unroll 1
              for (int c = 0; c < nkc; ++c, ++s) {
                if (s == g.ring) s = 0;
                if (!kready && !warp_wait(smem_u32(&sm.full[s]), s < rs ? rphase ^ 1 : rphase, &sm.abort)) { ok = false; break; }
                tc_fence_after();
                const uint64_t qa = dq + (uint64_t)(uint32_t)uniform(kStep * (nkc * t + c));
                const uint64_t kb = dk + (uint64_t)(uint32_t)uniform(kStep * s);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ss(ts, qa + 2 * k, kb + 2 * k, id_s, (c > 0 || k > 0) ? 1 : 0);
                if (t == 1 || j >= it.n[1]) commit_elected(smem_u32(&sm.empty[s]));  // the chunk's last use
              }
              if (!ok) break;
              kready = true;
              commit_elected(smem_u32(&sm.sfull[t]));
              if (j + 1 == n) commit_elected(smem_u32(&sm.qempty[t]));
            }
          }
          if (!ok) break;
          if (j < N) {
            advance(nkc);
            vs = rs;
            vturn = rphase;
            advance(nvc);
          }
        }
      }
      if (!ok && lane == 0) fail(sm, a.status);
      commit_elected(smem_u32(&sm.done));
    } else {
      // ------------------------------------------------ V of partial tiles --
      int rs = 0, k = 0, nv = 0;
      uint32_t rphase = 0;
      bool ok = true;
      Item it;
      while (ok && next_item(it)) {
        const int N = max(it.n[0], it.n[1]);
        const int nvc = (it.dv + kChunk - 1) / kChunk;
        const int jm = max(it.jm - it.j0, 0);
        int* odds = sm.odd[warp - 10];
        const int slot = k % (2 * kSlots);
        ++k;
        // Cleared two items ahead of its use.  It was item k - 6's: every warp
        // has read descriptor k - 4, so every softmax warp is done with k - 5.
        if (lane == 0) odds[(slot + 2) % (2 * kSlots)] = 0;
        auto step = [&] {
          if (++rs == g.ring) {
            rs = 0;
            rphase ^= 1;
          }
        };
        const int seen = visible(it.tok + min(2 * per, it.nq - it.tok) - 1, it.nq, it.nk);
        for (int j = 0; j < N && ok; ++j) {
          for (int c = 0; c < nkc; ++c) step();
          bool odd = false;
          // the copies of this lap of the ring are under way: only then does a
          // chunk's barrier tell this lap's completion from one before
          if (j >= jm && !count_wait(&sm.vissued, ++nv, &sm.abort, kItemNs)) { ok = false; break; }
          for (int c = 0; c < nvc && ok; ++c, step()) {
            if (j < jm) continue;
            if (!warp_wait(smem_u32(&sm.full[rs]), rphase, &sm.abort)) { ok = false; break; }
            uint4* chunk = reinterpret_cast<uint4*>(rptr + rs * kChunkBytes) + lane;  // 8 lanes a row of 128 bytes
            const int rows = min(seen - kTile * (it.j0 + j), kTile);  // of the tile that some row sees
            // One warp takes even groups of four rows, the other odd ones, eight at a
            // time: a sum of products with 0 is NaN if any element was none of the
            // finite ones (with every element looked at by itself, items of four tiles
            // took 43 us, 39 so).
#pragma unroll 1
            for (int i0 = warp - 10; i0 < kTile / 4; i0 += 16) {
              uint4 x[8];
              __nv_bfloat162 sum[4];
#pragma unroll
              for (int u = 0; u < 8; ++u)
                x[u] = 4 * (i0 + 2 * u) + (lane >> 3) < rows ? chunk[32 * (i0 + 2 * u)] : make_uint4(0, 0, 0, 0);
              const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[e] = zero;
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), zero, sum[e]);
              }
              const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
              const bool bad = __hisnan(all.x) || __hisnan(all.y);
              if (__any_sync(0xffffffffu, bad) || rows < kTile) {
                odd |= bad;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                  auto scrub = [](uint32_t w) {
                    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
                    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
                    return w;
                  };
                  chunk[32 * (i0 + 2 * u)] = make_uint4(scrub(x[u].x), scrub(x[u].y), scrub(x[u].z), scrub(x[u].w));
                }
              }
            }
          }
          if (!ok) break;
          if (j >= jm) {
            if (odd) odds[slot] = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) count_set(&sm.vclean[warp - 10], nv);
          }
        }
      }
      if (!ok && lane == 0) fail(sm, a.status);
    }
  } else {
    // ------------------------------------------------------------- softmax --
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lanes + kColS + 128 * t, to = tbase + lanes + kColO + 128 * t;
    const float c = a.scale_log2;
    uint32_t sphase = 0, ophase = 0;
    bool ok = true;
    int k = 0;
    for (; ok && wait_item(); item_done()) {
      const Item& it = sm.item[islot];
      auto token = [&] { return it.tok + t * per + (row >> g.lgp); };
      const bool brief = it.lim <= kShort;
      // (pass: what the maximum is raised for; -inf: for anything)
      float m = -INFINITY, pass = -INFINITY, l = 0.0f;
      float fa = 1.0f;    // factor of what the workspace holds of O
      bool kept = false;  // ... if it holds any
      auto sum_at = [&](int col) {  // of this row, four columns at a time
        return reinterpret_cast<float4*>(g.acc) + ((size_t)blockIdx.x * (kVWidth / 4) + col / 4) * kSlotRows + kTile * t + row;
      };
      // columns of the tile that this row sees
      int see = token() < it.nq ? visible(token(), it.nq, it.nk) - kTile * it.j0 : 0;
#pragma unroll 1
      for (int left = it.n[t], flush = kFlush; left > 0; --left, --flush, see -= kTile) {
        if (!warp_wait(smem_u32(&sm.sfull[t]), sphase, &sm.abort)) { ok = false; break; }
        sphase ^= 1;
        tc_fence_after();
        // All four quarters of a row for its maximum; for the weights the first two
        // are read again (128 scores and the rest do not fit in a thread's 168 registers).
        uint32_t z[2][32];  // quarters 2 and 3
        const bool part = __any_sync(0xffffffffu, see < kTile);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        {
          uint32_t y[2][32];
          tmem_ld_32cols(ts, y[0]);
          tmem_ld_32cols(ts + 32, y[1]);
          tmem_ld_32cols(ts + 64, z[0]);
          tmem_ld_32cols(ts + 96, z[1]);
          tmem_wait_ld();
          if (part) {
            hide(y[0], 0, see);
            hide(y[1], 1, see);
            hide(z[0], 2, see);
            hide(z[1], 3, see);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              mx[q] = max3(mx[q], __uint_as_float(y[q][i]), __uint_as_float(y[q][i + 1]));
              mx[2 + q] = max3(mx[2 + q], __uint_as_float(z[q][i]), __uint_as_float(z[q][i + 1]));
            }
        }
        const float mt = __fmul_rn(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), c);  // (rounded before it meets m)
        float f = 1.0f;
        bool rescale = false, far = false;
        if (__any_sync(0xffffffffu, mt > pass)) {
          bool resc = false;
          if (mt > pass && mt > m) {
            resc = m > -INFINITY;
            if (resc) f = exp2f(m - mt);
            m = mt;
            pass = fabsf(m) > kFar ? -INFINITY : m + kRescaleLog2;
          }
          rescale = __any_sync(0xffffffffu, resc);
          far = __any_sync(0xffffffffu, m > -INFINITY && fabsf(m) > kFar);
        }
        const float mm = m == -INFINITY ? 0.0f : m;
        const uint64_t c2 = pair2(c, c), r2 = pair2(-mm, -mm);
        uint64_t sum[2] = {pair2(kLong ? 0.0f : l * f, 0.0f), pair2(0.0f, 0.0f)};  // (small next to a long l)
        if (kLong && __builtin_expect(flush == 0, 0)) {
          flush = kFlush;
          // (S of this tile came after O of the tiles before)
#pragma unroll 1
          for (int i = 0; 16 * i < it.dv; ++i) {
            uint32_t v[16];
            tmem_ld_16cols(to + 16 * i, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float4* p = sum_at(16 * i + e);
              const float4 a = kept ? *p : make_float4(0.f, 0.f, 0.f, 0.f);
              *p = make_float4(fmaf(a.x, fa, __uint_as_float(v[e])), fmaf(a.y, fa, __uint_as_float(v[e + 1])),
                               fmaf(a.z, fa, __uint_as_float(v[e + 2])), fmaf(a.w, fa, __uint_as_float(v[e + 3])));
              v[e] = v[e + 1] = v[e + 2] = v[e + 3] = 0;
            }
            tmem_st_16cols(to + 16 * i, v);
          }
          tmem_wait_st();
          kept = true;
          fa = 1.0f;
        }
        if (kLong) fa *= f;
        // A quarter's weights over scores that were read: bf16 to columns `at`,
        // what that leaves (short items) 32 behind.
        auto weigh = [&](const uint32_t (&x)[32], uint32_t at, auto both, auto apart) {
#pragma unroll
          for (int i0 = 0; i0 < 32; i0 += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 e;
              if (decltype(apart)::value)
                e = make_float2(__fsub_rn(__fmul_rn(__uint_as_float(x[i0 + 2 * i]), c), mm),
                                __fsub_rn(__fmul_rn(__uint_as_float(x[i0 + 2 * i + 1]), c), mm));
              else
                e = split2(fma2(pair2(x[i0 + 2 * i], x[i0 + 2 * i + 1]), c2, r2));
              const float e0 = ex2_approx(e.x), e1 = ex2_approx(e.y);
              sum[i & 1] = add2(sum[i & 1], pair2(e0, e1));
              if (decltype(both)::value) {
                // hi cut off, so that lo is below 2^-7 and off by half a step of it, 2^-16
                const uint32_t u0 = __float_as_uint(e0), u1 = __float_as_uint(e1);
                hi[i] = __byte_perm(u0, u1, 0x7632);
                const float2 d = split2(fma2(pair2(__uint_as_float(u0 & 0xffff0000u), __uint_as_float(u1 & 0xffff0000u)),
                                             pair2(-1.0f, -1.0f), pair2(e0, e1)));
                const __nv_bfloat162 l2 = __floats2bfloat162_rn(d.x, d.y);
                lo[i] = *reinterpret_cast<const uint32_t*>(&l2);
              } else {
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(e0, e1);
                hi[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
            }
            tmem_st_8cols(at + i0 / 2, hi);
            if (decltype(both)::value) tmem_st_8cols(at + 32 + i0 / 2, lo);
          }
        };
        auto hand_over = [&](int h) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.pfull[t][h]);
        };
        // The second half of the keys first: its weights' products run while the
        // first half's are made.
        auto halves = [&](auto both, auto apart) {
#pragma unroll 1
          for (int h = 1;; h = 0) {
            weigh(z[0], ts + 64 * h, both, apart);
            weigh(z[1], ts + 64 * h + 16, both, apart);
            if (h == 0) break;
            if (rescale) {
              // O of the tiles before (S of this tile came after it)
#pragma unroll 1
              for (int i = 0; 16 * i < it.dv; ++i) {
                uint32_t v[16];
                tmem_ld_16cols(to + 16 * i, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                tmem_st_16cols(to + 16 * i, v);
              }
            }
            tmem_ld_32cols(ts, z[0]);
            tmem_ld_32cols(ts + 32, z[1]);
            hand_over(1);
            tmem_wait_ld();
            if (part) {
              hide(z[0], 0, see);
              hide(z[1], 1, see);
            }
          }
          hand_over(0);
        };
        // (in this order: with the rare case first long prompts take 2 % more)
        if (__builtin_expect(!far && !brief, 1)) {
          halves(std::false_type{}, std::false_type{});
        } else if (__builtin_expect(!far, 1)) {
          halves(std::true_type{}, std::false_type{});
        } else {
          brief ? halves(std::true_type{}, std::true_type{}) : halves(std::false_type{}, std::true_type{});
        }
        const float2 s0 = split2(add2(sum[0], sum[1]));
        l = kLong ? fmaf(l, f, s0.x + s0.y) : s0.x + s0.y;
      }
      if (!ok) break;
      // ---- O out of TMEM
      const bool any = it.n[t] > 0;
      const int slot = k % (2 * kSlots), tok = token();
      const int lim = tok < it.nq ? visible(tok, it.nq, it.nk) : 0;
      ++k;
      if (any) {
        if (!warp_wait(smem_u32(&sm.ofull[t]), ophase, &sm.abort)) { ok = false; break; }
        ophase ^= 1;
        tc_fence_after();
      }
      const bool mine = tok < it.nq;
      const int head = it.h0 + (row & ((1 << g.lgp) - 1));
      const long long tr = (long long)it.q0 + t * per + (row >> g.lgp);
      const int slot_out = it.slot;  // of a partial result
      const float inv = l == 0.0f ? 0.0f : slot_out >= 0 ? 1.0f : 1.0f / l;
      const bool odd = (sm.odd[0][slot] | sm.odd[1][slot]) != 0;
      __nv_bfloat16* out = a.out + tr * a.o_ts + (long long)head * a.o_hs + it.v0;
#pragma unroll 1
      for (int q = 0; 32 * q < it.dv; ++q) {
        uint32_t v[32];
        if (any) {
          tmem_ld_32cols(to + 32 * q, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if (kLong && __builtin_expect(kept, 0)) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            if (32 * q + i >= it.dv) break;
            const float4 a = *sum_at(32 * q + i);
            v[i] = __float_as_uint(fmaf(a.x, fa, __uint_as_float(v[i])));
            v[i + 1] = __float_as_uint(fmaf(a.y, fa, __uint_as_float(v[i + 1])));
            v[i + 2] = __float_as_uint(fmaf(a.z, fa, __uint_as_float(v[i + 2])));
            v[i + 3] = __float_as_uint(fmaf(a.w, fa, __uint_as_float(v[i + 3])));
          }
        }
        // (as few instructions as may be, for they run once an item and come from
        // memory: a multiplication and a selection for each element took 608 items of
        // 256 rows 51 us, this 45; 64 or all 128 columns at once 46 and 51)
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 y = split2(fma2(pair2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), pair2(inv, inv),
                                       pair2(-0.0f, -0.0f)));
          x[i] = y.x;
          x[i + 1] = y.y;
        }
        if (odd && mine) {
          // infinities and NaN that were kept out of the products
          const int p1 = (int)min((unsigned)lim, (unsigned)kTile * (unsigned)(it.j0 + it.n[t]));
          for (int p = max(it.jm, it.j0) * kTile; p < p1; ++p) {
            const __nv_bfloat16* vr = a.v + (long long)(it.k0 + p) * a.v_ts + (long long)it.hk * a.v_hs + it.v0;
            for (int i = 0; i < 32; ++i)
              if (32 * q + i < it.dv) {
                const float y = __bfloat162float(vr[32 * q + i]);
                if (!isfinite(y)) x[i] += y;
              }
          }
        }
        if (mine && slot_out >= 0) {
          float4* po = reinterpret_cast<float4*>(g.po) + ((size_t)slot_out * (kVWidth / 4) + 8 * q) * kSlotRows + kTile * t + row;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (32 * q + 4 * i < it.dv)
              po[(size_t)i * kSlotRows] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        } else if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (32 * q + 8 * i >= it.dv) break;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[8 * i + 2 * e], x[8 * i + 2 * e + 1]);
              w[e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            *reinterpret_cast<uint4*>(out + 32 * q + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
      if (mine && slot_out >= 0) g.ml[(size_t)slot_out * kSlotRows + kTile * t + row] = make_float2(m, l);
      if (mine && slot_out < 0 && a.lse && it.v0 == 0)
        a.lse[tr * a.Hq + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
    if (!ok && lane == 0) fail(sm, a.status);
  }

  __syncthreads();
  if (warp == 0) {
    int never = 0;
    pair_wait(smem_u32(&sm.done), 0, &never, 100000000ull);  // the products are done
    if (sm.abort) {  // and, after a failure, the copies in flight
      for (int i = 0; i < g.ring; ++i) {
        const int n = (sm.fills - i + g.ring - 1) / g.ring;
        if (n > 0) pair_wait(smem_u32(&sm.full[i]), (n - 1) & 1, &never, 10000000ull);
      }
      for (int t = 0; t < 2; ++t)
        if (sm.qfills[t] > 0) pair_wait(smem_u32(&sm.qfull[t]), (sm.qfills[t] - 1) & 1, &never, 10000000ull);
    }
    if (lane == 0) {  // the last CTA leaves both counters at zero for the next call
      __threadfence();
      if (atomicAdd(g.left, 1) == (int)gridDim.x - 1) {
        *g.next = 0;
        *g.left = 0;
        __threadfence();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// The join of the pieces of cut items: a block takes 32 rows of an item at a time
// (a lane each), a warp every eighth group of four columns.
__global__ void __launch_bounds__(256) k_prompt_merge(const __grid_constant__ Geo g) {
  constexpr int kBatch = 2;
  const PromptAttnParams& a = g.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  launch_dependents();
  const int joins = min(__ldcg(g.joins), g.slots);
  // unit u: item u / 8, 32 rows of it
  for (int u = blockIdx.x; u < 8 * joins; u += gridDim.x) {
    const int4* jp = reinterpret_cast<const int4*>(g.join + (u >> 3));
    const int4 j0 = __ldcg(jp), j1 = __ldcg(jp + 1);
    const int slot = j0.x, used = j0.y, per = kTile >> g.lgp;
    const int row = 32 * (u & 7) + lane;
    const int tok = (row / kTile) * per + ((row % kTile) >> g.lgp);
    const int head = j1.x + (row & ((1 << g.lgp) - 1));
    if (tok >= j0.w) continue;  // (a whole warp's or some lanes': no lane is waited for below)
    const long long tr = (long long)j0.z + tok;
    const int v0 = j1.y, dv = min(a.Dv - v0, kVWidth);
    const float2* ml = g.ml + (size_t)slot * kSlotRows + row;
    float M = -INFINITY, l_sum = 0.0f;
#pragma unroll 4
    for (int i = 0; i < used; ++i) M = fmaxf(M, __ldcg(&ml[(size_t)i * kSlotRows]).x);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll 4
    for (int i = 0; i < used; ++i) {
      const float2 st = __ldcg(&ml[(size_t)i * kSlotRows]);
      if (st.y != 0.0f) l_sum = fmaf(st.y, exp2f(st.x - ref), l_sum);
    }
    const float inv = l_sum == 0.0f ? 0.0f : 1.0f / l_sum;
    // the warp's four groups of columns at once, two partials in flight
    constexpr int kGroups = kVWidth / 4 / 8;
    const float4* po = reinterpret_cast<const float4*>(g.po) + ((size_t)slot * (kVWidth / 4) + warp) * kSlotRows + row;
    float4 acc[kGroups];
#pragma unroll
    for (int d = 0; d < kGroups; ++d) acc[d] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < used; i0 += kBatch) {
      float2 st[kBatch];
      float4 v[kBatch][kGroups];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        st[e] = make_float2(-INFINITY, 0.0f);
        if (i0 + e < used) st[e] = __ldcg(&ml[(size_t)(i0 + e) * kSlotRows]);
#pragma unroll
        for (int d = 0; d < kGroups; ++d) {
          v[e][d] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + e < used && 4 * (warp + 8 * d) < dv)
            v[e][d] = __ldcg(po + ((size_t)(i0 + e) * (kVWidth / 4) + 8 * d) * kSlotRows);
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (st[e].y == 0.0f) continue;  // the row sees no key of the piece
        const float w = exp2f(st[e].x - ref);
#pragma unroll
        for (int d = 0; d < kGroups; ++d) {
          acc[d].x = fmaf(v[e][d].x, w, acc[d].x);
          acc[d].y = fmaf(v[e][d].y, w, acc[d].y);
          acc[d].z = fmaf(v[e][d].z, w, acc[d].z);
          acc[d].w = fmaf(v[e][d].w, w, acc[d].w);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < kGroups; ++d) {
      const int x0 = 4 * (warp + 8 * d);
      if (x0 >= dv) break;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[d].x * inv, acc[d].y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[d].z * inv, acc[d].w * inv);
      *reinterpret_cast<uint2*>(a.out + tr * a.o_ts + (long long)head * a.o_hs + v0 + x0) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (warp == 0 && a.lse && v0 == 0)
      a.lse[tr * a.Hq + head] = l_sum == 0.0f ? -INFINITY : (M + log2f(l_sum)) * 0.6931471805599453f;
  }
  // the last block leaves both counters at zero for the next call
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(g.jleft, 1) == (int)gridDim.x - 1) {
    *g.joins = 0;
    *g.jleft = 0;
  }
}

// Partial results that a call may need: none where there are items for every SM
// several times over, else at most about two pieces per SM and one remainder each.
constexpr int kMaxSlots = 384;
struct Shape {
  int G, lgp, HB, VH;
  long long HH;     // items per pair of tiles
  long long items;  // at most
};
Shape shape_of(int B, int Nq, int Hq, int Hk, int Dv) {
  Shape s{};
  s.G = Hq / Hk;
  while (s.lgp < 7 && s.G % (2 << s.lgp) == 0) ++s.lgp;
  s.HB = s.G >> s.lgp;
  s.VH = (Dv + kVWidth - 1) / kVWidth;
  s.HH = (long long)Hk * s.HB * s.VH;
  const long long pairs = (long long)Nq / (2 * kTile >> s.lgp) + B;
  s.items = pairs > (1LL << 62) / s.HH ? 1LL << 62 : pairs * s.HH;
  return s;
}
bool may_cut(const Shape& s) { return s.items < 12LL * sm_count(); }
size_t ml_bytes() { return sizeof(float2) * kMaxSlots * kSlotRows; }

int ring_of(int nkc) {
  const int room = 227 * 1024 - 1024 - (int)sizeof(Smem) - 2 * nkc * kChunkBytes;
  return std::min(kMaxRing, room / kChunkBytes);
}

}  // namespace

size_t prompt_attn_ws() {
  return kWsHeader + ml_bytes() + sizeof(Join) * kMaxSlots + sizeof(float) * (kMaxSlots + kMaxCtas) * kSlotRows * kVWidth;
}

size_t prompt_attn_uses(int B, int Nq, int Nk, int Hq, int Hk, int Dv) {
  return may_cut(shape_of(B, Nq, Hq, Hk, Dv)) || Nk > kLongKeys ? prompt_attn_ws() : kWsHeader;
}

int launch_prompt_attn(const PromptAttnParams& p, void* ws, cudaStream_t s) {
  Geo g{};
  g.a = p;
  const Shape sh = shape_of(p.B, p.Nq, p.Hq, p.Hk, p.Dv);
  if (sh.items > 0x7fff0000LL)
    return set_error(DSA_ERR_UNSUPPORTED, "prompt_attn: rows beyond 2^31 pairs of tiles of 128");
  g.G = sh.G;
  g.lgp = sh.lgp;
  g.HB = sh.HB;
  g.lgpair = 8 - sh.lgp;
  g.VH = sh.VH;
  g.HH = (int)sh.HH;
  const int sms = std::min(sm_count(), kMaxCtas);
  g.ctas = (int)std::min<long long>(sms, sh.items);
  g.many = sh.items > sms;
  // Whether anything may be cut: for one sequence its lengths say so, several may
  // have any (but none more keys than there are).  Whole prompts of one and a half
  // items for every SM and more even out by themselves, the small ones coming last;
  // the join's launch would cost them ~5 us.
  bool cut = may_cut(sh) && ((long long)p.Nk + kTile - 1) / kTile >= 3 * kMinPiece &&
             (2 * sh.items < 3LL * sms || p.Nk >= 2LL * p.Nq);
  if (cut && p.B == 1) {
    Seq one{};
    one.nq = p.Nq;
    one.nk = p.Nk;
    one.shape(g.lgpair);
    const long long items = (long long)one.pairs * g.HH;
    const int rest = (int)(items % sms), tail = std::min((rest + g.HH - 1) / g.HH, one.pairs);
    // (three tiles less on the longest item pay for the join)
    cut = one.most >= 2 * piece_of(one.work(g.lgpair), g.HH, sms) + 3 ||
          (tail > 0 && cut_tail(items, sms, rest, one.tiles_of(g.lgpair, one.pairs - tail)));
  }
  g.ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(ws) + kWsHeader);
  g.join = reinterpret_cast<Join*>(reinterpret_cast<char*>(ws) + kWsHeader + ml_bytes());
  g.po = reinterpret_cast<float*>(g.join + kMaxSlots);
  g.acc = g.po + (size_t)kMaxSlots * kSlotRows * kVWidth;
  if (cut) {
    g.slots = kMaxSlots;
    g.ctas = sms;
  }
  g.nkc = (p.Dk + kChunk - 1) / kChunk;
  g.ring = ring_of(g.nkc);
  int* counters = reinterpret_cast<int*>(reinterpret_cast<char*>(ws) + kPromptCounters);
  g.next = counters;
  g.left = counters + 8;
  g.joins = counters + 16;
  g.jleft = counters + 24;
  Maps m{};
  int rc = make_tmap_heads(&m.q, p.q, p.Dk, p.Hq, p.Nq, p.q_hs, p.q_ts, kChunk, 1u << g.lgp, kTile >> g.lgp);
  // no keys at all: nothing is loaded, the maps only have to exist
  const void *k = p.Nk > 0 ? p.k : p.q, *v = p.Nk > 0 ? p.v : p.q;
  if (!rc) rc = make_tmap_heads(&m.k, k, p.Dk, p.Hk, p.Nk, p.k_hs, p.k_ts, kChunk, 1, kTile);
  if (!rc) rc = make_tmap_heads(&m.v, v, p.Dv, p.Hk, p.Nk, p.v_hs, p.v_ts, kChunk, 1, kTile);
  if (rc) return rc;
  const int smem = 1024 + (2 * g.nkc + g.ring) * kChunkBytes + (int)sizeof(Smem);
  const auto kernel = p.Nk > kLongKeys ? k_prompt_attn<true> : k_prompt_attn<false>;
  rc = ensure_dynamic_smem((const void*)kernel, smem, "prompt_attn");
  if (rc) return rc;
  cudaError_t e = launch_pdl(kernel, dim3((unsigned)g.ctas), dim3(kThreads), (size_t)smem, s, m, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  rc = check_launch("prompt_attn");
  if (rc || g.slots == 0) return rc;
  e = launch_pdl(k_prompt_merge, dim3((unsigned)(4 * sm_count())), dim3(256), 0, s, g);
  count_launch();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, cudaGetErrorString(e));
  return check_launch("prompt_attn merge");
}

}  // namespace dsa
