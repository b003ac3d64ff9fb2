// fa_fwd_paged.cuh -- tensor-core attention of each sequence's newest tokens
// over a cache in pages, for sm_103a: the kernel of fa_fwd_paged.cu (bf16 pages)
// and of fa_fwd_paged_fp8.cu (pages of e4m3 codes, KV8 below).
//
// Method ("FlashAttention: Faster Attention Without Dropping a Single
// Interaction"): S = scale Q K^T (+ ALiBi), O = softmax(S) V by tiles of 128
// keys with a running reference max m and sum l; parts of a row's keys are
// merged with the pages' (m, l, O) rule (Key design 2):
//     m = max_s m_s,  l = sum_s 2^(m_s - m) l_s,  O = sum_s 2^(m_s - m) O_s / l.
//
// Rows.  The query heads of one kv head share its keys, so they share tiles:
// row r of a 128-row tile is token r / group, head r % group (a TMA box of
// group heads x 128 / group tokens).  An item is (sequence, kv head, block of
// two such tiles): up to 256 rows against the keys any of them sees.
//   two tiles   both run over the same K/V tiles, each with its own S, P, O in
//               TMEM: one tile's softmax overlaps the other's products.
//               Bound by the products: 32 of them take 2600 of the about 3400
//               cycles of a step of 128 keys (two chunks of 2048 tokens over
//               31k keys, 32 heads on 8, d = 128: 1535-1575 us on the GPU by
//               the box, 1320-1350 TFLOP/s, 70 % of the measured cuBLAS rate;
//               1680-1745 us in a long loop of calls, where the power cap lowers
//               the clock).  What an item costs beside its steps, 14600 cycles
//               of first loads, first softmax and epilogue, shows where items
//               are short (8192 tokens from scratch: 480-510 us, 1110 TFLOP/s).
//               P is rounded to bf16 once, as in the dense forward: two parts
//               would be half as many products again.  O is then off by 0.0023
//               of its norm against 64 bits, of which 0.0017 are O's own bf16.
//   one tile    (a token or a few per sequence) the same two streams share the
//               rows and take the key tiles in turn; their O and (m, l) are
//               merged at the end.  64 KB of K/V per 128 keys come from HBM
//               (1.4 us of one SM's share at d = 128) against 0.8 us of
//               products, so HBM bounds it, and the tensor cores have time to
//               take P as two bf16 parts (high and low, 16 bits of P instead
//               of 8): O then carries its own rounding only (0.0016).  16 caches
//               of 1k-32k tokens, one new token each: 161 us, 6.24 TB/s, 92 % of
//               the measured copy rate.  A chunk's last block of at most one tile
//               has these rows too, so its rows are closer than those before it.
//
// Work.  Lengths are known on the device alone (so a captured call can be
// replayed with others).  Every CTA, one per SM, adds up the key tiles of all
// items, weighed by their measured times (a tile of a two-tile item 9, of
// another 8; what an item costs beside its tiles 36 and 16: without that the
// SMs with the short items ended last, 658 us instead of 490 for the 8192
// tokens; measured at d = 128 and with items of one kind at a time, where the
// other cases took no figures of their own), and takes an equal run of this one line.  A run begins and ends
// inside items; such parts go to the workspace, two at most per CTA, and
// paged_merge_kernel joins an item's parts in a fixed order.  No SM waits for
// a long sequence and nothing depends on timing: the result is the same from
// run to run.  Plan, first loads and merge are what a short call costs (one
// sequence of 777 tokens, 16 heads of 64: 15.5 us on the GPU, where a bare
// launch takes about 3; some 30 us through the Python call).
//
// Roles:
//   warp 10    walker: finds the CTA's items one after the other and passes
//              them on through a ring of four, so that no other role waits
//              for the lengths and the divisions this takes.
//   warp 8     TMA producer: Q of an item, then per step one slot with K of
//              this step's tile and V of the step before.  A tile is 128 /
//              page_size boxes, one lane each, at the pages the table names;
//              pages with no visible key are not read.  Page numbers of the
//              next step are loaded before the wait for its slot.
//   warp 9     MMA issuer (one lane), not on the scheduler of warps 0 and 4,
//              which do all the softmax of a few rows (176 instead of 187 us
//              for the 16 caches).  Where a V tile reaches past the visible
//              keys, the warp first zeroes those rows: a slot no token filled
//              may hold NaN, and 0 x NaN would reach O.
//   warps 0-3  softmax of stream 0 (one TMEM lane = one row), warps 4-7 of
//              stream 1, then the item's epilogue.
// Steps, rings and TMEM buffers run on across items: an item's first loads
// and products overlap the previous item's last ones.  Key tiles are visited
// from the newest backwards (ALiBi's largest scores come first).
// Registers: three warps share a quarter of the SM, so a thread has 168, too
// few for a row's 128 scores and what is done with them.  The softmax takes a
// row's scores from TMEM 16 columns at a time, the next 16 in flight, and
// holds P (64 registers), not S; the ALiBi instance with two-tile items still
// spills 72 bytes.  (Raised register limits by setmaxnreg would hold S, but a
// first form with them did not end once in some hundred calls.  The cause was
// not found: the registers come from the CTA's own pool, which no other grid
// can draw on.)
// Waits.  Every wait for another role is bounded: a role whose wait runs out
// sets the abort flag and leaves, the others' waits see it, and the CTA's parts
// are taken off the record.  Rows are right or as they were.
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D);
// P overwrites S: 64 columns, or all 128 (each 16 keys' high part, then low).
//
// Codes (KV8).  With k = 2^ek ck and v = 2^ev cv, one pair of exponents for every
// 16 keys:
//   S  = 2^(ek - up) (Qhi + Qlo) ck: the keys' codes go to the tensor cores as they
//        are, e4m3 by e4m3 at twice the rate of bf16, and q 2^up is the sum of two
//        e4m3 parts (fa_fwd_paged_fp8.cu).  The exponents are in the softmax's scale.
//   O  = 2^(er - 6) sum_j P_j cv_j,  P_j = 2^(S_j - m + ev_j - er + 6),  er the largest
//        ev so far: two warps turn the values' codes to f16, which holds them exactly
//        and without a scale (two instructions for four codes; turned to bf16 with
//        their scales they took five times as many, and the two chunks 1817 us), and
//        P, in f16 too, takes their powers of two.  l is the sum of P without them,
//        in float32.  P has 11 bits here, so one part does for one-tile items too; it
//        is at most 2^16, so a tile's sum past 1000 (of 64 keys) is not let stand.
// Warp 8 is walker and producer (K's codes and the exponents into the slot, V's codes
// into a stage), warps 10 and 11 turn V, 64 rows of a tile each, and write it where
// TMA would have.  In two-tile items a tile's P is given away in halves of 64 keys: the
// first half's product runs while the softmax takes the second (1457 -> 1434 us), and
// the registers of half of P suffice.  O stays over 2^(er - 6) until it is divided by
// l: times it, values of 2^117 and more would have sums that are no floats.  A part
// whose power lies that far from 1 takes it along (part_power).
// Bound by the step's chain, softmax (1900 cycles) and products (2600 of the step's
// 4000), as with bf16: two chunks of 2048 tokens behind 24k-32k keys, 32 heads on 8,
// d = 128: 1430 us, 1277 TFLOP/s, 65 % of the measured cuBLAS rate.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fa_host_util.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 384;         // bf16 pages: warp 11 has no role
constexpr int kMmaWarp = 9;
constexpr int kLoadWarp = 8;           // codes: also the walker
constexpr int kWalkWarp = 10;          // bf16 pages alone
constexpr int kConvWarp = 10;          // codes alone: the first of kConvWarps
constexpr int kConvWarps = 2;
constexpr int kBarBytes = 576;         // barriers and what the plan finds
constexpr int kSegs = 4;               // items that the walker may be ahead
constexpr float kTau = 8.0f;           // lazy rescale: raise m beyond this (log2 units)
constexpr float kRaiseSum = 256.0f;    // 2^kTau
constexpr float kMaxSum = 1.0995116e12f;   // 2^40
constexpr int kUpP = 6;                // codes: P in f16 is times 2^6, ..
constexpr float kMaxSumF16 = 1000.0f;  // .. and no more than 2^16
constexpr int kWeightTwo = 9, kWeightOne = 8;   // of one key tile of an item
constexpr int kHeadTwo = 36, kHeadOne = 16;     // of its Q, first tile and epilogue beside that
// The same over codes, measured again (least squares over the CTAs of eight batches):
// 4075 cycles a tile of a two-tile item and 2420 of another, 21800 and 6040 beside
// them at d = 128, whose weights d = 64 takes too (3670, 2240, 14100, 4390: there an
// item's head weighs 20 to 27 % too much).  A mixed batch's CTAs ended 23 % after their
// mean with bf16's weights.
constexpr int kWeightTwoCodes = 18, kWeightOneCodes = 11, kHeadTwoCodes = 88, kHeadOneCodes = 26;
// Of an item of the kernel for few rows, whose tiles are 8.  With 16 an item more cost
// a CTA 7000 cycles beyond its weight and a tile 1570 at d = 128, 3300 and 1220 at
// d = 64: 16 + 8 x 7000 / 1570 = 52 and 38, of which 44 lies between (16 caches of 8
// heads: 132 us with 16, 125 with 44).
constexpr int kHeadFew = 44;
// A CTA's run is at least this long, so that none lies between the beginnings
// of an item's first two tiles: an item's parts are in CTAs next to each other.
constexpr int kMinRunTwo = kHeadTwo + kWeightTwo + 2, kMinRunOne = kHeadOne + kWeightOne + 2;
constexpr int kMinRunTwoCodes = kWeightTwoCodes + 2, kMinRunOneCodes = kWeightOneCodes + 2;

template <int D, bool KV8>
struct Cfg {
  static constexpr int NB = D / 64;                 // 64-column boxes per row
  static constexpr int BOX_BYTES = 128 * 64 * 2;
  static constexpr int TILE_BYTES = NB * BOX_BYTES;
  // slots: K of a step, V of the one before
  static constexpr int NS = D == 128 ? 2 : KV8 ? 4 : 5;
  static constexpr int K_SLOT = KV8 ? 128 * D : TILE_BYTES;   // codes: K as it is, V in f16
  static constexpr int NV = D == 128 ? 3 : 4;       // codes: tiles of V's codes on their way
  static constexpr int NH = 8;                      // codes: steps whose exponents are kept
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * TILE_BYTES;
  static constexpr int V_OFF = K_OFF + NS * K_SLOT;
  static constexpr int STG_OFF = V_OFF + NS * TILE_BYTES;
  static constexpr int HEAD_OFF = STG_OFF + (KV8 ? NV * 128 * D : 0);     // exponents, then the rows of V's tiles that count
  static constexpr int ML_OFF = HEAD_OFF + (KV8 ? NH * 128 + NV * 16 : 0);   // (m, l, l~ or O's power of two) of both streams' rows
  static constexpr int SEG_OFF = ML_OFF + 2 * 128 * 3 * 4;          // ring of items
  static constexpr int PAR_OFF = SEG_OFF + kSegs * 96;              // a copy of the parameters
  static constexpr int BAR_OFF = PAR_OFF + 256;
  static constexpr int SMEM_BYTES = BAR_OFF + kBarBytes + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  // the work plan's prefix sums borrow the K/V slots before the first load
  static_assert(kPagedMaxBatch * 8 <= NS * (K_SLOT + TILE_BYTES), "plan");
  static constexpr uint32_t S_COL0 = 0, S_COL1 = 128;
  static constexpr uint32_t O_COL0 = 256, O_COL1 = 256 + D;
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[5], kv_empty[5];
  uint64_t s_full[2], p_full[2];
  uint64_t o_done, o_free, drain;
  uint64_t joined;              // (m, l, l~) of both streams' rows of a one-tile item are there
  uint64_t stage_full[4], stage_empty[4];   // codes: V's on their way
  uint64_t p_half[2], half_done[2];         // codes, two tiles: P of 64 keys, its product
#ifdef FA_PAGED_STOP
  uint64_t never;               // nothing arrives on it
#endif
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem_base;
  int abort_flag;
  int part_lost[2];             // the part's item met a page outside the pool
  // the plan: where this CTA's run begins
  unsigned long long warp_sum[16];
  long long w0, w1, base;
  int b, g, qb;
  int unit;                     // few rows: the values' largest power of two that a warp met in the item
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

#ifdef FA_PAGED_STOP
// Test build: the wait of warp g_stop[0] of CTA g_stop[1] for its item number
// g_stop[2] runs out, as if the item's arrival had been lost.
__device__ int g_stop[3] = {-1, -1, -1};
constexpr unsigned long long kStopLimitNs = 1000000;
#endif

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// New tokens [c0, c0 + n) of sequence b and its cached length L; n = 0 where
// there is nothing to do.  False: malformed (n is 0 then).  PICK: of the kernels
// that share a call, one has the sequences of up to few_rows rows per kv head.
template <bool PICK>
__device__ __forceinline__ bool load_seq(const PagedParams& p, int b, int* c0, int* n, int* L) {
  int c1;
  if (p.cu_seqlens) {
    *c0 = __ldg(p.cu_seqlens + b);
    c1 = __ldg(p.cu_seqlens + b + 1);
  } else {
    *c0 = b * p.N;
    c1 = *c0 + p.N;
  }
  *L = __ldg(p.cache_seqlens + b);
  *n = 0;
  if (*c0 < 0 || (b == 0 && *c0 != 0) || c1 < *c0 || (long long)c1 > p.T || c1 - *c0 > p.N) return false;
  if (c1 == *c0) return true;
  if (*L < (p.causal ? c1 - *c0 : 0) || (long long)*L > (long long)p.max_pages * p.page_size) return false;
  if (PICK && ((long long)(c1 - *c0) * p.group <= p.few_rows) != (p.few != 0)) return true;
  *n = c1 - *c0;
  return true;
}

// The block of query tokens from tok0 on of a sequence (n new tokens, L
// cached): tile t holds nt[t] tokens at positions f[t] .. and needs key tiles
// lo[t] .. hi[t]; the item's steps visit key tiles hi_all, hi_all - 1, ...
// (kt of them).  Keys outside [vlo, vhi) are seen by no row.
struct Block {
  int nt[2], f[2], lo[2], hi[2];
  int hi_all, kt, vlo, vhi;
  bool two;
};

__device__ __forceinline__ void block_geometry(const PagedParams& p, int n, int L, int tok0, Block& k) {
  const int left = n - tok0;
  k.two = left > p.tpt;
  k.nt[0] = min(left, p.tpt);
  k.nt[1] = min(max(left - p.tpt, 0), p.tpt);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    k.f[t] = L - n + tok0 + t * p.tpt;
    const int last = p.causal ? k.f[t] + k.nt[t] - 1 : L - 1;
    k.hi[t] = max(last, 0) >> 7;
    k.lo[t] = max(k.f[t] - p.window, 0) >> 7;      // window: kNoWindow without a band
    if (!p.causal) k.lo[t] = 0;
  }
  if (!k.two) {
    k.hi[1] = k.hi[0];
    k.lo[1] = k.lo[0];
  }
  k.hi_all = k.hi[1];
  k.kt = k.hi_all - k.lo[0] + 1;
  k.vlo = p.causal ? max(k.f[0] - p.window, 0) : 0;
  k.vhi = p.causal ? k.f[0] + k.nt[0] + k.nt[1] : L;
}

template <bool PICK>
__device__ __forceinline__ int tile_weight(const PagedParams& p, const Block& k) {
  if (PICK && !p.few) return k.two ? kWeightTwoCodes : kWeightOneCodes;
  return k.two ? kWeightTwo : kWeightOne;
}
template <bool PICK>
__device__ __forceinline__ int head_weight(const PagedParams& p, const Block& k) {
  if (PICK) return p.few ? kHeadFew : k.two ? kHeadTwoCodes : kHeadOneCodes;
  return k.two ? kHeadTwo : kHeadOne;
}

// Weight of the block of query tokens from tok0 on (0 behind the last).  Not
// inlined: a short call runs through code that no SM has cached yet, so each
// copy of this would cost more than the calls.
template <bool PICK>
static __device__ __noinline__ int block_weight(const PagedParams& p, int n, int L, int tok0) {
  if (tok0 >= n) return 0;
  Block k;
  block_geometry(p, n, L, tok0, k);
  return head_weight<PICK>(p, k) + k.kt * tile_weight<PICK>(p, k);
}

// A part of an item, as the walker passes it on: steps [ib, ie) of the item's
// kt; end of the run: ie < 0.
struct Seg {
  Block k;
  int g, tok, ntok;            // kv head; first token (row of q) and tokens of the item
  int b, L, ib, ie;            // sequence, its length
  int lost;                    // the producer met a page outside the pool
};
static_assert(sizeof(Seg) <= 96, "segment ring");

// A CTA's walk over its run [w0, w1) of the line of tiles.
struct Walk {
  long long w0, w1, base;      // base: place of item (b, g, qb) on the line
  int b, g, qb, c0, n, L;
};

template <bool PICK>
__device__ __forceinline__ void walk_begin(const PagedParams& p, const Bars* bars, Walk& w) {
  w.w0 = bars->w0;
  w.w1 = bars->w1;
  w.base = bars->base;
  w.b = bars->b;
  w.g = bars->g;
  w.qb = bars->qb;
  w.c0 = w.n = w.L = 0;
  if (w.w0 < w.w1) load_seq<PICK>(p, w.b, &w.c0, &w.n, &w.L);
}

// The next part of an item in the run; false at its end.
template <bool PICK>
__device__ __forceinline__ bool walk_next(const PagedParams& p, Walk& w, Seg& s) {
  while (w.base < w.w1) {
    if (w.qb * 2 * p.tpt >= w.n) {
      w.qb = 0;
      if (++w.g >= p.Hkv) {
        w.g = 0;
        do {
          if (++w.b >= p.B) return false;              // not reached: the run ends with an item
          load_seq<PICK>(p, w.b, &w.c0, &w.n, &w.L);
        } while (w.n == 0);
      }
    }
    const int tok0 = w.qb * 2 * p.tpt;
    block_geometry(p, w.n, w.L, tok0, s.k);
    // On the line an item is its head and then its tiles; the first tile
    // begins with the head.  A CTA has the tiles that begin in its run.
    const int wt = tile_weight<PICK>(p, s.k), head = head_weight<PICK>(p, s.k);
    const long long len = head + (long long)s.k.kt * wt;
    if (PICK) {
      // Codes: the first tile begins behind the head, so that a run that ends in an
      // item's head leaves the item to the next.
      const long long t0 = w.base + head;
      s.ib = w.w0 <= t0 ? 0 : (int)((w.w0 - t0 + wt - 1) / wt);
      s.ie = w.w1 <= t0 ? 0 : (int)min((long long)s.k.kt, (w.w1 - t0 + wt - 1) / wt);
    } else {
      s.ib = w.base >= w.w0 ? 0 : max(1, ((int)(w.w0 - w.base) - head + wt - 1) / wt);
      s.ie = w.w1 - w.base >= len ? s.k.kt : min(s.k.kt, max(1, ((int)(w.w1 - w.base) - head + wt - 1) / wt));
    }
    s.b = w.b;
    s.L = w.L;
    s.g = w.g;
    s.tok = w.c0 + tok0;
    s.ntok = s.k.nt[0] + s.k.nt[1];
    w.base += len;
    ++w.qb;
    if (s.ib < s.ie) return true;
  }
  return false;
}

// Cuts the line of tiles: fills bars->w0, w1 and the place they begin.  All
// threads; `pre` holds B 64-bit words of shared memory.
template <int NT, bool PICK>
__device__ __forceinline__ void make_plan(const PagedParams& p, Bars* bars, unsigned long long* pre, unsigned min_run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // 1. every sequence's weight, nl lanes per sequence
  const int nl = p.plan_lanes;
  const int sub = lane & (nl - 1);
  for (int b0 = 0; b0 < p.B; b0 += NT / nl) {
    const int b = b0 + tid / nl;
    long long wsum = 0;
    if (b < p.B) {
      int c0, n, L;
      if (!load_seq<PICK>(p, b, &c0, &n, &L) && blockIdx.x == 0 && sub == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
      for (int tok0 = sub * 2 * p.tpt; tok0 < n; tok0 += nl * 2 * p.tpt) wsum += block_weight<PICK>(p, n, L, tok0);
    }
    for (int o = nl / 2; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
    if (b < p.B && sub == 0) pre[b] = (unsigned long long)wsum;      // of one kv head
  }
  __syncthreads();
  // 2. exclusive prefix sums: each thread a run of sequences
  const int per = (p.B + NT - 1) / NT;
  const int f = min(tid * per, p.B), e = min(f + per, p.B);
  unsigned long long own = 0;
  for (int b = f; b < e; ++b) own += pre[b] * p.Hkv;
  unsigned long long inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) bars->warp_sum[warp] = inc;
  __syncthreads();
  unsigned long long before = 0, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += bars->warp_sum[w];
    total += bars->warp_sum[w];
  }
  before += inc - own;
  // 3. this CTA's run, and the sequence it begins in.  Cut in float: the
  // same for a CTA's end and its neighbour's beginning, and never falling,
  // which is all that is needed.
  const int active = (int)min((unsigned long long)gridDim.x, max(1ull, total / min_run));
  const int c = min((int)blockIdx.x, active);
  auto cut = [&](int i) {
    if (i >= active) return (long long)total;
    return min((long long)(__ull2float_rz(total) * ((float)i / (float)active)), (long long)total);
  };
  const long long w0 = cut(c), w1 = cut(c + 1);
  if (tid == 0) {
    bars->w0 = w0;
    bars->w1 = w1;
    bars->base = w1;             // an empty run
    bars->b = bars->g = bars->qb = 0;
  }
  __syncthreads();
  if (w0 < w1) {
    unsigned long long at = before;
    for (int b = f; b < e; ++b) {
      const unsigned long long x = pre[b] * p.Hkv;
      if (at <= (unsigned long long)w0 && (unsigned long long)w0 < at + x) {
        bars->b = b;
        bars->base = (long long)at;
      }
      at += x;
    }
  }
  __syncthreads();
  // 4. the kv head and the q block
  if (warp == 0 && w0 < w1) {
    const int b = bars->b;
    const long long sw = (long long)pre[b];
    int c0, n, L;
    load_seq<PICK>(p, b, &c0, &n, &L);
    // the head: a float quotient, put right by at most a step
    int g = min((int)((float)(w0 - bars->base) / (float)sw), p.Hkv - 1);
    while (g > 0 && bars->base + g * sw > w0) --g;
    while (bars->base + (g + 1) * sw <= w0) ++g;
    long long base = bars->base + g * sw;
    int qb = 0;
    for (int q0 = 0;; q0 += 32) {
      const int x = block_weight<PICK>(p, n, L, (q0 + lane) * 2 * p.tpt);
      long long run = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x > 0 && base + run > w0);
      if (hit) {
        const int src = __ffs(hit) - 1;
        qb = q0 + src;
        base += __shfl_sync(0xffffffffu, run - x, src);
        break;
      }
      base += __shfl_sync(0xffffffffu, run, 31);
      if ((q0 + 32) * 2 * p.tpt >= n) break;      // not reached: w0 lies in this head's blocks
    }
    __syncwarp();
    if (lane == 0) {
      bars->g = g;
      bars->qb = qb;
      bars->base = base;
    }
  }
  __syncthreads();
}

// O row (D columns at tO) *= alpha, in TMEM.  Warp-collective.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 16) {
    uint32_t o[16];
    tmem_ld16(tO + c0, o);
    tmem_wait_ld();
    reg_fence16(o);
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
    tmem_st16(tO + c0, o);
  }
}

// 16 columns of a row, as float32 or bf16, `at` 32-byte aligned.  A warp's rows
// lie apart, so each store of it touches 32 lines whatever its width.
__device__ __forceinline__ void store32(void* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" :: "l"(at), FA_W8(v, 0) : "memory");
}

__device__ __forceinline__ void store_row16(const float* v, bool f32, char* at) {
  uint32_t w[16];
  if (f32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
    store32(at, w);
    store32(at + 32, w + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    store32(at, w);
  }
}

// 4 codes as f16.
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
  uint2 r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.x) : "h"((uint16_t)w));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.y) : "h"((uint16_t)(w >> 16)));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 4 bytes from global to shared memory, asynchronously; only the first `bytes` are
// read, zeros for the others.
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" :: "r"(at), "r"(v) : "memory");
}

// A descriptor as smem_desc_sw128 of rows of 64 bytes, swizzled over them (layout
// type 4), `sbo_bytes` from one eight of them to the next.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t sbo_bytes) {
  return (smem_desc_sw128(saddr, 16, sbo_bytes) & ~((uint64_t)7 << 61)) | (uint64_t)4 << 61;
}

// D[tmem] (+)= A[smem] * B[smem], 128 x 128 over 32: e4m3, both K-major, float32.
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t accumulate) {
  constexpr uint32_t idesc = (1u << 4) | (128u >> 3 << 17) | (128u >> 4 << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// Completes one of the arrivals that `bar` waits for when this thread's copies
// so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

// 2^e, the exponent cut to what a float holds.
__device__ __forceinline__ float pow2_cut(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }

// The exponent that a block's header holds: a word of the scales, the byte's place.
__device__ __forceinline__ int exponent_of(uint32_t word, uint32_t shift) {
  return (int)min(word >> shift & 0xffu, (uint32_t)kScaleHigh + 127) - 127;
}

// Whether the phase is over, without a wait (mbar_try_wait may take its time).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// wait_warp_slow of one thread.
static __device__ __noinline__ bool wait_thread_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* status,
                                                     unsigned long long limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      record_status(status, FA_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  return true;
}

// 2^e for e from -127 to 127.
__device__ __forceinline__ float pow2_of(int e) { return __int_as_float(e > -127 ? (e + 127) << 23 : 0x00400000); }

// 2^e for e up to 127, down to the least that a float holds.
__device__ __forceinline__ float pow2_any(int e) {
  return __int_as_float(e >= -126 ? (e + 127) << 23 : 1 << (max(e, -149) + 149));
}

// Codes: what is kept of O's power of two, the values' largest and P's, behind a
// part's sums.  The part is not divided, and what l times the largest value is may
// be no float; nor is what little a scale below those of a write leaves.
__device__ __forceinline__ int part_power(int values, int p) { return values > 60 || values < kScaleLow ? values + p : 0; }

// ONE: no item has two tiles (the host knows from N).  KV8: the pages hold
// codes.
template <int D, bool ALIBI, bool ONE, bool KV8>
__global__ void __launch_bounds__(kThreads, 1)
fwd_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = Cfg<D, KV8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // The functions that are not inlined read the parameters here: through a
  // pointer to the kernel's own they would come from memory.
  static_assert(sizeof(PagedParams) <= 256 && sizeof(PagedParams) % 4 == 0, "parameters");
  const PagedParams& ps = *reinterpret_cast<const PagedParams*>(smem + C::PAR_OFF);
  if (threadIdx.x < sizeof(PagedParams) / 4)
    reinterpret_cast<uint32_t*>(smem + C::PAR_OFF)[threadIdx.x] = reinterpret_cast<const uint32_t*>(&p)[threadIdx.x];

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->p_half[t], 4);
      mbar_init(&bars->half_done[t], 1);
    }
    for (int s = 0; s < C::NS; ++s) {
      // codes: K, the exponents, V in f16
      mbar_init(&bars->kv_full[s], KV8 ? 1 + 8 + kConvWarps : 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      // producer (or the warps that turn V's codes), MMA issuer, 8 softmax warps
      mbar_init(&bars->seg_empty[i], KV8 ? kConvWarps + 9 : 10);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->stage_full[i], 1);
      mbar_init(&bars->stage_empty[i], kConvWarps);
    }
    mbar_init(&bars->o_done, 1);
    mbar_init(&bars->o_free, 8);
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->joined, 8);
#ifdef FA_PAGED_STOP
    mbar_init(&bars->never, 1);
#endif
    bars->abort_flag = bars->part_lost[0] = bars->part_lost[1] = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  // Q rows past the box (128 % group of them) are zero for good.
  const int rows_box = p.tpt * p.group;
  if (!KV8) {
    for (int i = threadIdx.x; i < 2 * C::NB * (128 - rows_box) * 8; i += kThreads) {
      const int box = i / ((128 - rows_box) * 8), j = i % ((128 - rows_box) * 8);
      reinterpret_cast<uint4*>(smem + C::Q_OFF + box * C::BOX_BYTES + rows_box * 128)[j] = make_uint4(0, 0, 0, 0);
    }
  } else {                             // both parts of both tiles
    const int per = (128 - rows_box) * (D / 16);
    for (int i = threadIdx.x; i < 4 * per; i += kThreads)
      reinterpret_cast<uint4*>(smem + C::Q_OFF + i / per * (C::TILE_BYTES / 2) + rows_box * D)[i % per] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  make_plan<kThreads, KV8>(ps, bars, reinterpret_cast<unsigned long long*>(smem + C::K_OFF), KV8 ? (ONE ? kMinRunOneCodes : kMinRunTwoCodes) : ONE ? kMinRunOne : kMinRunTwo);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  if (KV8) grid_dependency_wait();     // q's parts are made by the kernel before this one
  const uint32_t tmem = bars->tmem_base;
  const WaitCtx wc{&bars->abort_flag, p.status};
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_warp(bar, parity, wc); };
  // The ring of items: item n is ring[n % kSegs]; false at the run's end (or if
  // the wait ran out).  A reader gives the place back with seg_done.
  const Seg* ring = reinterpret_cast<const Seg*>(smem + C::SEG_OFF);
  int nitem = 0;
  auto next_seg = [&](bool& ok) -> bool {
#ifdef FA_PAGED_STOP
    if (warp == g_stop[0] && (int)blockIdx.x == g_stop[1] && nitem == g_stop[2])
      return ok = wait_warp(&bars->never, 0, WaitCtx{&bars->abort_flag, p.status, kStopLimitNs});
#endif
    if (!wait(&bars->seg_full[nitem % kSegs], (nitem / kSegs) & 1)) return ok = false;
    return ring[nitem % kSegs].ie >= 0;
  };
  auto seg_done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->seg_empty[nitem % kSegs]);
    ++nitem;
  };

  if (!KV8 && warp == kLoadWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int box_rows = min(p.page_size, 128);
    const int nbox = 128 / box_rows;
    const uint32_t box_bytes = box_rows * 128;
    bool ok = true;
    unsigned q_any = 0, q_par = 0;   // bit x: Q buffer x was loaded; its last load's parity
    int qsel = 0;              // buffer of the next one-tile item
    int gs = 0;                // steps over all items
    int vrow = -1, vg = 0;     // the step before: this lane's page row (-1: no box), kv head
    while (ok && next_seg(ok)) {
      const Seg& s = ring[nitem % kSegs];
      const bool two = !ONE && s.k.two;
      const int g = s.g, ib = s.ib, ie = s.ie, vlo = s.k.vlo, vhi = s.k.vhi, hi_all = s.k.hi_all;
      const int tok = s.tok, b = s.b;
      // (the place in the ring stays this item's until its epilogue is done)
      int* lost = const_cast<int*>(&s.lost);
      seg_done();
      for (int t = 0; t < (two ? 2 : 1); ++t) {
        const int x = two ? t : qsel;
        if ((q_any >> x & 1) && !(ok = wait(&bars->q_empty[x], q_par >> x & 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[x], C::NB * rows_box * 128);
#pragma unroll
          for (int bx = 0; bx < C::NB; ++bx)
            tma_load_3d(smem + C::Q_OFF + x * C::TILE_BYTES + bx * C::BOX_BYTES, &tmQ, bx * 64, g * p.group,
                        tok + t * p.tpt, &bars->q_full[x]);
        }
        __syncwarp();
        if (q_any >> x & 1) q_par ^= 1u << x;
        q_any |= 1u << x;
      }
      if (!ok) break;
      if (!two) qsel ^= 1;
      const int32_t* table = p.block_table + (long long)b * p.max_pages;
      for (int i = ib; i < ie; ++i, ++gs) {
        const int key0 = (hi_all - i) * 128 + lane * box_rows;
        int krow = -1;
        bool bad = false;
        if (lane < nbox && key0 < vhi && key0 + box_rows > vlo) {
          const int page = __ldg(table + (key0 >> p.page_shift));
          if (page >= 0 && page < p.num_pages) {
            krow = page * p.page_size + (key0 & (p.page_size - 1));
          } else {
            // nothing is loaded, and the item's rows are not written
            record_status(p.status, FA_ERR_PAGE);
            bad = true;
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) *lost = 1;      // (the lane whose arrival publishes it)
        const int sl = gs % C::NS;
        if (gs >= C::NS && !(ok = wait(&bars->kv_empty[sl], ((gs / C::NS) - 1) & 1))) break;
        const int boxes = __popc(__ballot_sync(0xffffffffu, krow >= 0)) + __popc(__ballot_sync(0xffffffffu, vrow >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&bars->kv_full[sl], boxes * C::NB * box_bytes);
        __syncwarp();
#pragma unroll
        for (int bx = 0; bx < C::NB; ++bx) {
          const int off = sl * C::TILE_BYTES + bx * C::BOX_BYTES + lane * box_bytes;
          if (krow >= 0) tma_load_3d(smem + C::K_OFF + off, &tmK, bx * 64, g, krow, &bars->kv_full[sl]);
          if (vrow >= 0) tma_load_3d(smem + C::V_OFF + off, &tmV, bx * 64, vg, vrow, &bars->kv_full[sl]);
        }
        __syncwarp();
        vrow = krow;
        vg = g;
      }
    }
    if (ok && gs > 0) {                           // the last step's V
      const int sl = gs % C::NS;
      if (gs < C::NS || (ok = wait(&bars->kv_empty[sl], ((gs / C::NS) - 1) & 1))) {
        const int boxes = __popc(__ballot_sync(0xffffffffu, vrow >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&bars->kv_full[sl], boxes * C::NB * box_bytes);
        __syncwarp();
#pragma unroll
        for (int bx = 0; bx < C::NB; ++bx)
          if (vrow >= 0)
            tma_load_3d(smem + C::V_OFF + sl * C::TILE_BYTES + bx * C::BOX_BYTES + lane * box_bytes, &tmV, bx * 64, vg,
                        vrow, &bars->kv_full[sl]);
        __syncwarp();
        ++gs;
      }
    }
    // Loads in flight must land before this CTA's shared memory goes away.
    for (int x = 0; x < 2; ++x)
      if (q_any >> x & 1) wait_warp_drain(&bars->q_full[x], q_par >> x & 1);
    for (int i = max(0, gs - C::NS); i < gs; ++i) wait_warp_drain(&bars->kv_full[i % C::NS], (i / C::NS) & 1);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, 0, 0);
    // (codes: f16 where the others have bf16)
    constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, 0, 1) & ~(KV8 ? 1u << 7 | 1u << 10 : 0u);
    // Product kk of S's D / 16.  Codes: D / 32 of Q's first part, then of its second.
    auto s_product = [&](uint32_t colS, uint64_t qd, uint64_t kd, int kk) {
      if (KV8) {
        const uint32_t off = kk % (D / 32) * 32;
        mma_ss_e4m3(colS, desc_add(qd, kk / (D / 32) * (C::TILE_BYTES / 2) + off), desc_add(kd, off), kk > 0 ? 1u : 0u);
      } else {
        const uint32_t off = (kk >> 2) * C::BOX_BYTES + (kk & 3) * 32;
        mma_ss(colS, desc_add(qd, off), desc_add(kd, off), IDESC_S, kk > 0 ? 1u : 0u);
      }
    };
    const uint64_t qdesc0 = KV8 && D == 64 ? smem_desc_sw64(smem_u32(smem + C::Q_OFF), 512)
                                           : smem_desc_sw128(smem_u32(smem + C::Q_OFF), 16, 1024);
    const uint64_t kdesc0 = KV8 && D == 64 ? smem_desc_sw64(smem_u32(smem + C::K_OFF), 512)
                                           : smem_desc_sw128(smem_u32(smem + C::K_OFF), 16, 1024);
    const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::V_OFF), C::BOX_BYTES, 1024);
    bool ok = true;
    int gs = 0, nseg = 0;
    unsigned q_par = 0;          // bit x: parity of Q buffer x's next load
    int qsel = 0, flip = 0;
    unsigned p_par = 0, h_par = 0;   // bit t: parity of stream t's next p_full, p_half
    // The step before, whose PV products are due: streams (bit t), those
    // that begin an item there (bit t), whether its item is a one-tile one,
    // whether it ends its item, and the V rows [vlo, vhi) that are visible.
    int pv = 0, pv_first = 0, v_lo = 0, v_hi = 128;
    bool pv_dual = false, pv_last = false;
    auto issue_s = [&](int t, int x, int sl) {
      if (lane == 0) {
        const uint64_t qd = desc_add(qdesc0, x * C::TILE_BYTES), kd = desc_add(kdesc0, sl * C::K_SLOT);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) s_product(tmem + (t ? C::S_COL1 : C::S_COL0), qd, kd, kk);
        mma_commit(&bars->s_full[t]);
      }
      __syncwarp();
    };
    // Codes, two tiles: products of the keys' half h.
    auto pv_half = [&](int t, int h, int sl, uint32_t accumulate) {
      const uint64_t vd = desc_add(vdesc0, sl * C::TILE_BYTES + h * 4 * 2048);
      const uint32_t colP = tmem + (t ? C::S_COL1 : C::S_COL0) + h * 32, colO = tmem + (t ? C::O_COL1 : C::O_COL0);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_ts(colO, colP + kk * 8, desc_add(vd, kk * 2048), IDESC_O, kk > 0 ? 1u : accumulate);
    };
    auto issue_pv = [&](int t, int sl) -> bool {
      if (KV8 && !ONE && !pv_dual) {
        if (!wait(&bars->p_half[t], h_par >> t & 1)) return false;
        h_par ^= 1u << t;
        const bool first = (pv_first >> t) & 1;
        if (first && nseg > 0 && !wait(&bars->o_free, (nseg - 1) & 1)) return false;
        tc_fence_after();
        if (lane == 0) {
          pv_half(t, 0, sl, !first);
          mma_commit(&bars->half_done[t]);
        }
        __syncwarp();
        if (!wait(&bars->p_full[t], p_par >> t & 1)) return false;
        p_par ^= 1u << t;
        tc_fence_after();
        if (lane == 0) pv_half(t, 1, sl, 1u);
        __syncwarp();
        return true;
      }
      if (!wait(&bars->p_full[t], p_par >> t & 1)) return false;
      p_par ^= 1u << t;
      // the first PV_t of an item overwrites O_t, which the item before
      // must have read
      const bool first = (pv_first >> t) & 1;
      if (first && nseg > 0 && !wait(&bars->o_free, (nseg - 1) & 1)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t vd = desc_add(vdesc0, sl * C::TILE_BYTES);
        const uint32_t colP = tmem + (t ? C::S_COL1 : C::S_COL0), colO = tmem + (t ? C::O_COL1 : C::O_COL0);
        if (!KV8 && (ONE || pv_dual)) {                   // 16 keys of P: high part, low part
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            mma_ts(colO, colP + kk * 16, desc_add(vd, kk * 2048), IDESC_O, (!first || kk > 0) ? 1u : 0u);
            mma_ts(colO, colP + kk * 16 + 8, desc_add(vd, kk * 2048), IDESC_O, 1u);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(colO, colP + kk * 8, desc_add(vd, kk * 2048), IDESC_O, (!first || kk > 0) ? 1u : 0u);
        }
      }
      __syncwarp();
      return true;
    };
    // V rows that no row sees are zeroed before the tile's products.
    auto clean_v = [&](int sl) {
      if constexpr (!KV8) {                               // (of codes, such rows came as zeros)
        if (v_lo <= 0 && v_hi >= 128) return;
        for (int i = lane; i < 128 * 8; i += 32) {
          const int r = i >> 3;
          if (r >= v_lo && r < v_hi) continue;
#pragma unroll
          for (int bx = 0; bx < C::NB; ++bx)
            reinterpret_cast<uint4*>(smem + C::V_OFF + sl * C::TILE_BYTES + bx * C::BOX_BYTES)[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
    };
    while (ok && next_seg(ok)) {
      const Seg& s = ring[nitem % kSegs];
      const bool two = !ONE && s.k.two;
      const int ib = s.ib, ie = s.ie, hi_all = s.k.hi_all, vlo = s.k.vlo, vhi = s.k.vhi;
      const int lo0 = s.k.lo[0], hi0 = s.k.hi[0], lo1 = s.k.lo[1], hi1 = s.k.hi[1];
      seg_done();
      int started = 0;                                  // streams that have begun this item
      for (int i = ib; ok && i < ie; ++i, ++gs) {
        const int sl = gs % C::NS;
        const int kt = hi_all - i;
        const int cur = two ? ((kt >= lo0 && kt <= hi0) | ((kt >= lo1 && kt <= hi1) << 1)) : 1 << ((flip + i - ib) & 1);
        // Inside an item, with nothing but products to issue.  The tensor pipe
        // takes only a couple of products ahead, so what this warp does
        // between two batches is time the pipe idles.
        const bool inside = !pv_first && !pv_last && i > ib && i < ie - 1 && (KV8 || (v_lo <= 0 && v_hi >= 128));
        if (!ONE && two && inside && cur == 3 && pv == 3) {
          // Two tiles: PV0, S0, PV1, S1.  The slot's loads were waited for by
          // softmax warp 0 (before p_full[0]), which these products rest on: a
          // softmax without that wait would let them read a slot that is being
          // filled.  P1 is asked for while the last products of the first batch
          // run.
          const uint64_t kd = desc_add(kdesc0, sl * C::K_SLOT), vd = desc_add(vdesc0, sl * C::TILE_BYTES);
          if constexpr (KV8) {
            // Four parts: each stream's P of 64 keys, then of the others and S.  The next
            // part's P is asked for before the last products of one.  One lane does it
            // all, straight on, so that the descriptors are constants but for the slot.
            auto ready_bar = [&](int k) { return k & 1 ? &bars->p_full[k >> 1] : &bars->p_half[k >> 1]; };
            auto ready_par = [&](int k) { return (k & 1 ? p_par : h_par) >> (k >> 1) & 1; };
            if (lane == 0) {
              bool there = mbar_try_wait(ready_bar(0), ready_par(0));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int t = k >> 1;
                if (!there && !(ok = wait_thread_slow(ready_bar(k), ready_par(k), wc.abort_flag, wc.status, wc.limit_ns))) break;
                tc_fence_after();
                pv_half(t, k & 1, sl, 1u);
                if (k & 1) {
                  const uint32_t colS = tmem + (t ? C::S_COL1 : C::S_COL0);
#pragma unroll
                  for (int kk = 0; kk < D / 16; ++kk) {
                    if (k < 3 && kk == D / 16 - 2) there = mbar_test(ready_bar(k + 1), ready_par(k + 1));
                    s_product(colS, desc_add(qdesc0, t * C::TILE_BYTES), kd, kk);
                  }
                  mma_commit(&bars->s_full[t]);
                  if (t) mma_commit(&bars->kv_empty[sl]);
                } else {
                  mma_commit(&bars->half_done[t]);
                  there = mbar_try_wait(ready_bar(k + 1), ready_par(k + 1));
                }
              }
            }
            if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0))) break;
            p_par ^= 3u;
            h_par ^= 3u;
            v_lo = vlo - kt * 128;
            v_hi = vhi - kt * 128;
            continue;
          }
          auto batch = [&](int t, bool ask) -> bool {
            const uint32_t colS = tmem + (t ? C::S_COL1 : C::S_COL0), colO = tmem + (t ? C::O_COL1 : C::O_COL0);
            bool there = false;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) mma_ts(colO, colS + kk * 8, desc_add(vd, kk * 2048), IDESC_O, 1u);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              if (ask && kk == D / 16 - 2) there = mbar_try_wait(&bars->p_full[1], p_par >> 1 & 1);
              s_product(colS, desc_add(qdesc0, t * C::TILE_BYTES), kd, kk);
            }
            mma_commit(&bars->s_full[t]);
            if (t) mma_commit(&bars->kv_empty[sl]);
            return there;
          };
          if (!(ok = wait(&bars->p_full[0], p_par & 1))) break;
          bool there = false;
          if (lane == 0) {
            tc_fence_after();
            there = batch(0, true);
            if (there) {
              tc_fence_after();
              batch(1, false);
            }
          }
          if (!__shfl_sync(0xffffffffu, (int)there, 0)) {
            if (!(ok = wait(&bars->p_full[1], p_par >> 1 & 1))) break;
            if (lane == 0) {
              tc_fence_after();
              batch(1, false);
            }
            __syncwarp();
          }
          p_par ^= 3u;
          v_lo = vlo - kt * 128;
          v_hi = vhi - kt * 128;
          continue;
        }
        if (!(ok = wait(&bars->kv_full[sl], (gs / C::NS) & 1))) break;
        if ((ONE || !two) && inside) {
          // One tile: S of this step's stream, PV of the other's.
          const int t = cur >> 1, u = t ^ 1;
          if (lane == 0) {
            const uint64_t kd = desc_add(kdesc0, sl * C::K_SLOT), qd = desc_add(qdesc0, qsel * C::TILE_BYTES);
            const uint32_t colS = tmem + C::S_COL0 + t * (C::S_COL1 - C::S_COL0);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) s_product(colS, qd, kd, kk);
            mma_commit(&bars->s_full[t]);
          }
          __syncwarp();
          if (!(ok = wait(&bars->p_full[u], p_par >> u & 1))) break;
          if (lane == 0) {
            tc_fence_after();
            const uint64_t vd = desc_add(vdesc0, sl * C::TILE_BYTES);
            const uint32_t colP = tmem + C::S_COL0 + u * (C::S_COL1 - C::S_COL0);
            const uint32_t colO = tmem + C::O_COL0 + u * (C::O_COL1 - C::O_COL0);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              mma_ts(colO, colP + kk * (KV8 ? 8 : 16), desc_add(vd, kk * 2048), IDESC_O, 1u);
              if (!KV8) mma_ts(colO, colP + kk * 16 + 8, desc_add(vd, kk * 2048), IDESC_O, 1u);
            }
            mma_commit(&bars->kv_empty[sl]);
          }
          __syncwarp();
          p_par ^= 1u << u;
          pv = cur;
          v_lo = vlo - kt * 128;
          v_hi = vhi - kt * 128;
          continue;
        }
        // S of a stream whose P is not waited for comes first; but at an
        // item's head, whose Q may be on its way, PV of the item before.
        const int s_first = i == ib && two ? 0 : cur & ~pv, s_last = i == ib && two ? cur : 0;
        if (i == ib && !two && !(ok = wait(&bars->q_full[qsel], q_par >> qsel & 1))) break;
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
          if (s_first >> t & 1) issue_s(t, two ? t : qsel, sl);
        clean_v(sl);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (pv >> t & 1)
            if (!(ok = issue_pv(t, sl))) break;
          if ((cur & ~s_first & ~s_last) >> t & 1) issue_s(t, two ? t : qsel, sl);
        }
        if (!ok) break;
#pragma unroll 1
        for (int t = 0; s_last && t < 2; ++t) {
          const int x = two ? t : qsel;
          if ((two || t == 0) && !(ok = wait(&bars->q_full[x], q_par >> x & 1))) break;
          if (s_last >> t & 1) issue_s(t, x, sl);
        }
        if (!ok) break;
        if (lane == 0) {
          if (pv_last) mma_commit(&bars->o_done);
          mma_commit(&bars->kv_empty[sl]);
          if (i == ie - 1) {
            mma_commit(&bars->q_empty[two ? 0 : qsel]);
            if (two) mma_commit(&bars->q_empty[1]);
          }
        }
        __syncwarp();
        nseg += pv_last;
        pv = cur;
        pv_first = cur & ~started;
        started |= cur;
        pv_dual = !two;
        pv_last = i == ie - 1;
        v_lo = vlo - kt * 128;
        v_hi = vhi - kt * 128;
      }
      if (!ok) break;
      if (two) {
        q_par ^= 3u;
      } else {
        q_par ^= 1u << qsel;
        qsel ^= 1;
        flip = (flip + ie - ib) & 1;
      }
    }
    if (ok && gs > 0) {                                 // the last step's PV
      const int sl = gs % C::NS;
      if ((ok = wait(&bars->kv_full[sl], (gs / C::NS) & 1))) {
        clean_v(sl);
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
          if (ok && (pv >> t & 1)) ok = issue_pv(t, sl);
        if (ok && lane == 0) mma_commit(&bars->o_done);
        __syncwarp();
      }
    }
    // Tensor-core work must be finished before the TMEM is released.
    if (lane == 0) mma_commit(&bars->drain);
    __syncwarp();
    wait_warp_drain(&bars->drain, 0);
  } else if (!KV8 && warp == kWalkWarp) {
    // -------------------------------------------------------------- walker
    Walk w;
    Seg s;
    s.lost = 0;
    walk_begin<KV8>(p, bars, w);
    // what the parts of this CTA are, for the merge: kind of the part that
    // goes on from the CTA before (2: the item's last), and the item begun here
    int cont = 0;
    int4 begun = make_int4(0, 0, 0, 0);
    bool more = true;
    for (; more; ++nitem) {
      more = walk_next<KV8>(p, w, s);
      if (more) {
        if (s.ib > 0) cont = s.ie == s.k.kt ? 2 : 1;
        else if (s.ie < s.k.kt) begun = make_int4(1, s.tok, s.ntok, s.g);
      } else {
        s.ie = -1;
        if (lane == 0) {
          p.part_meta[2 * blockIdx.x] = make_int4(cont, 0, 0, 0);
          p.part_meta[2 * blockIdx.x + 1] = begun;
        }
      }
      if (nitem >= kSegs && !wait(&bars->seg_empty[nitem % kSegs], (nitem / kSegs - 1) & 1)) break;
      if (lane == 0) {
        const_cast<Seg*>(ring)[nitem % kSegs] = s;
        mbar_arrive(&bars->seg_full[nitem % kSegs]);
      }
      __syncwarp();
    }
  } else if (KV8 && warp == kLoadWarp) {
    // -------------------------------------------- codes: walker and producer
    // Finds the items, one ahead of the steps it fetches.  Per step: K's codes and
    // lane i the exponents of the tile's block i into a slot, V's codes into a stage
    // (128 / page_size boxes of each, one lane each, one box for larger pages).
    Walk w;
    Seg s;
    s.lost = 0;
    walk_begin<KV8>(p, bars, w);
    int cont = 0;
    int4 begun = make_int4(0, 0, 0, 0);
    bool more = true, ok = true;
    auto publish = [&](int n) {
      if (n >= kSegs && !wait(&bars->seg_empty[n % kSegs], (n / kSegs - 1) & 1)) return false;
      more = walk_next<KV8>(p, w, s);
      if (more) {
        if (s.ib > 0) cont = s.ie == s.k.kt ? 2 : 1;
        else if (s.ie < s.k.kt) begun = make_int4(1, s.tok, s.ntok, s.g);
      } else {
        s.ie = -1;
        if (lane == 0) {
          p.part_meta[2 * blockIdx.x] = make_int4(cont, 0, 0, 0);
          p.part_meta[2 * blockIdx.x + 1] = begun;
        }
      }
      if (lane == 0) {
        const_cast<Seg*>(ring)[n % kSegs] = s;
        mbar_arrive(&bars->seg_full[n % kSegs]);
      }
      __syncwarp();
      return true;
    };
    const long long scale_bytes = (long long)p.num_pages * (p.page_size >> 4) * p.Hkv;
    const int box_rows = min(p.page_size, 128), boxes = 128 / box_rows, blocks = box_rows >> 4;
    constexpr int kNoPage = -0x7fffffff - 1;            // no row sees these keys
    unsigned q_any = 0, q_par = 0;   // bit x: Q buffer x was loaded; its last load's parity
    int qsel = 0;              // buffer of the next one-tile item
    int gs = 0, ks = 0;        // steps over all items: V's loads, K's
    // a block's exponents in 16 bytes: the words of the scales that hold its byte, the byte's place
    const uint32_t heads = smem_u32(smem + C::HEAD_OFF);
    uint32_t* const limits = reinterpret_cast<uint32_t*>(smem + C::HEAD_OFF + C::NH * 128);
    ok = publish(0);
    for (int n = 0; ok && more; ++n) {
      const bool two = !ONE && s.k.two;
      const int g = s.g, ib = s.ib, ie = s.ie, vlo = s.k.vlo, vhi = s.k.vhi, hi_all = s.k.hi_all, tok = s.tok;
      const int32_t* table = p.block_table + (long long)s.b * p.max_pages;
      int* const lost = &const_cast<Seg*>(ring)[n % kSegs].lost;
      auto look_up = [&](int i) {                       // page of this lane's block
        const int key = (hi_all - i) * 128 + 16 * lane;
        return lane < 8 && i < ie && key < vhi && key + 16 > vlo ? max(__ldg(table + (key >> p.page_shift)), -1) : kNoPage;
      };
      int page = look_up(ib);
      if (!(ok = publish(n + 1))) break;
      for (int t = 0; t < (two ? 2 : 1); ++t) {
        const int x = two ? t : qsel;
        if ((q_any >> x & 1) && !(ok = wait(&bars->q_empty[x], q_par >> x & 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[x], 2 * D * rows_box);
#pragma unroll
          for (int part = 0; part < 2; ++part)
            tma_load_3d(smem + C::Q_OFF + x * C::TILE_BYTES + part * (C::TILE_BYTES / 2), &tmQ, 0, g * p.group,
                        (part ? (int)p.T : 0) + tok + t * p.tpt, &bars->q_full[x]);
        }
        __syncwarp();
        if (q_any >> x & 1) q_par ^= 1u << x;
        q_any |= 1u << x;
      }
      if (!ok) break;
      if (!two) qsel ^= 1;
      for (int i = ib; i < ie; ++i, ++gs) {
        const int next_page = look_up(i + 1);
        const int key = (hi_all - i) * 128 + 16 * lane;
        const bool good = (unsigned)page < (unsigned)p.num_pages;
        const uint32_t row = good ? (uint32_t)page * p.page_size + (key & (p.page_size - 1)) : 0;
        // a page that is not there is not read, and the item's rows are not written
        const bool bad = __any_sync(0xffffffffu, !good && page != kNoPage);
        const unsigned seen = __ballot_sync(0xffffffffu, good) & 0xffu;
        const unsigned mine = lane < boxes ? seen >> (lane * blocks) & ((1u << blocks) - 1) : 0;
        const int row_of = (int)__shfl_sync(0xffffffffu, row, mine ? lane * blocks + __ffs(mine) - 1 : 0) & ~(box_rows - 1);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine != 0)) * box_rows * D;
        const long long j = good ? (long long)(row >> 4) * p.Hkv + g : 0;
        const uint32_t few = good ? (uint32_t)min(4ll, scale_bytes - (j & ~3ll)) : 0;
        const int sl = gs % C::NS, st = gs % C::NV;
        if (gs >= C::NS && !(ok = wait(&bars->kv_empty[sl], ((gs / C::NS) - 1) & 1))) break;
        if (lane < 8) {
          const uint32_t at = heads + (gs % C::NH) * 128 + lane * 16;
          copy_async4(at, p.k_scales + (j & ~3ll), few);
          copy_async4(at + 4, p.v_scales + (j & ~3ll), few);
          sts32(at + 8, (uint32_t)(j & 3) * 8);
        }
        __syncwarp();                                   // lane 0 publishes what the others wrote
        if (lane == 0) {
          if (bad) {
            record_status(p.status, FA_ERR_PAGE);
            *lost = 1;
          }
          mbar_arrive_expect_tx(&bars->kv_full[sl], bytes);
        }
        __syncwarp();
        if (mine) tma_load_3d(smem + C::K_OFF + sl * C::K_SLOT + lane * box_rows * D, &tmK, 0, g, row_of, &bars->kv_full[sl]);
        if (lane < 8) copies_arrive(&bars->kv_full[sl]);
        __syncwarp();
        ++ks;
        if (gs >= C::NV && !(ok = wait(&bars->stage_empty[st], ((gs / C::NV) - 1) & 1))) break;
        if (lane == 0) {
          limits[4 * st] = vlo - (hi_all - i) * 128;    // rows that some row of the item sees
          limits[4 * st + 1] = vhi - (hi_all - i) * 128;
          mbar_arrive_expect_tx(&bars->stage_full[st], bytes);
        }
        __syncwarp();
        if (mine) tma_load_3d(smem + C::STG_OFF + st * 128 * D + lane * box_rows * D, &tmV, 0, g, row_of, &bars->stage_full[st]);
        __syncwarp();
        page = next_page;
      }
    }
    if (ok && gs > 0) {                                 // the last step's V: a slot without K
      const int sl = gs % C::NS;
      if (gs < C::NS || (ok = wait(&bars->kv_empty[sl], ((gs / C::NS) - 1) & 1))) {
        if (lane == 0) mbar_arrive(&bars->kv_full[sl]);
        __syncwarp();
        if (lane < 8) copies_arrive(&bars->kv_full[sl]);
        __syncwarp();
        ++ks;
      }
    }
    // Copies in flight must land before this CTA's shared memory goes away.
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int x = 0; x < 2; ++x)
      if (q_any >> x & 1) wait_warp_drain(&bars->q_full[x], q_par >> x & 1);
    for (int i = max(0, ks - C::NS); i < ks; ++i) wait_warp_drain(&bars->kv_full[i % C::NS], (i / C::NS) & 1);
    for (int i = max(0, gs - C::NV); i < gs; ++i) wait_warp_drain(&bars->stage_full[i % C::NV], (i / C::NV) & 1);
  } else if (KV8 && warp >= kConvWarp) {
    // ------------------------------- codes: V's to f16, 64 rows of a tile per warp
    // Written where TMA puts bf16 pages: 64 columns per box, swizzled over 128
    // bytes.  Rows that no row of the item sees become zeros.
    // A lane has 16 codes of a row.  Eight lanes' loads and their stores each take
    // eight different places of 128 bytes: at d = 128 four lanes of row r and four
    // of row r ^ 5.
    constexpr int RPU = 512 / D;                        // rows per load
    const int cw = warp - kConvWarp;
    const int rl = D == 128 ? (lane >> 4) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    const int jj = D == 128 ? (lane >> 1 & 4) | (lane & 3) : lane & 3, j0 = 2 * (jj & 3);
    auto row_of = [&](int u) { return D == 128 ? (u >> 1) * 8 + ((u & 1) * 2 ^ rl) : u * RPU + rl; };
    const uint32_t* const limits = reinterpret_cast<const uint32_t*>(smem + C::HEAD_OFF + C::NH * 128);
    bool ok = true;
    int cs = 0;                                         // steps turned: V of step cs goes to slot cs + 1
    while (ok && next_seg(ok)) {
      const Seg& s = ring[nitem % kSegs];
      const int steps = s.ie - s.ib;
      seg_done();
      if (cs == 0 && lane == 0) mbar_arrive(&bars->kv_full[0]);      // the first slot has no V
      for (int i = 0; i < steps; ++i, ++cs) {
        const int st = cs % C::NV, to = cs + 1, sl = to % C::NS;
        if (!(ok = wait(&bars->stage_full[st], (cs / C::NV) & 1))) break;
        if (to >= C::NS && !(ok = wait(&bars->kv_empty[sl], ((to / C::NS) - 1) & 1))) break;
        const int lo = (int)limits[4 * st], hi = (int)limits[4 * st + 1];
        const bool all = lo <= 0 && hi >= 128;
        const uint32_t from = smem_u32(smem + C::STG_OFF) + st * 128 * D;
        const uint32_t box = smem_u32(smem + C::V_OFF) + sl * C::TILE_BYTES + (jj >> 2) * C::BOX_BYTES;
#pragma unroll 1
        for (int r0 = 64 * cw; r0 < 64 * cw + 64; r0 += 16) {
          uint4 c[16 / RPU];
#pragma unroll
          for (int u = 0; u < 16 / RPU; ++u) {
            const int r = row_of(u);
            c[u] = lds128(from + r0 * D + r * D + (jj ^ (D == 128 ? r & 7 : r >> 1 & 3)) * 16);
          }
          if (!all) {
#pragma unroll
            for (int u = 0; u < 16 / RPU; ++u) {
              const int r = r0 + row_of(u);
              if (r < lo || r >= hi) c[u] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int u = 0; u < 16 / RPU; ++u) {
            const uint2 x0 = codes_to_f16(c[u].x), x1 = codes_to_f16(c[u].y);
            const uint2 x2 = codes_to_f16(c[u].z), x3 = codes_to_f16(c[u].w);
            const uint32_t at = box + r0 * 128 + row_of(u) * 128, sw = row_of(u) & 7;
            sts128(at + ((j0 ^ sw) << 4), make_uint4(x0.x, x0.y, x1.x, x1.y));
            sts128(at + ((j0 ^ 1 ^ sw) << 4), make_uint4(x2.x, x2.y, x3.x, x3.y));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->stage_empty[st]);
          mbar_arrive(&bars->kv_full[sl]);
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int q4 = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t tS = lane_base + (t ? C::S_COL1 : C::S_COL0);
    const uint32_t tO = lane_base + (t ? C::O_COL1 : C::O_COL0);
    const float c2 = p.scale_log2;
    float* mls = reinterpret_cast<float*>(smem + C::ML_OFF);
    bool ok = true;
    int cs = 0;                  // S products consumed (s_full phases)
    int nseg = 0, flip = 0;
    int gs = 0;                  // steps before this item
    int njoin = 0;               // one-tile items before this one
    int nhalf = 0;               // codes: tiles whose P went in halves
    // A warp whose wait ran out leaves; the others' waits for it run out or
    // see the abort flag.
    while (true) {
      int n0, steps, diag, low, kend;
      bool valid, dual;
      float slope2 = 0.f;
      int vslot = 0;             // step of this stream's next tile
      int hs0 = 0;               // codes: that step, whose exponents are its keys'
      float c2q = c2;            // codes: over the power of two that Q's row is times
      int eref = -127;           // codes: O is over 2^eref
      {
        if (!next_seg(ok)) break;
        const Seg& s = ring[nitem % kSegs];
        const int r = 32 * q4 + lane, rq = r / p.group;  // row of the tile, its token
        dual = ONE || !s.k.two;
        const bool second = !dual && t;                 // holds the second tile's rows
        const int f = second ? s.k.f[1] : s.k.f[0], nt = second ? s.k.nt[1] : s.k.nt[0];
        int kt0;
        if (dual) {
          const int first = (t - flip) & 1;             // this stream's first step
          kt0 = s.k.hi_all - s.ib - first;
          steps = (s.ie - s.ib - first + 1) >> 1;
          flip = (flip + s.ie - s.ib) & 1;
        } else {
          kt0 = min(s.k.hi_all - s.ib, second ? s.k.hi[1] : s.k.hi[0]);
          steps = max(0, kt0 - max(s.k.hi_all - s.ie + 1, second ? s.k.lo[1] : s.k.lo[0]) + 1);
        }
        n0 = 128 * kt0;                                 // first key of the tile
        valid = rq < nt;
        kend = p.causal ? f + rq : s.L - 1;             // last key this row sees
        // tiles that reach past `diag` or begin before `low` hold keys that
        // some row does not see
        diag = p.causal ? f : s.L - 1;
        low = f + nt - 1 - p.window;
        if (ALIBI) slope2 = valid ? __ldg(p.alibi + s.g * p.group + r % p.group) * kLog2e : 0.f;
        if (KV8 && valid) c2q = c2 * pow2_of(-p.q_exps[(long long)(s.tok + (second ? p.tpt : 0) + rq) * p.Hq + s.g * p.group + r % p.group]);
        vslot = hs0 = gs + s.k.hi_all - s.ib - kt0;
        gs += s.ie - s.ib;
      }
      const bool warp_rows = __any_sync(0xffffffffu, valid);
      float m_ref = -INFINITY;
      float l = 0.f;     // sum of p in fp32: gives the LSE
      float lr = 0.f;    // sum of the p that the PV products see: normalises O
      float grow = 0.f;  // log2 by which the reference is to rise before the next tile
      for (int j = 0; ok && j < steps; ++j, ++cs, n0 -= dual ? 256 : 128) {
        if (!(ok = wait(&bars->s_full[t], cs & 1))) break;
        // Codes, two tiles: P of the first 64 keys is given away before the others'.
        const bool halves = KV8 && !ONE && !dual;
        if (!warp_rows) {                               // no row of this warp holds a token
          if (lane == 0) {
            if (halves) mbar_arrive(&bars->p_half[t]);
            mbar_arrive(&bars->p_full[t]);
          }
          nhalf += halves;
          continue;
        }
        tc_fence_after();
        // Codes: lane i has the exponents of the tile's block i, of its keys and, over
        // the reference, of its values.  A score of column c is S c2q 2^(its keys').
        // P takes the power of two of its values, so that the products take the
        // values' codes: O is over 2^eref, the largest so far.
        float kpow = 1.f, vlog = 0.f, vinv = 1.f;
        if (KV8) {
          const uint4 hd = lds128(smem_u32(smem + C::HEAD_OFF) + ((hs0 + (dual ? 2 : 1) * j) % C::NH) * 128 + (lane & 7) * 16);
          kpow = pow2_of(exponent_of(hd.x, hd.z));
          const int ev = exponent_of(hd.y, hd.z), top = __reduce_max_sync(0xffffffffu, ev);
          if (top > eref) {
            if (j > 0) rescale_row<D>(tO, pow2_cut(eref - top));
            eref = top;
          }
          // 2^-60 and less of a P below 2^10 is 0 in f16
          const int up = max(ev - eref, -60) + kUpP;
          vlog = (float)up;
          vinv = pow2_of(-up);
        }
        // (a scale below 2^-100 makes 0 of any score, and must not make NaN of -inf)
        auto c2_of = [&](int c) { return KV8 ? fmaxf(c2q * __shfl_sync(0xffffffffu, kpow, c >> 4), 7.8886091e-31f) : c2; };
        // The commit that published S_t also covers this stream's last PV, so
        // O may be rescaled now.
        if (!ONE && __any_sync(0xffffffffu, grow > 0.f)) {
          const float alpha = ex2_approx(-grow);
          l *= alpha;
          lr *= alpha;
          m_ref += grow;
          grow = 0.f;
          rescale_row<D>(tO, alpha);
        }
        // ALiBi bias of column c in log2 units: slope2 * (n0 + c - position);
        // causal, so the row's position is its last key.
        const float base = ALIBI ? slope2 * (float)(n0 - kend) : 0.f;
        // p = 2^(x - mb) of 16 scores from column c on: 8 packed pairs, and
        // with LOW what the rounding left of them; sums of p, of the rounded p
        uint64_t acc[2], accr[2];
        // (codes: what their block takes, asked for ahead of them)
        struct Of16 { float c2, vlog, vinv; };
        auto of16 = [&](int c) -> Of16 {
          if (!KV8) return {c2, 0.f, 1.f};
          return {c2_of(c), __shfl_sync(0xffffffffu, vlog, c >> 4), __shfl_sync(0xffffffffu, vinv, c >> 4)};
        };
        auto exp16 = [&](auto low_part, int c, const Of16& of, const uint32_t* x, float mb, uint32_t* hi, uint32_t* lo) {
          constexpr bool LOW = decltype(low_part)::value;
          const float mv = KV8 ? mb - of.vlog : mb;
          uint64_t bm = f2(-mv, -mv);
          if (ALIBI) {
            const float b0 = fmaf(slope2, (float)c, base - mv);
            bm = f2(b0, b0 + slope2);
          }
          const float c2c = of.c2;
          const uint64_t step = f2(2.f * slope2, 2.f * slope2), c2p = f2(c2c, c2c);
          uint64_t sum[2] = {0, 0};                     // codes: of these 16
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t ex = ffma2(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2p, bm);
            if (ALIBI) bm = fadd2(bm, step);
            float e0, e1;
            f2split(ex, e0, e1);
            const float p0 = ex2_approx(e0);
            const float p1 = ex2_approx(e1);
            const uint64_t pp = f2(p0, p1);
            if (KV8) {
              sum[i & 1] = i < 2 ? pp : fadd2(sum[i & 1], pp);
              hi[i] = pack_f16x2(p0, p1);
              continue;
            }
            acc[i & 1] = fadd2(acc[i & 1], pp);
            hi[i] = pack_bf16x2(p0, p1);
            const uint64_t ph = f2(__uint_as_float(hi[i] << 16), __uint_as_float(hi[i] & 0xFFFF0000u));
            if (LOW) {
              float r0, r1;
              f2split(fsub2(pp, ph), r0, r1);
              lo[i] = pack_bf16x2(r0, r1);
            } else {
              accr[i & 1] = fadd2(accr[i & 1], ph);
            }
          }
          if (KV8) acc[0] = ffma2(fadd2(sum[0], sum[1]), f2(of.vinv, of.vinv), acc[0]);
        };
        auto pair_sum = [](const uint64_t* a) {
          float x, y;
          f2split(fadd2(a[0], a[1]), x, y);
          return x + y;
        };
        bool settled = false, given = false;            // given: P of the first 64 keys
        // Tiles on the diagonal, at the end or at the band's lower edge hold
        // scores of keys that a row does not see.
        const bool masked = n0 + 127 > diag || n0 < low;
        if (!ONE && !dual && !masked && !__any_sync(0xffffffffu, valid && m_ref == -INFINITY)) {
          // P with the reference as it is; kept in registers until its sum
          // shows that it may stand.  P and O are floats, so a reference that
          // is too low costs no precision: a sum up to 2^40 stands, and one
          // above 2^8 raises the reference for the next tile.
          if constexpr (KV8) {
            // The same for 64 keys and then for the others.
            uint32_t pk[32], x[2][16];
            auto half = [&](int h) -> float {
              acc[0] = acc[1] = 0;
              tmem_ld16(tS + 64 * h, x[0]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const Of16 of = of16(64 * h + 16 * c);
                tmem_wait_ld();
                reg_fence16(x[c & 1]);
                if (c < 3) tmem_ld16(tS + 64 * h + 16 * (c + 1), x[(c + 1) & 1]);
                exp16(std::false_type{}, 64 * h + 16 * c, of, x[c & 1], m_ref, pk + 8 * c, nullptr);
              }
              return pair_sum(acc);
            };
            float ts = half(0);
            settled = !__any_sync(0xffffffffu, valid && !(ts <= kMaxSumF16));
            if (settled) {
              tmem_st32(tS, pk);
              tmem_wait_st();
              tc_fence_before();
              if (warp == 0) {                          // on behalf of the MMA issuer, as below
                ++vslot;
                if (!(ok = wait(&bars->kv_full[vslot % C::NS], (vslot / C::NS) & 1))) break;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->p_half[t]);
              given = true;
              const float tb = half(1);
              if (!__any_sync(0xffffffffu, valid && !(tb <= kMaxSumF16))) {
                tmem_st32(tS + 32, pk);
                ts += tb;
                l += ts;
                if (valid && ts > kRaiseSum) grow = ceilf(lg2_approx(ts));
              } else {
                // Rare: the first half's product stays under the reference it was
                // given away with, and O takes the new one when that is done.
                l += ts;
                if (!(ok = wait(&bars->half_done[t], nhalf & 1))) break;
                tc_fence_after();
                settled = false;
              }
            }
          } else {
            uint32_t pk[64], x[2][16];
            acc[0] = acc[1] = accr[0] = accr[1] = 0;
            tmem_ld16(tS, x[0]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const Of16 of = of16(16 * c);
              tmem_wait_ld();
              reg_fence16(x[c & 1]);
              if (c < 7) tmem_ld16(tS + 16 * (c + 1), x[(c + 1) & 1]);
              exp16(std::false_type{}, 16 * c, of, x[c & 1], m_ref, pk + 8 * c, nullptr);
            }
            const float ts = pair_sum(acc);
            settled = !__any_sync(0xffffffffu, valid && !(ts <= kMaxSum));   // also inf / nan
            if (settled) {
              tmem_st32(tS, pk);
              tmem_st32(tS + 32, pk + 32);
              l += ts;
              lr += pair_sum(accr);
              if (valid && ts > kRaiseSum) grow = ceilf(lg2_approx(ts));
            }
          }
        }
        if (!settled) {
          // The tile's max first: a masked tile, a row's first, a sum past
          // 2^40, and every tile of a one-tile item (HBM sets its pace).
          // Masked scores become -inf, in TMEM too, whatever the slots hold.
          const int ub = kend - n0, lb = p.causal ? ub - p.window : 0;
          const int c_first = given ? 64 : 0;
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = c_first; c < 128; c += 32) {
            uint32_t x[32];
            tmem_ld32(tS + c, x);
            const float ca = c2_of(c), cb = c2_of(c + 16);
            tmem_wait_ld();
            reg_fence32(x);
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c + i > ub) x[i] = __float_as_uint(-INFINITY);
              if (n0 < low)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (c + i < lb) x[i] = __float_as_uint(-INFINITY);
              tmem_st32(tS + c, x);
            }
            float m4[4] = {KV8 ? -INFINITY : mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
              if (ALIBI) {
                x0 = fmaf(x0, i < 16 ? ca : cb, fmaf(slope2, (float)(c + i), base));
                x1 = fmaf(x1, i < 16 ? ca : cb, fmaf(slope2, (float)(c + i + 1), base));
              }
              // codes: columns 0 .. 15 and 16 .. 31 apart, as their scales are
              const int k = KV8 ? i / 16 * 2 + (i / 2 & 1) : i / 2 & 3;
              m4[k] = fmax3(m4[k], x0, x1);
            }
            if (KV8) {
              const float a = fmaxf(m4[0], m4[1]), b = fmaxf(m4[2], m4[3]);
              mx = fmax3(mx, ALIBI ? a : a * ca, ALIBI ? b : b * cb);
            } else {
              mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
            }
          }
          if (masked) tmem_wait_st();
          if (!ALIBI && !KV8) mx *= c2;
          // Any reference gives the same result: it stays until the max has
          // grown by more than tau.
          const bool raise = mx > m_ref + kTau;
          if (__any_sync(0xffffffffu, raise)) {
            const float m_new = raise ? mx : m_ref;
            const float alpha = raise ? ex2_approx(m_ref - m_new) : 1.f;
            l *= alpha;
            lr *= alpha;
            m_ref = m_new;
            if (j > 0) rescale_row<D>(tO, alpha);
          }
          const float mb = m_ref == -INFINITY ? 0.f : m_ref;
          acc[0] = acc[1] = accr[0] = accr[1] = 0;
          // P over the scores just read: with two parts each 16 keys' high and
          // low part take the 16 columns of their scores, else 16 keys take 8
#pragma unroll 1
          for (int c = c_first; c < 128; c += 32) {
            uint32_t x[32], y[32];
            tmem_ld32(tS + c, x);
            const Of16 of0 = of16(c), of1 = of16(c + 16);
            tmem_wait_ld();
            reg_fence32(x);
            if (!KV8 && (ONE || dual)) {
              exp16(std::true_type{}, c, of0, x, mb, y, y + 8);
              exp16(std::true_type{}, c + 16, of1, x + 16, mb, y + 16, y + 24);
              tmem_st32(tS + c, y);
            } else {
              exp16(std::false_type{}, c, of0, x, mb, y, nullptr);
              exp16(std::false_type{}, c + 16, of1, x + 16, mb, y + 8, nullptr);
              tmem_st16(tS + c / 2, y);
            }
          }
          const float ts = pair_sum(acc);
          l += ts;
          if (!KV8) lr += ONE || dual ? ts : pair_sum(accr);
        }
        tmem_wait_st();
        tc_fence_before();
        // On behalf of the MMA issuer: the next step's slot has been loaded.
        if (!ONE && warp == 0 && !dual && !given) {
          ++vslot;
          if (!(ok = wait(&bars->kv_full[vslot % C::NS], (vslot / C::NS) & 1))) break;
        }
        __syncwarp();
        if (lane == 0) {
          if (halves && !given) mbar_arrive(&bars->p_half[t]);
          mbar_arrive(&bars->p_full[t]);
        }
        nhalf += halves;
      }
      // ---------------------------------------------------------- epilogue
      if (!ok || !wait(&bars->o_done, nseg & 1)) break;
      tc_fence_after();
      // A stream without a step in this part has no O: its columns are not
      // used.
      const int r = 32 * q4 + lane;
      const Seg& s = ring[nitem % kSegs];
      // 0: the whole item; else the slot of the part: 1 its continuation from
      // the CTA before, 2 its beginning
      const int part = s.ib > 0 ? 1 : s.ie < s.k.kt ? 2 : 0;
      if (s.lost) {
        valid = false;
        if (part) bars->part_lost[part - 1] = 1;
      }
      const bool use0 = steps > 0, use1 = dual && (steps == 0 || s.ie - s.ib > 1);
      if (KV8) lr = l;
      float w0 = 1.f, w1 = 0.f;                         // of the own columns, of the other stream's
      int c_from = 0, c_to = D;
      if (dual) {
        // join the two streams: each warp takes half of the columns
        float* own = mls + (t * 128 + r) * 3;
        const float* oth = mls + ((t ^ 1) * 128 + r) * 3;
        own[0] = m_ref;
        own[1] = l;
        own[2] = KV8 ? __int_as_float(eref) : lr;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->joined);
        // Only the time limit ends this wait, not the abort flag: a row's two
        // halves are written by both streams' warps or by neither.
        const uint32_t par = njoin++ & 1;
        if (!__all_sync(0xffffffffu, mbar_try_wait(&bars->joined, par)) && !wait_warp_drain(&bars->joined, par)) {
          if (lane == 0) {
            *wc.abort_flag = 1;
            record_status(p.status, FA_ERR_DEVICE_TIMEOUT);
          }
          break;
        }
        const float mo = oth[0];
        const float M = fmaxf(m_ref, mo);
        w0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - M);
        w1 = mo == -INFINITY ? 0.f : ex2_approx(mo - M);
        l = fmaf(w0, l, w1 * oth[1]);
        lr = KV8 ? l : fmaf(w0, lr, w1 * oth[2]);
        if (KV8) {
          const int eo = __float_as_int(oth[2]), top = max(eref, eo);
          w0 *= pow2_cut(eref - top);
          w1 *= pow2_cut(eo - top);
          eref = top;
        }
        m_ref = M;
        c_from = t * (D / 2);
        c_to = c_from + D / 2;
      }
      const uint32_t tX = lane_base + (t ? C::O_COL0 : C::O_COL1);    // the other stream's O
      const int tl = (dual ? 0 : t * p.tpt) + r / p.group;            // token of the item
      const int rh = r % p.group, head = s.g * p.group + rh;
      const long long tok = s.tok + tl;
      const long long orow = tok * p.Hq + head;
      const int slot = 2 * (int)blockIdx.x + part - 1;
      const long long prow = (long long)slot * p.part_rows + tl * p.group + rh;
      const bool f32 = part || p.o_f32;                 // a part is float32, not divided
      char* out = part ? reinterpret_cast<char*>(p.part_o + prow * D)
                       : static_cast<char*>(p.o) + orow * D * (f32 ? 4 : 2);
      float sc = 1.f;
      if (part == 0) sc = lr > 0.f ? 1.f / lr : 0.f;
      // codes: O is over 2^eref, and P was times 2^kUpP
      const int kept = KV8 && part && (use0 || use1) ? part_power(eref, -kUpP) : 0;
      const float opow = KV8 ? pow2_any(eref - kUpP - kept) : 1.f;
      if (warp_rows) {
#pragma unroll 1
        for (int c = c_from; c < c_to; c += 16) {
          uint32_t a[16], b[16];
          if (use0) tmem_ld16(tO + c, a);
          if (use1) tmem_ld16(tX + c, b);
          tmem_wait_ld();
          reg_fence16(a);
          reg_fence16(b);
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = use0 ? __uint_as_float(a[i]) * w0 : 0.f;
            if (use1) v[i] = fmaf(__uint_as_float(b[i]), w1, v[i]);
            v[i] *= sc;
            if (KV8) v[i] *= opow;
          }
          if (valid) store_row16(v, f32, out + c * (f32 ? 4 : 2));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free);
      if (valid && !(dual && t)) {                      // a one-tile item's rows: stream 0 reports
        if (part) {
          float* ml = p.part_ml + prow * 4;
          *reinterpret_cast<float4*>(ml) = make_float4(m_ref, l, lr, __int_as_float(kept));
        } else {
          p.lse[(long long)head * p.T + tok] = l == 0.f ? -INFINITY : (m_ref + lg2_approx(l)) * kLn2;
        }
      }
      ++nseg;
      seg_done();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // A wait ran out, so parts may be missing, whatever the walker put on record
  // ahead of them: the merge must not take what the workspace held.  Nor a part
  // of an item that met a page outside the pool.
  if (threadIdx.x < 2 && (bars->abort_flag || bars->part_lost[threadIdx.x]))
    p.part_meta[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
}

// Joins the parts of the item that begins in CTA blockIdx.x and goes on in the
// following ones, in their order; an item of which a CTA has no part to show
// is left alone.  POWERS: O of a part may be over the power of two that stands behind
// its sums (part_power).  A warp has RPW rows, D / 32 columns per lane;
// four parts' loads at a time, so that a row costs two waits for memory: what
// the parts are, and the parts.
template <int D, int RPW, bool POWERS>
__device__ __forceinline__ void merge_parts(const PagedParams& p, const int nctas, const int y) {
  const int c = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int row0 = y * 8 * RPW + (threadIdx.x >> 5);
  const int4 it = p.part_meta[2 * c + 1];
  int kind = c + 1 + lane < nctas ? p.part_meta[2 * (c + 1 + lane)].x : 0;
  if (it.x == 0 || row0 >= it.z * p.group) return;
  // parts: slot 2 c + 1, then slot 2 c' of c' = c + 1 .. until an end (kind 2)
  int nparts = 1;
  for (int c0 = c + 1;; c0 += 32) {
    const unsigned stop = __ballot_sync(0xffffffffu, kind != 1);
    if (stop) {
      const int at = __ffs(stop) - 1;
      if (__shfl_sync(0xffffffffu, kind, at) != 2) return;
      nparts += at + 1;
      break;
    }
    nparts += 32;
    kind = c0 + 32 + lane < nctas ? p.part_meta[2 * (c0 + 32 + lane)].x : 0;
  }
  constexpr int PER = D / 32;
  struct alignas(4 * PER) Cols { float v[PER]; };
  auto slot = [&](int s, int row) { return (long long)(s == 0 ? 2 * c + 1 : 2 * (c + s)) * p.part_rows + row; };
  auto sums = [&](int s, int row) { return *reinterpret_cast<const float4*>(p.part_ml + slot(s, row) * 4); };
  auto cols = [&](int s, int row) { return *reinterpret_cast<const Cols*>(p.part_o + slot(s, row) * D + lane * PER); };
#pragma unroll 1
  for (int i = 0; i < RPW; ++i) {
    const int row = row0 + 8 * i;
    if (i > 0 && row >= it.z * p.group) break;
    Cols o;
#pragma unroll
    for (int i = 0; i < PER; ++i) o.v[i] = 0.f;
    float M = -INFINITY, l = 0.f, lr = 0.f;
    int powers = 0;                                     // not 0: some part's O is over a power of two
    for (int s0 = 0; s0 < nparts; s0 += 4) {
      float4 ml[4];
      Cols x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = min(s0 + i, nparts - 1);
        ml[i] = sums(s, row);
        // volatile: the columns are asked for with the sums, not behind their first use
        // (one sequence of 777 tokens: 11.2 us, 11.6 otherwise)
        const float* at = p.part_o + slot(s, row) * D + lane * PER;
        if constexpr (PER == 4)
          asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(x[i].v[0]), "=f"(x[i].v[1]), "=f"(x[i].v[2]), "=f"(x[i].v[3]) : "l"(at));
        else
          asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(x[i].v[0]), "=f"(x[i].v[1]) : "l"(at));
        if (POWERS) powers |= __float_as_int(ml[i].w);
      }
      float mx = M;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s0 + i < nparts) mx = fmaxf(mx, ml[i].x);
      const float a = M == -INFINITY ? 0.f : ex2_approx(M - mx);
      l *= a;
      lr *= a;
#pragma unroll
      for (int k = 0; k < PER; ++k) o.v[k] *= a;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // no key seen there, or (l not 0) a score that is not a number
        if (s0 + i >= nparts || (ml[i].x == -INFINITY && ml[i].y == 0.f)) continue;
        const float w = ex2_approx(ml[i].x - mx);
        l = fmaf(w, ml[i].y, l);
        lr = fmaf(w, ml[i].z, lr);
#pragma unroll
        for (int k = 0; k < PER; ++k) o.v[k] = fmaf(w, x[i].v[k], o.v[k]);
      }
      M = mx;
    }
    float opow = 1.f;
    if (POWERS && powers) {                             // O anew, over the largest power so far
      int top = -1000;
      M = -INFINITY;
#pragma unroll
      for (int k = 0; k < PER; ++k) o.v[k] = 0.f;
#pragma unroll 1
      for (int s = 0; s < nparts; ++s) {
        const float4 ml = sums(s, row);
        const Cols x = cols(s, row);
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float mx = fmaxf(M, ml.x), a = M == -INFINITY ? 0.f : ex2_approx(M - mx), w = ex2_approx(ml.x - mx);
        const int up = __float_as_int(ml.w), was = top;
        top = max(top, up);
        const float pa = pow2_any(was - top), pw = pow2_any(up - top);
#pragma unroll
        for (int k = 0; k < PER; ++k) o.v[k] = fmaf(w, x.v[k] * pw, o.v[k] * a * pa);
        M = mx;
      }
      opow = pow2_any(top);
    }
    const float inv = lr > 0.f ? 1.f / lr : 0.f;
    const long long tok = it.y + row / p.group;
    const int h = it.w * p.group + row % p.group;
    const long long at = (tok * p.Hq + h) * D + lane * PER;
#pragma unroll
    for (int k = 0; k < PER; ++k) o.v[k] *= inv;
    if (POWERS) {
#pragma unroll
      for (int k = 0; k < PER; ++k) o.v[k] *= opow;
    }
    if (p.o_f32) {
      *reinterpret_cast<Cols*>(static_cast<float*>(p.o) + at) = o;
    } else {
#pragma unroll
      for (int k = 0; k < PER; k += 2)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + at + k) = pack_bf16x2(o.v[k], o.v[k + 1]);
    }
    if (lane == 0) p.lse[(long long)h * p.T + tok] = l == 0.f ? -INFINITY : (M + lg2_approx(l)) * kLn2;
  }
}

template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedParams p, const int nctas) {
  grid_dependency_wait();
  merge_parts<D, 1, false>(p, nctas, blockIdx.y);
}

// Those of the two kernels of a call over codes: `ym` rows of blocks for those of
// `many`, of whose up to 256 rows an item a warp takes four (a block costs more than
// its rows: the parts of a mixed batch, not in L2, 18.8 us with one row per warp, 16.4
// with four), the others for those of `few`.
template <int D>
__global__ void __launch_bounds__(256)
paged_merge_two_kernel(const PagedParams few, const PagedParams many, const int ym, const int nctas) {
  grid_dependency_wait();
  const int y = blockIdx.y;
  if (y < ym) merge_parts<D, 4, true>(many, nctas, y);
  else merge_parts<D, 1, true>(few, nctas, y - ym);
}

// Codes: begins while the kernel that makes q's parts runs, and waits for it behind
// the plan; the merge is the caller's.
template <int D, bool ALIBI, bool ONE, bool KV8>
int launch_impl(const PagedParams& p, cudaStream_t stream) {
  using C = Cfg<D, KV8>;
  auto kern = fwd_paged_kernel<D, ALIBI, ONE, KV8>;
  if (const int ea = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return ea;
  CUtensorMap tq, tk, tv;
  const long long slots = (long long)p.num_pages * p.page_size;
  const int box = std::min(p.page_size, 128);
  int r = KV8 ? make_tmap_codes_3d(&tq, p.q_codes, D, p.Hq, 2 * p.T, p.group, p.tpt)
              : make_tmap_bf16_3d_box(&tq, p.q, D, p.Hq, p.T, p.group, p.tpt);
  if (!r) r = KV8 ? make_tmap_codes_3d(&tk, p.k, D, p.Hkv, slots, 1, box) : make_tmap_bf16_3d(&tk, p.k, D, p.Hkv, slots, box);
  if (!r) r = KV8 ? make_tmap_codes_3d(&tv, p.v, D, p.Hkv, slots, 1, box) : make_tmap_bf16_3d(&tv, p.v, D, p.Hkv, slots, box);
  if (r) return r;
  int nsm = 0;
  if (const int es = sm_count(&nsm)) return es;
  const int grid = std::min(nsm, kPagedCtas);
  if constexpr (KV8) {
    return launch_dependent(kern, dim3(grid), dim3(kThreads), C::SMEM_BYTES, stream, tq, tk, tv, p);
  } else {
    kern<<<grid, kThreads, C::SMEM_BYTES, stream>>>(tq, tk, tv, p);
    if (const cudaError_t e = cudaGetLastError()) return (int)e;
    return launch_dependent(paged_merge_kernel<D>, dim3(grid, std::max(1, (p.part_rows + 7) / 8)), dim3(256), 0, stream, p, grid);
  }
}

template <int D, bool KV8>
int launch_d(const PagedParams& p, cudaStream_t stream) {
  // no sequence brings more tokens than one tile holds
  const bool one = p.N <= p.tpt;
  if (p.alibi) return one ? launch_impl<D, true, true, KV8>(p, stream) : launch_impl<D, true, false, KV8>(p, stream);
  return one ? launch_impl<D, false, true, KV8>(p, stream) : launch_impl<D, false, false, KV8>(p, stream);
}

}  // namespace
}  // namespace fa
