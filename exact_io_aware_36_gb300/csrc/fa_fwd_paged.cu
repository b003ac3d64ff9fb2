// fa_fwd_paged.cu -- tensor-core attention of each sequence's newest tokens
// over a cache in pages, for sm_103a.
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
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fa_host_util.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 384;         // warp 11 has no role
constexpr int kMmaWarp = 9;
constexpr int kLoadWarp = 8;
constexpr int kWalkWarp = 10;
constexpr int kSegs = 4;               // items that the walker may be ahead
constexpr float kTau = 8.0f;           // lazy rescale: raise m beyond this (log2 units)
constexpr float kRaiseSum = 256.0f;    // 2^kTau
constexpr float kMaxSum = 1.0995116e12f;   // 2^40
constexpr int kWeightTwo = 9, kWeightOne = 8;   // of one key tile of an item
constexpr int kHeadTwo = 36, kHeadOne = 16;     // of its Q, first tile and epilogue beside that
// A CTA's run is at least this long, so that none lies between the beginnings
// of an item's first two tiles: an item's parts are in CTAs next to each other.
constexpr int kMinRunTwo = kHeadTwo + kWeightTwo + 2, kMinRunOne = kHeadOne + kWeightOne + 2;

template <int D>
struct Cfg {
  static constexpr int NB = D / 64;                 // 64-column boxes per row
  static constexpr int BOX_BYTES = 128 * 64 * 2;
  static constexpr int TILE_BYTES = NB * BOX_BYTES;
  static constexpr int NS = D == 128 ? 2 : 5;       // slots (K of a step, V of the one before)
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * TILE_BYTES;
  static constexpr int V_OFF = K_OFF + NS * TILE_BYTES;
  static constexpr int ML_OFF = V_OFF + NS * TILE_BYTES;   // (m, l, l~) of both streams' rows
  static constexpr int SEG_OFF = ML_OFF + 2 * 128 * 3 * 4;          // ring of items
  static constexpr int PAR_OFF = SEG_OFF + kSegs * 96;              // a copy of the parameters
  static constexpr int BAR_OFF = PAR_OFF + 256;
  static constexpr int SMEM_BYTES = BAR_OFF + 512 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  // the work plan's prefix sums borrow the K/V slots before the first load
  static_assert(kPagedMaxBatch * 8 <= 2 * NS * TILE_BYTES, "plan");
  static constexpr uint32_t S_COL0 = 0, S_COL1 = 128;
  static constexpr uint32_t O_COL0 = 256, O_COL1 = 256 + D;
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[2], p_full[2];
  uint64_t o_done, o_free, drain;
  uint64_t joined;              // (m, l, l~) of both streams' rows of a one-tile item are there
#ifdef FA_PAGED_STOP
  uint64_t never;               // nothing arrives on it
#endif
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem_base;
  int abort_flag;
  int part_lost[2];             // the part's item met a page outside the pool
  // the plan: where this CTA's run begins
  unsigned long long warp_sum[kThreads / 32];
  long long w0, w1, base;
  int b, g, qb;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

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
// there is nothing to do.  False: malformed (n is 0 then).
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

__device__ __forceinline__ int tile_weight(const Block& k) { return k.two ? kWeightTwo : kWeightOne; }
__device__ __forceinline__ int head_weight(const Block& k) { return k.two ? kHeadTwo : kHeadOne; }

// Weight of the block of query tokens from tok0 on (0 behind the last).  Not
// inlined: a short call runs through code that no SM has cached yet, so each
// copy of this would cost more than the calls.
static __device__ __noinline__ int block_weight(const PagedParams& p, int n, int L, int tok0) {
  if (tok0 >= n) return 0;
  Block k;
  block_geometry(p, n, L, tok0, k);
  return head_weight(k) + k.kt * tile_weight(k);
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

__device__ __forceinline__ void walk_begin(const PagedParams& p, const Bars* bars, Walk& w) {
  w.w0 = bars->w0;
  w.w1 = bars->w1;
  w.base = bars->base;
  w.b = bars->b;
  w.g = bars->g;
  w.qb = bars->qb;
  w.c0 = w.n = w.L = 0;
  if (w.w0 < w.w1) load_seq(p, w.b, &w.c0, &w.n, &w.L);
}

// The next part of an item in the run; false at its end.
__device__ __forceinline__ bool walk_next(const PagedParams& p, Walk& w, Seg& s) {
  while (w.base < w.w1) {
    if (w.qb * 2 * p.tpt >= w.n) {
      w.qb = 0;
      if (++w.g >= p.Hkv) {
        w.g = 0;
        do {
          if (++w.b >= p.B) return false;              // not reached: the run ends with an item
          load_seq(p, w.b, &w.c0, &w.n, &w.L);
        } while (w.n == 0);
      }
    }
    const int tok0 = w.qb * 2 * p.tpt;
    block_geometry(p, w.n, w.L, tok0, s.k);
    // On the line an item is its head and then its tiles; the first tile
    // begins with the head.  A CTA has the tiles that begin in its run.
    const int wt = tile_weight(s.k), head = head_weight(s.k);
    const long long len = head + (long long)s.k.kt * wt;
    s.ib = w.base >= w.w0 ? 0 : max(1, ((int)(w.w0 - w.base) - head + wt - 1) / wt);
    s.ie = w.w1 - w.base >= len ? s.k.kt : min(s.k.kt, max(1, ((int)(w.w1 - w.base) - head + wt - 1) / wt));
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
__device__ __forceinline__ void make_plan(const PagedParams& p, Bars* bars, unsigned long long* pre, unsigned min_run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // 1. every sequence's weight, nl lanes per sequence
  const int nl = p.plan_lanes;
  const int sub = lane & (nl - 1);
  for (int b0 = 0; b0 < p.B; b0 += kThreads / nl) {
    const int b = b0 + tid / nl;
    long long wsum = 0;
    if (b < p.B) {
      int c0, n, L;
      if (!load_seq(p, b, &c0, &n, &L) && blockIdx.x == 0 && sub == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
      for (int tok0 = sub * 2 * p.tpt; tok0 < n; tok0 += nl * 2 * p.tpt) wsum += block_weight(p, n, L, tok0);
    }
    for (int o = nl / 2; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
    if (b < p.B && sub == 0) pre[b] = (unsigned long long)wsum;      // of one kv head
  }
  __syncthreads();
  // 2. exclusive prefix sums: each thread a run of sequences
  const int per = (p.B + kThreads - 1) / kThreads;
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
  for (int w = 0; w < kThreads / 32; ++w) {
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
    load_seq(p, b, &c0, &n, &L);
    // the head: a float quotient, put right by at most a step
    int g = min((int)((float)(w0 - bars->base) / (float)sw), p.Hkv - 1);
    while (g > 0 && bars->base + g * sw > w0) --g;
    while (bars->base + (g + 1) * sw <= w0) ++g;
    long long base = bars->base + g * sw;
    int qb = 0;
    for (int q0 = 0;; q0 += 32) {
      const int x = block_weight(p, n, L, (q0 + lane) * 2 * p.tpt);
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

// ONE: no item has two tiles (the host knows from N).
template <int D, bool ALIBI, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
fwd_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = Cfg<D>;
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
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      mbar_init(&bars->seg_empty[i], 10);     // producer, MMA issuer, 8 softmax warps
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
  for (int i = threadIdx.x; i < 2 * C::NB * (128 - rows_box) * 8; i += kThreads) {
    const int box = i / ((128 - rows_box) * 8), j = i % ((128 - rows_box) * 8);
    reinterpret_cast<uint4*>(smem + C::Q_OFF + box * C::BOX_BYTES + rows_box * 128)[j] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  make_plan(ps, bars, reinterpret_cast<unsigned long long*>(smem + C::K_OFF), ONE ? kMinRunOne : kMinRunTwo);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
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

  if (warp == kLoadWarp) {
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
    constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t qdesc0 = smem_desc_sw128(smem_u32(smem + C::Q_OFF), 16, 1024);
    const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::K_OFF), 16, 1024);
    const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::V_OFF), C::BOX_BYTES, 1024);
    bool ok = true;
    int gs = 0, nseg = 0;
    unsigned q_par = 0;          // bit x: parity of Q buffer x's next load
    int qsel = 0, flip = 0;
    unsigned p_par = 0;          // bit t: parity of stream t's next p_full
    // The step before, whose PV products are due: streams (bit t), those
    // that begin an item there (bit t), whether its item is a one-tile one,
    // whether it ends its item, and the V rows [vlo, vhi) that are visible.
    int pv = 0, pv_first = 0, v_lo = 0, v_hi = 128;
    bool pv_dual = false, pv_last = false;
    auto issue_s = [&](int t, int x, int sl) {
      if (lane == 0) {
        const uint64_t qd = desc_add(qdesc0, x * C::TILE_BYTES), kd = desc_add(kdesc0, sl * C::TILE_BYTES);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::BOX_BYTES + (kk & 3) * 32;
          mma_ss(tmem + (t ? C::S_COL1 : C::S_COL0), desc_add(qd, off), desc_add(kd, off), IDESC_S, kk > 0 ? 1u : 0u);
        }
        mma_commit(&bars->s_full[t]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int sl) -> bool {
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
        if (ONE || pv_dual) {                             // 16 keys of P: high part, low part
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
        const bool inside = !pv_first && !pv_last && i > ib && i < ie - 1 && v_lo <= 0 && v_hi >= 128;
        if (!ONE && two && inside && cur == 3 && pv == 3) {
          // Two tiles: PV0, S0, PV1, S1.  The slot's loads were waited for by
          // softmax warp 0 (before p_full[0]), which these products rest on: a
          // softmax without that wait would let them read a slot that is being
          // filled.  P1 is asked for while the last products of the first batch
          // run.
          const uint64_t kd = desc_add(kdesc0, sl * C::TILE_BYTES), vd = desc_add(vdesc0, sl * C::TILE_BYTES);
          auto batch = [&](int t, bool ask) -> bool {
            const uint32_t colS = tmem + (t ? C::S_COL1 : C::S_COL0), colO = tmem + (t ? C::O_COL1 : C::O_COL0);
            bool there = false;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) mma_ts(colO, colS + kk * 8, desc_add(vd, kk * 2048), IDESC_O, 1u);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::BOX_BYTES + (kk & 3) * 32;
              if (ask && kk == D / 16 - 2) there = mbar_try_wait(&bars->p_full[1], p_par >> 1 & 1);
              mma_ss(colS, desc_add(qdesc0, t * C::TILE_BYTES + off), desc_add(kd, off), IDESC_S, kk > 0 ? 1u : 0u);
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
            const uint64_t kd = desc_add(kdesc0, sl * C::TILE_BYTES), qd = desc_add(qdesc0, qsel * C::TILE_BYTES);
            const uint32_t colS = tmem + C::S_COL0 + t * (C::S_COL1 - C::S_COL0);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::BOX_BYTES + (kk & 3) * 32;
              mma_ss(colS, desc_add(qd, off), desc_add(kd, off), IDESC_S, kk > 0 ? 1u : 0u);
            }
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
              mma_ts(colO, colP + kk * 16, desc_add(vd, kk * 2048), IDESC_O, 1u);
              mma_ts(colO, colP + kk * 16 + 8, desc_add(vd, kk * 2048), IDESC_O, 1u);
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
  } else if (warp == kWalkWarp) {
    // -------------------------------------------------------------- walker
    Walk w;
    Seg s;
    s.lost = 0;
    walk_begin(p, bars, w);
    // what the parts of this CTA are, for the merge: kind of the part that
    // goes on from the CTA before (2: the item's last), and the item begun here
    int cont = 0;
    int4 begun = make_int4(0, 0, 0, 0);
    bool more = true;
    for (; more; ++nitem) {
      more = walk_next(p, w, s);
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
    // A warp whose wait ran out leaves; the others' waits for it run out or
    // see the abort flag.
    while (true) {
      int n0, steps, diag, low, kend;
      bool valid, dual;
      float slope2 = 0.f;
      int vslot = 0;             // step of this stream's next tile
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
        vslot = gs + s.k.hi_all - s.ib - kt0;
        gs += s.ie - s.ib;
      }
      const bool warp_rows = __any_sync(0xffffffffu, valid);
      float m_ref = -INFINITY;
      float l = 0.f;     // sum of p in fp32: gives the LSE
      float lr = 0.f;    // sum of the p that the PV products see: normalises O
      float grow = 0.f;  // log2 by which the reference is to rise before the next tile
      for (int j = 0; ok && j < steps; ++j, ++cs, n0 -= dual ? 256 : 128) {
        if (!(ok = wait(&bars->s_full[t], cs & 1))) break;
        if (!warp_rows) {                               // no row of this warp holds a token
          if (lane == 0) mbar_arrive(&bars->p_full[t]);
          continue;
        }
        tc_fence_after();
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
        auto exp16 = [&](auto low_part, int c, const uint32_t* x, float mb, uint32_t* hi, uint32_t* lo) {
          constexpr bool LOW = decltype(low_part)::value;
          uint64_t bm = f2(-mb, -mb);
          if (ALIBI) {
            const float b0 = fmaf(slope2, (float)c, base - mb);
            bm = f2(b0, b0 + slope2);
          }
          const uint64_t step = f2(2.f * slope2, 2.f * slope2), c2p = f2(c2, c2);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t ex = ffma2(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2p, bm);
            if (ALIBI) bm = fadd2(bm, step);
            float e0, e1;
            f2split(ex, e0, e1);
            const float p0 = ex2_approx(e0);
            const float p1 = ex2_approx(e1);
            const uint64_t pp = f2(p0, p1);
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
        };
        auto pair_sum = [](const uint64_t* a) {
          float x, y;
          f2split(fadd2(a[0], a[1]), x, y);
          return x + y;
        };
        bool settled = false;
        // Tiles on the diagonal, at the end or at the band's lower edge hold
        // scores of keys that a row does not see.
        const bool masked = n0 + 127 > diag || n0 < low;
        if (!ONE && !dual && !masked && !__any_sync(0xffffffffu, valid && m_ref == -INFINITY)) {
          // P with the reference as it is; kept in registers until its sum
          // shows that it may stand.  P and O are floats, so a reference that
          // is too low costs no precision: a sum up to 2^40 stands, and one
          // above 2^8 raises the reference for the next tile.
          uint32_t pk[64], x[2][16];
          acc[0] = acc[1] = accr[0] = accr[1] = 0;
          tmem_ld16(tS, x[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_wait_ld();
            reg_fence16(x[c & 1]);
            if (c < 7) tmem_ld16(tS + 16 * (c + 1), x[(c + 1) & 1]);
            exp16(std::false_type{}, 16 * c, x[c & 1], m_ref, pk + 8 * c, nullptr);
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
        if (!settled) {
          // The tile's max first: a masked tile, a row's first, a sum past
          // 2^40, and every tile of a one-tile item (HBM sets its pace).
          // Masked scores become -inf, in TMEM too, whatever the slots hold.
          const int ub = kend - n0, lb = p.causal ? ub - p.window : 0;
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t x[32];
            tmem_ld32(tS + c, x);
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
            float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
              if (ALIBI) {
                x0 = fmaf(x0, c2, fmaf(slope2, (float)(c + i), base));
                x1 = fmaf(x1, c2, fmaf(slope2, (float)(c + i + 1), base));
              }
              m4[i / 2 & 3] = fmax3(m4[i / 2 & 3], x0, x1);
            }
            mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
          }
          if (masked) tmem_wait_st();
          if (!ALIBI) mx *= c2;
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
          for (int c = 0; c < 128; c += 32) {
            uint32_t x[32], y[32];
            tmem_ld32(tS + c, x);
            tmem_wait_ld();
            reg_fence32(x);
            if (ONE || dual) {
              exp16(std::true_type{}, c, x, mb, y, y + 8);
              exp16(std::true_type{}, c + 16, x + 16, mb, y + 16, y + 24);
              tmem_st32(tS + c, y);
            } else {
              exp16(std::false_type{}, c, x, mb, y, nullptr);
              exp16(std::false_type{}, c + 16, x + 16, mb, y + 8, nullptr);
              tmem_st16(tS + c / 2, y);
            }
          }
          const float ts = pair_sum(acc);
          l += ts;
          lr += ONE || dual ? ts : pair_sum(accr);
        }
        tmem_wait_st();
        tc_fence_before();
        // On behalf of the MMA issuer: the next step's slot has been loaded.
        if (!ONE && warp == 0 && !dual) {
          ++vslot;
          if (!(ok = wait(&bars->kv_full[vslot % C::NS], (vslot / C::NS) & 1))) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
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
      float w0 = 1.f, w1 = 0.f;                         // of the own columns, of the other stream's
      int c_from = 0, c_to = D;
      if (dual) {
        // join the two streams: each warp takes half of the columns
        float* own = mls + (t * 128 + r) * 3;
        const float* oth = mls + ((t ^ 1) * 128 + r) * 3;
        own[0] = m_ref;
        own[1] = l;
        own[2] = lr;
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
        lr = fmaf(w0, lr, w1 * oth[2]);
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
          *reinterpret_cast<float4*>(ml) = make_float4(m_ref, l, lr, 0.f);
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
// is left alone.  One warp per row, D / 32 columns per lane;
// four parts' loads at a time, so that a row costs two waits for memory: what
// the parts are, and the parts.
template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedParams p, const int nctas) {
  grid_dependency_wait();
  const int c = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int4 it = p.part_meta[2 * c + 1];
  int kind = c + 1 + lane < nctas ? p.part_meta[2 * (c + 1 + lane)].x : 0;
  if (it.x == 0 || row >= it.z * p.group) return;
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
  Cols o;
#pragma unroll
  for (int i = 0; i < PER; ++i) o.v[i] = 0.f;
  float M = -INFINITY, l = 0.f, lr = 0.f;
  for (int s0 = 0; s0 < nparts; s0 += 4) {
    float4 ml[4];
    Cols x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = min(s0 + i, nparts - 1);
      const long long at = (long long)(s == 0 ? 2 * c + 1 : 2 * (c + s)) * p.part_rows + row;
      ml[i] = *reinterpret_cast<const float4*>(p.part_ml + at * 4);
      x[i] = *reinterpret_cast<const Cols*>(p.part_o + at * D + lane * PER);
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
  const float inv = lr > 0.f ? 1.f / lr : 0.f;
  const long long tok = it.y + row / p.group;
  const int h = it.w * p.group + row % p.group;
  const long long at = (tok * p.Hq + h) * D + lane * PER;
#pragma unroll
  for (int k = 0; k < PER; ++k) o.v[k] *= inv;
  if (p.o_f32) {
    *reinterpret_cast<Cols*>(static_cast<float*>(p.o) + at) = o;
  } else {
#pragma unroll
    for (int k = 0; k < PER; k += 2)
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + at + k) = pack_bf16x2(o.v[k], o.v[k + 1]);
  }
  if (lane == 0) p.lse[(long long)h * p.T + tok] = l == 0.f ? -INFINITY : (M + lg2_approx(l)) * kLn2;
}

template <int D, bool ALIBI, bool ONE>
int launch_impl(const PagedParams& p, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = fwd_paged_kernel<D, ALIBI, ONE>;
  if (const int ea = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return ea;
  CUtensorMap tq, tk, tv;
  const long long slots = (long long)p.num_pages * p.page_size;
  const int box = std::min(p.page_size, 128);
  int r = make_tmap_bf16_3d_box(&tq, p.q, D, p.Hq, p.T, p.group, p.tpt);
  if (!r) r = make_tmap_bf16_3d(&tk, p.k, D, p.Hkv, slots, box);
  if (!r) r = make_tmap_bf16_3d(&tv, p.v, D, p.Hkv, slots, box);
  if (r) return r;
  int nsm = 0;
  if (const int es = sm_count(&nsm)) return es;
  const int grid = std::min(nsm, kPagedCtas);
  kern<<<grid, kThreads, C::SMEM_BYTES, stream>>>(tq, tk, tv, p);
  if (const cudaError_t e = cudaGetLastError()) return (int)e;
  return launch_dependent(paged_merge_kernel<D>, dim3(grid, std::max(1, (p.part_rows + 7) / 8)), dim3(256), 0, stream, p, grid);
}

template <int D>
int launch_d(const PagedParams& p, cudaStream_t stream) {
  // no sequence brings more tokens than one tile holds
  const bool one = p.N <= p.tpt;
  if (p.alibi) return one ? launch_impl<D, true, true>(p, stream) : launch_impl<D, true, false>(p, stream);
  return one ? launch_impl<D, false, true>(p, stream) : launch_impl<D, false, false>(p, stream);
}

}  // namespace

#ifdef FA_PAGED_STOP
extern "C" int fa_selftest_paged_stop(int warp, int cta, int item) {
  const int at[3] = {warp, cta, item};
  return (int)cudaMemcpyToSymbol(g_stop, at, sizeof(at));
}
#endif

int launch_fwd_paged(const PagedParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return p.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace fa
