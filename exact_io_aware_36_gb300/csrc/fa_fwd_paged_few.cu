// fa_fwd_paged_few.cu -- attention over pages of e4m3 codes where a sequence
// brings few rows (new tokens x query heads of a kv head: at most 32 where no
// sequence of the call brings more, else at most those of one token), as in
// decoding: bound by the bytes of the cache.
//
//     S = scale Q K^T (+ ALiBi),   O = softmax(S) V,   k = 2^ek ck,  v = 2^ev cv
// with codes c and one pair of exponents for every 16 slots of a kv head.
//
// Two warps bring the codes, one the keys' and one the values': TMA into a ring of
// tiles of 128 keys and cp.async for their exponents, ahead and on into the next
// items.  (One warp is not enough: a TMA takes it about 140 cycles, a tile in
// pages of 32 slots takes 8 of them, and HBM 1400 for the tile.)  The others take
// steps of 32 keys in turn, each by itself (its own m, l and O), and meet
// when an item ends.
// Codes become fp16 (exact) in registers: two instructions for four of them.
// (mma.sync with e4m3 operands is no way around that: it is taken apart into the
// same conversions and fp16 products, and took 1.4 times as long.)
//   Q  is scaled by a power of two per row to at most 2^15 and rounded to fp16:
//      exact for elements down to 2^-22 of the row's largest, and what the
//      others lose is below 2^-39 of that one.
//   P  is rounded to fp16 once (11 bits); m is a reference that a row's scores
//      exceed by at most 2^8, and 2^7 P at most 2^15, so that P's normal range
//      reaches down to 2^-21 and its smallest step is 2^-31.
// O is over a power of two, that of the values it has met, until it is divided by l.
// Both products are taken transposed (S^T = K Q^T, O^T = V^T P^T): keys and
// elements of V fill the 16 rows of an instruction, and up to 8 rows of Q its
// columns, so that eight rows cost half of what 16 x 8 the other way round would
// (registers of O, products, exponentials).
//
// The work is cut as in fa_fwd_paged.cuh (equal runs of the line of key tiles,
// parts joined in a fixed order), so nothing depends on timing.  A warp whose
// wait for its copies runs out gives its items up: their rows are left alone.
#include <cuda_fp16.h>

#include "fa_fwd_paged.cuh"

namespace fa {
namespace {

template <int D, int NR>
struct Few {
  static constexpr int ROWS = 8 * NR;
  // Warps that take steps, beside the two that bring the codes; O alone takes D NR / 4
  // registers of a lane.  9 to 12 warps in all have 168 registers a lane, 8 have 255,
  // 13 to 16 have 128.  Measured with so many in all: one token of 16 caches (8 rows,
  // d = 128) 8 108.4 us, 10 107.9, 12 107.4, 14 112.7, 16 116.2 (the last two spill);
  // four tokens of such (16 rows) 8 99.4, 10 97.3, 12 104.8; seven tokens of 40
  // sequences (32 rows of 64) 8 62.5, 12 54.8; five of 32 (24 rows) 8 123, 10 203 (it
  // spills 404 bytes).  As chosen, 8 of the 16 instances spill 4 to 104 bytes.
  static constexpr int W = (NR * D <= 192 ? 12 : NR * D > 256 ? 8 : D == 128 ? 10 : 12) - 2;
  static constexpr int NT = 32 * (W + 2);
  // Blocks of a step that are taken together: both, unless that spills (32 rows).
  // 24 rows, d = 128 (five tokens of 32 sequences, 32 heads on 8): 123 us, with one
  // 131.
  static constexpr int XB = NR <= 3 ? 2 : 1;
  static constexpr int POOL = 128 * D;                      // codes of a tile in one pool
  static constexpr int TILE_BYTES = 2 * POOL;
  static constexpr int RED_STRIDE = 68;                     // floats per row of 64 columns
  // Q of an item and of the next, as fragments, the rows' exponents, their slopes
  static constexpr int Q_FRAGS = NR * (D / 16) * 256;
  static constexpr int Q_BYTES = Q_FRAGS + ROWS * 8;
  // Tiles of the ring: what the rest leaves of shared memory, at most 192 KB (what
  // HBM's latency asks for is about 60).
  static constexpr int REST = W * ROWS * (RED_STRIDE * 4 + 8) + ROWS * 12 + 2 * Q_BYTES + kSegs * 96 + 256 + kBarBytes + 1024;
  static constexpr int FIT = (227 * 1024 - REST) / (TILE_BYTES + 128 + 16);
  static constexpr int NS = FIT < 196608 / TILE_BYTES ? FIT : 196608 / TILE_BYTES;
  static constexpr int RING_OFF = 0;
  static constexpr int HEAD_OFF = RING_OFF + NS * TILE_BYTES;        // exponents of the tiles' blocks
  static constexpr int RED_OFF = HEAD_OFF + NS * 128;
  static constexpr int ML_OFF = RED_OFF + W * ROWS * RED_STRIDE * 4;
  static constexpr int STAT_OFF = ML_OFF + W * ROWS * 8;
  static constexpr int Q_OFF = STAT_OFF + ROWS * 8;
  static constexpr int TOK_OFF = Q_OFF + 2 * Q_BYTES;       // each row's token
  static constexpr int SEG_OFF = TOK_OFF + ROWS * 4;
  static constexpr int PAR_OFF = SEG_OFF + kSegs * 96;
  static constexpr int RINGBAR_OFF = PAR_OFF + 256;         // full and empty of the ring's tiles
  static constexpr int BAR_OFF = RINGBAR_OFF + NS * 16;
  static constexpr int SMEM_BYTES = BAR_OFF + kBarBytes + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  // Each tile's steps belong to different warps, and a warp's next step lies at
  // most NS - 1 tiles on.
  static_assert(W >= 4 && (W + 3) / 4 <= NS - 1, "ring");
  static_assert(kPagedMaxBatch * 8 <= NS * TILE_BYTES && NS >= 3, "plan");
  static_assert(Q_OFF % 16 == 0 && Q_BYTES % 16 == 0 && RED_OFF % 16 == 0 && BAR_OFF % 8 == 0, "alignment");
};

// D += A B: 16 x 8, over 16.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four codes as fp16: the low two, the high two.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

// An 8 x 8 matrix of 16-bit elements, transposed: row lane / 4, columns 2 (lane %
// 4) and the next.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" :: "r"(smem_u32(bar)), "r"(n) : "memory");
}

template <int D, int NR, bool ALIBI>
__global__ void __launch_bounds__(Few<D, NR>::NT, 1)
fwd_paged_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PagedParams p) {
  using C = Few<D, NR>;
  constexpr int W = C::W, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedParams& ps = *reinterpret_cast<const PagedParams*>(smem + C::PAR_OFF);
  if (threadIdx.x < sizeof(PagedParams) / 4)
    reinterpret_cast<uint32_t*>(smem + C::PAR_OFF)[threadIdx.x] = reinterpret_cast<const uint32_t*>(&p)[threadIdx.x];
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + C::RINGBAR_OFF);
  uint64_t* const empty = full + NS;
  if (threadIdx.x < NS) {
    mbar_init(&full[threadIdx.x], 2 * (1 + 8));        // of each pool the codes and eight exponents
    mbar_init(&empty[threadIdx.x], 4);                 // the tile's steps
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      mbar_init(&bars->seg_empty[i], W + 1);           // all but the warp that finds them
    }
#ifdef FA_PAGED_STOP
    mbar_init(&bars->never, 1);
#endif
    bars->abort_flag = bars->part_lost[0] = bars->part_lost[1] = 0;
    bars->unit = -1000;
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  fence_mbarrier_init();
  __syncthreads();
  make_plan<C::NT, true>(ps, bars, reinterpret_cast<unsigned long long*>(smem + C::RING_OFF), kWeightOne + 2);
  fence_proxy_async_smem();                            // (the plan's sums lay where TMA will write)
  __syncthreads();
  grid_launch_dependents();
  const WaitCtx wc{&bars->abort_flag, p.status};
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_warp_inl(bar, parity, wc); };
  // The run's items: segs[n % kSegs] is item n (ie < 0: the end).
  Seg* segs = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  auto wait_seg = [&](int n) -> bool {
#ifdef FA_PAGED_STOP
    if (warp == g_stop[0] && (int)blockIdx.x == g_stop[1] && n == g_stop[2])
      return wait_warp(&bars->never, 0, WaitCtx{&bars->abort_flag, p.status, kStopLimitNs});
#endif
    return wait(&bars->seg_full[n % kSegs], (n / kSegs) & 1);
  };
  auto first_step = [](const Seg& s) { return max((s.k.hi_all - s.ie + 1) * 4, s.k.vlo >> 5); };
  auto end_step = [](const Seg& s) { return min((s.k.hi_all - s.ib + 1) * 4, (s.k.vhi + 31) >> 5); };

  if (warp >= W) {
    // ----------------------------------------------------------- producers
    // Warp W brings the keys' codes and finds the run's items, one ahead of the
    // tiles it fetches; warp W + 1 brings the values'.  Two tiles at a time, as most
    // of what a tile costs them does not depend on how many there are (1200 cycles
    // one by one, of 1400 that HBM takes).  A tile is 128 / page_size boxes, one lane
    // each (one of them for larger pages), and lane i of its eight brings the
    // exponents of block i.
    const bool values = warp > W;
    const int second = lane >> 3 & 1, blk = lane & 7;  // (lanes 16 .. 31: as 0 .. 15, but without a copy)
    Walk w;
    Seg s;
    s.lost = 0;
    // what the parts of this CTA are, for the merge: kind of the part that goes on
    // from the CTA before (2: the item's last), and the item begun here
    int cont = 0;
    int4 begun = make_int4(0, 0, 0, 0);
    bool more = true, ok = true;
    auto publish = [&](int n) {
      if (n >= kSegs && !wait(&bars->seg_empty[n % kSegs], (n / kSegs - 1) & 1)) return false;
      more = walk_next<true>(p, w, s);
      if (more) {
        if (s.ib > 0) cont = s.ie == s.k.kt ? 2 : 1;
        else if (s.ie < s.k.kt) begun = make_int4(1, s.tok, s.ntok, s.g);
      } else {
        s.ie = -1;
      }
      if (lane == 0) {
        segs[n % kSegs] = s;
        mbar_arrive(&bars->seg_full[n % kSegs]);
      }
      __syncwarp();
      return true;
    };
    const long long scale_bytes = (long long)p.num_pages * (p.page_size >> 4) * p.Hkv;
    const uint8_t* const scales = values ? p.v_scales : p.k_scales;
    const CUtensorMap* const tm = values ? &tmV : &tmK;
    const int box_rows = min(p.page_size, 128), boxes = 128 / box_rows;
    constexpr int kNoPage = -0x7fffffff - 1;           // no row sees these keys
    int place = 0;                                     // of the next tile in the ring
    unsigned par = 1;                                  // parity of its last emptying (at first none is waited for)
    if (!values) {
      walk_begin<true>(p, bars, w);
      ok = publish(0);
    }
    for (int n = 0; ok; ++n) {
      if (values) {
        if (!(ok = wait_seg(n))) break;
        s = segs[n % kSegs];
        more = s.ie >= 0;
      }
      if (!more) break;
      const int b0 = first_step(s), b1 = end_step(s), head = s.g, vlo = s.k.vlo, vhi = s.k.vhi;
      const int32_t* table = p.block_table + (long long)s.b * p.max_pages;
      int* const lost = &segs[n % kSegs].lost;
      // page of the lane's 16 slots of its tile
      auto look_up = [&](int tile) {
        const int key = ((tile + second) << 7) + 16 * blk;
        return key < vhi && key + 16 > vlo ? max(__ldg(table + (key >> p.page_shift)), -1) : kNoPage;
      };
      int tile = b0 >> 2;
      const int end = b0 < b1 ? (b1 + 3) >> 2 : tile;
      int page = tile < end ? look_up(tile) : kNoPage;
      if (!values && !(ok = publish(n + 1))) break;
      for (; tile < end; tile += 2) {
        const int next_page = tile + 2 < end ? look_up(tile + 2) : kNoPage;
        // this lane's tile and its place; the second may be missing
        const bool there = tile + second < end;
        int at_place = place + second;
        const bool over = at_place >= NS;
        if (over) at_place -= NS;
        if (!(ok = wait(&empty[there ? at_place : place], there && over ? par ^ 1 : par))) break;
        if (!there) page = kNoPage;
        const bool good = (unsigned)page < (unsigned)p.num_pages;
        // a page that is not there is not read, and the item's rows are not written
        const bool bad = __any_sync(0xffffffffu, !good && page != kNoPage);
        const int key = ((tile + second) << 7) + 16 * blk;
        const uint32_t row = good ? (uint32_t)page * p.page_size + (key & (p.page_size - 1)) : 0;
        const bool copies = lane < 16 && there;
        if (copies) {
          const uint32_t hd = smem_u32(smem + C::HEAD_OFF) + at_place * 128 + blk * 16;
          const long long j = good ? (long long)(row >> 4) * p.Hkv + head : 0;
          copy_async4(hd + 4 * values, scales + (j & ~3ll), good ? (int)min(4ll, scale_bytes - (j & ~3ll)) : 0);
          if (!values) sts32(hd + 8, (uint32_t)(j & 3) * 8);
        }
        // The box of the tile's lane i begins at block i box_rows / 16.  Its page is
        // known to the lane of any of its blocks that a row sees.
        const int blocks = box_rows >> 4;              // of a box
        const unsigned seen = __ballot_sync(0xffffffffu, good) >> (8 * second) & 0xffu;
        const unsigned mine = blk < boxes ? seen >> (blk * blocks) & ((1u << blocks) - 1) : 0;
        const uint32_t row_of = __shfl_sync(0xffffffffu, row, 8 * second + (mine ? blk * blocks + __ffs(mine) - 1 : 0));
        const int fetched = __popc(__ballot_sync(0xffffffffu, mine != 0) >> (8 * second) & 0xffu);
        __syncwarp();                                  // lanes 0 and 8 publish what the others wrote
        if (copies && blk == 0) {
          if (bad) {
            record_status(p.status, FA_ERR_PAGE);
            *lost = 1;
          }
          mbar_arrive_expect_tx(&full[at_place], fetched * box_rows * D);
        }
        __syncwarp();
        if (copies && mine)
          tma_load_3d(smem + C::RING_OFF + at_place * C::TILE_BYTES + (values ? C::POOL : 0) + blk * box_rows * D, tm, 0, head,
                      (int)row_of & ~(box_rows - 1), &full[at_place]);
        if (copies) copies_arrive(&full[at_place]);
        __syncwarp();
        place += min(2, end - tile);
        if (place >= NS) {
          place -= NS;
          par ^= 1;
        }
        page = next_page;
      }
      if (values) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_empty[n % kSegs]);
      }
    }
    // Copies in flight must land before this CTA's shared memory goes away: of
    // every place that was filled (its parity: the emptying it waited for, turned).
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int i = 0; i < NS; ++i) wait_warp_drain(&full[i], (i < place ? par : par ^ 1) ^ 1);
    __syncthreads();
    // A wait ran out, so parts may be missing: the merge must not take what the
    // workspace held.  Nor a part of an item that met a page outside the pool.
    grid_dependency_wait();                            // (see the end of the kernel)
    if (!values && lane < 2)
      p.part_meta[2 * blockIdx.x + lane] = bars->abort_flag || bars->part_lost[lane] ? make_int4(0, 0, 0, 0)
                                           : lane ? begun : make_int4(cont, 0, 0, 0);
    return;
  }

  // -------------------------------------------------------- the other warps
  if (threadIdx.x < C::ROWS) reinterpret_cast<int*>(smem + C::TOK_OFF)[threadIdx.x] = (int)threadIdx.x / p.group;
  auto meet = [] { named_bar_sync(1, 32 * W); };       // barrier of these warps
  // ---- Q: a warp prepares rows warp, warp + W, .. of the next item, a lane D /
  // 32 elements, while it works on this one
  constexpr int QP = (C::ROWS + W - 1) / W;
  constexpr int QE = D / 32;
  uint32_t xq[QP][QE / 2];
  float xslope[QP];
  auto load_q = [&](const Seg& s) {
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int r = warp + i * W;
#pragma unroll
      for (int j = 0; j < QE / 2; ++j) xq[i][j] = 0;
      xslope[i] = 0.f;
      if (r < s.ntok * p.group) {
        const int tok = r / p.group, hq = s.g * p.group + r - tok * p.group;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                ((long long)(s.tok + tok) * p.Hq + hq) * D + QE * lane);
        if (D == 128) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
          xq[i][0] = v.x;
          xq[i][QE / 2 - 1] = v.y;
        } else {
          xq[i][0] = __ldg(src);
        }
        if (ALIBI) xslope[i] = __ldg(p.alibi + hq) * kLog2e;
      }
    }
  };
  // Fragment k of 8 rows is 8 bytes of every lane: elements (D / 4) c4 + 4 k .. + 3
  // of row g8 (g8 = lane / 4, c4 = lane % 4); two of them lie side by side.
  auto store_q = [&](int n) {
    uint8_t* at = smem + C::Q_OFF + (n & 1) * C::Q_BYTES;
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int r = warp + i * W;
      if (r >= C::ROWS) break;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < QE / 2; ++j) top = max(top, max(xq[i][j] << 16 & 0x7fff0000u, xq[i][j] & 0x7fff0000u));
      top = __reduce_max_sync(0xffffffffu, top);
      // the largest element to [2^14, 2^15)
      const int up = min(14 - (max((int)(top >> 23), 1) - 127), 127);
      const float mul = pow2_cut(up);
      const int k = D == 128 ? lane & 7 : (lane & 7) >> 1, to_lane = (r & 7) * 4 + (lane >> 3);
      uint32_t* frag = reinterpret_cast<uint32_t*>(at + ((r >> 3) * (D / 32) + (k >> 1)) * 512 + to_lane * 16 + (k & 1) * 8);
#pragma unroll
      for (int j = 0; j < QE / 2; ++j)
        frag[D == 128 ? j : lane & 1] =
            pack_f16x2(__uint_as_float(xq[i][j] << 16) * mul, __uint_as_float(xq[i][j] & 0xFFFF0000u) * mul);
      if (lane == 0) {
        reinterpret_cast<int*>(at + C::Q_FRAGS)[r] = up;
        reinterpret_cast<float*>(at + C::Q_FRAGS)[C::ROWS + r] = xslope[i];
      }
    }
  };
  // Items n and n + 1 are known; the same answer for every warp.
  auto known = [&](int n) {
    bool ok = wait_seg(n);
    if (ok && segs[n % kSegs].ie >= 0) ok = wait_seg(n + 1);
    return !named_bar_any(1, 32 * W, !ok);
  };
  bool go = known(0) && segs[0].ie >= 0;
  if (go) {
    load_q(segs[0]);
    store_q(0);
    meet();
  }

  const int g8 = lane >> 2, c4 = lane & 3;
  float* red = reinterpret_cast<float*>(smem + C::RED_OFF);
  float2* mls = reinterpret_cast<float2*>(smem + C::ML_OFF);
  float2* stat = reinterpret_cast<float2*>(smem + C::STAT_OFF);
  bool dead = false;                                   // a wait for a step ran out
  int turn = warp;                                     // this warp's first step of the item
  int from = 0;                                        // place of the item's first tile in the ring
  unsigned par = 0;                                    // parity of its filling

#pragma unroll 1
  for (int cur = 0; go; ++cur) {
    const Seg& s = segs[cur % kSegs];
    const bool next = segs[(cur + 1) % kSegs].ie >= 0;
    if (next) load_q(segs[(cur + 1) % kSegs]);
    const int rows = s.ntok * p.group;
    const int f = s.k.f[0];
    // blocks beyond `diag` or below `low` hold keys that some row does not see
    const int diag = p.causal ? f : s.L - 1, low = f + s.ntok - 1 - p.window;
    const uint32_t qat = smem_u32(smem + C::Q_OFF + (cur & 1) * C::Q_BYTES) + lane * 16;
    uint32_t qf[NR == 1 ? D / 16 : 1][2];              // of 8 rows they stay in registers
    if (NR == 1) {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2) {
        const uint4 v = lds128(qat + (k >> 1) * 512);
        qf[NR == 1 ? k : 0][0] = v.x;
        qf[NR == 1 ? k : 0][1] = v.y;
        qf[NR == 1 ? k + 1 : 0][0] = v.z;
        qf[NR == 1 ? k + 1 : 0][1] = v.w;
      }
    }
    // A lane's rows are 8 n + 2 c4 and the next; what is kept of each beside m and l
    // lies in shared memory.
    const uint32_t row_at = smem_u32(smem + C::Q_OFF + (cur & 1) * C::Q_BYTES + C::Q_FRAGS) + 8 * c4;
    const uint32_t tok_at = smem_u32(smem + C::TOK_OFF) + 8 * c4;
    float mref[NR][2], l[NR][2];
    float o[NR][D / 16][4];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      mref[n][0] = mref[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][t][i] = 0.f;
    }
    int eref = -1000, etop = -1000;                    // O's unit, the largest it had
    // ------------------------------------------------------------- steps
    const int b0 = first_step(s), b1 = max(end_step(s), b0), vlo = s.k.vlo, vhi = s.k.vhi;
    const int tile0 = b0 >> 2;
#pragma unroll 1
    for (int b = b0 + turn; b < b1; b += W) {
      const int nth = from + (b >> 2) - tile0, place = nth % NS;
      const unsigned lap = par ^ (nth / NS & 1);
      // A wait for one parity of a barrier says that the last phase of that parity
      // is over, so it must not be asked two phases ahead.  This warp's tile is at
      // most NS - 1 behind one that it saw full (or behind the last item's, which
      // all saw), and tiles are filled in order: when that one was, the fill of this
      // place before the last had been used up.  So first the wait for the last
      // one's being used up, then that for this fill.
      if (dead || !wait(&empty[place], lap ^ 1) || !wait(&full[place], lap)) {
        // this item's rows and those of all that follow are left alone
        dead = true;
        if (lane == 0) segs[cur % kSegs].lost = 1;
        break;
      }
      const uint32_t at = smem_u32(smem + C::RING_OFF) + place * C::TILE_BYTES + (b & 3) * 32 * D;
      const uint32_t heads = smem_u32(smem + C::HEAD_OFF) + place * 128 + (b & 3) * 32;
      const int k0 = b << 5;
      const bool masked = k0 + 31 > diag || k0 < low;
#pragma unroll 1
      for (int y = 0; y < 2; y += C::XB) {             // blocks y .. y + XB - 1
        if (C::XB == 1 && !(y ? k0 + 16 < vhi : k0 + 16 > vlo)) continue;
        constexpr int XB = C::XB;
        // S transposed, 16 keys x 8 rows: row g8 and g8 + 8 of a block, columns 2 c4 and
        // the next
        float sc[NR][XB][4];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int x = 0; x < XB; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[n][x][i] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint4 kw[2 * XB];
          // (d = 128: pieces 2 c4 and 2 c4 + 1 of a row, swizzled by it, so that the
          // rows of eight lanes take different places of a line)
#pragma unroll
          for (int t = 0; t < 2 * XB; ++t)
            kw[t] = lds128(at + (16 * y + 8 * t + g8) * D + (D == 128 ? (2 * c4 + i) ^ g8 : c4 ^ (g8 >> 1)) * 16);
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            uint4 q[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n)
              q[n] = NR > 1 ? lds128(qat + (n * (D / 32) + 2 * i + (k >> 1)) * 512)
                            : make_uint4(qf[NR == 1 ? 4 * i + k : 0][0], qf[NR == 1 ? 4 * i + k : 0][1],
                                         qf[NR == 1 ? 4 * i + k + 1 : 0][0], qf[NR == 1 ? 4 * i + k + 1 : 0][1]);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int x = 0; x < XB; ++x) {
                uint32_t a[4];
                codes_f16(reinterpret_cast<const uint32_t*>(&kw[2 * x])[k + kk], a[0], a[2]);
                codes_f16(reinterpret_cast<const uint32_t*>(&kw[2 * x + 1])[k + kk], a[1], a[3]);
#pragma unroll
                for (int n = 0; n < NR; ++n) mma_f16(sc[n][x], a, kk ? q[n].z : q[n].x, kk ? q[n].w : q[n].y);
              }
          }
        }
        // Scores in log2 units are x cs (+ the bias); -inf where a row does not see
        // a key.  With a bias, or where a row does not see all, they are made here.
        int ek[XB], ev[XB];
#pragma unroll
        for (int x = 0; x < XB; ++x) {
          const uint4 hd = lds128(heads + (y + x) * 16);
          ek[x] = exponent_of(hd.x, hd.z);
          ev[x] = exponent_of(hd.y, hd.z);
        }
        if (XB == 2) {                                   // (a block that no row sees has no exponents)
          if (k0 + 16 <= vlo) ev[0] = ev[XB - 1];
          if (k0 + 16 >= vhi) ev[XB - 1] = ev[0];
        }
        float cs[NR][2][XB];                             // of a row's blocks
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const uint2 up = lds64(row_at + 32 * n);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < XB; ++x) cs[n][j][x] = p.scale_log2 * pow2_cut(ek[x] - (int)(j ? up.y : up.x));
        }
        if (ALIBI || masked) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const uint2 slopes = lds64(row_at + 32 * n + 4 * C::ROWS), toks = lds64(tok_at + 32 * n);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // the last key that the row sees; a row without a token sees none
              const int r = 8 * n + 2 * c4 + j;
              const int kend = r >= rows ? -1 : p.causal ? f + (int)(j ? toks.y : toks.x) : s.L - 1;
              const float slope2 = __uint_as_float(j ? slopes.y : slopes.x);
#pragma unroll
              for (int x = 0; x < XB; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float& v = sc[n][x][2 * h + j];
                  const int key = k0 + 16 * (y + x) + 8 * h + g8;
                  v = ALIBI ? fmaf(v, cs[n][j][x], slope2 * (float)(key - kend)) : v * cs[n][j][x];
                  if (masked && (key > kend || (p.causal && key < kend - p.window))) v = -INFINITY;
                }
              cs[n][j][0] = cs[n][j][XB - 1] = 1.f;
            }
          }
        }
        float mx[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mx[n][j] = fmaxf(sc[n][0][j], sc[n][0][2 + j]) * cs[n][j][0];
            if (XB == 2) mx[n][j] = fmaxf(mx[n][j], fmaxf(sc[n][XB - 1][j], sc[n][XB - 1][2 + j]) * cs[n][j][XB - 1]);
            raise |= mx[n][j] > mref[n][j] + kTau;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float x = mx[n][j];
#pragma unroll
              for (int q = 4; q < 32; q <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, q));
              const bool up = x > mref[n][j] + kTau;
              const float alpha = up ? ex2_approx(mref[n][j] - x) : 1.f;
              if (up) mref[n][j] = x;
              l[n][j] *= alpha;
#pragma unroll
              for (int t = 0; t < D / 16; ++t) {
                o[n][t][j] *= alpha;
                o[n][t][2 + j] *= alpha;
              }
            }
        }
        // O's unit follows the values' exponents, at most 2^80 below the largest so
        // far (which O's float32 holds).  Two blocks further apart than 2^8 take the
        // products one after the other (the other's P is 0).
        const int top = max(ev[0], ev[XB - 1]), bottom = min(ev[0], ev[XB - 1]);
        const int passes = XB == 2 && top - bottom > 8 ? 2 : 1;
#pragma unroll 1
        for (int pass = 0; pass < passes; ++pass) {
          const int own = pass ? ev[XB - 1] : ev[0], hi = passes == 1 ? top : own, lo = passes == 1 ? bottom : own;
          if (hi > eref || lo < eref - 8) {
            etop = max(etop, hi);
            const int e = max(hi, etop - 80);
            const float alpha = pow2_cut(eref - e);
            eref = e;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][t][i] *= alpha;
          }
          // P in O's unit: 2^(x - m + ev - eref + 7); its sum is brought back to 1.
          // (x - m is at most 8, so with 2^-60 and less P is 0 in f16; a smaller
          // one would make 0 of it in float32 too, and l would miss the key.)
          float lsv[XB], back[XB];
#pragma unroll
          for (int x = 0; x < XB; ++x) {
            const int up = max(ev[x] - eref + 7, -60);
            const bool on = passes == 1 || pass == x;
            lsv[x] = on ? (float)up : -1e6f;
            back[x] = pow2_cut(-up);
          }
          uint32_t pf[NR][XB][2];
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float mr[2] = {mref[n][0] == -INFINITY ? 0.f : mref[n][0], mref[n][1] == -INFINITY ? 0.f : mref[n][1]};
#pragma unroll
            for (int x = 0; x < XB; ++x) {
              float e[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = ex2_approx(fmaf(sc[n][x][i], cs[n][i & 1][x], lsv[x] - mr[i & 1]));
#pragma unroll
              for (int j = 0; j < 2; ++j) l[n][j] = fmaf(e[j] + e[2 + j], back[x], l[n][j]);
              pf[n][x][0] = transposed(pack_f16x2(e[0], e[1]));
              pf[n][x][1] = transposed(pack_f16x2(e[2], e[3]));
            }
          }
          // O transposed, 16 elements x 8 rows, D / 16 times: row g8 of product t is
          // element g8 D / 8 + 2 t, row g8 + 8 the next
#pragma unroll
          for (int x = 0; x < XB; ++x) {
            const uint32_t vat = at + C::POOL + (y + x) * 16 * D;
            uint32_t w[4][D / 32];                       // of the block's keys 2 c4, 2 c4 + 1, 8 + 2 c4, 9 + 2 c4
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * (i >> 1) + 2 * c4 + (i & 1);
              if (D == 128) {
                const uint4 v = lds128(vat + r * 128 + (g8 ^ (r & 7)) * 16);
                w[i][0] = v.x;
                w[i][1] = v.y;
                w[i][D / 32 - 2] = v.z;
                w[i][D / 32 - 1] = v.w;
              } else {
                const uint2 v = lds64(vat + r * 64 + ((g8 >> 1) ^ (r >> 1 & 3)) * 16 + (g8 & 1) * 8);
                w[i][0] = v.x;
                w[i][1] = v.y;
              }
            }
            // a slot that no row sees may hold NaN, and 0 x NaN would reach O
            if (masked && (k0 < vlo || k0 + 32 > vhi)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = k0 + 16 * (y + x) + 8 * (i >> 1) + 2 * c4 + (i & 1);
                if (key < vlo || key >= vhi)
#pragma unroll
                  for (int j = 0; j < D / 32; ++j) w[i][j] = 0;
              }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              uint32_t b0[4], b1[4];
              codes_f16(__byte_perm(w[0][i], w[1][i], 0x5140), b0[0], b0[1]);
              codes_f16(__byte_perm(w[0][i], w[1][i], 0x7362), b0[2], b0[3]);
              codes_f16(__byte_perm(w[2][i], w[3][i], 0x5140), b1[0], b1[1]);
              codes_f16(__byte_perm(w[2][i], w[3][i], 0x7362), b1[2], b1[3]);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1]};
#pragma unroll
                for (int n = 0; n < NR; ++n) mma_f16(o[n][2 * i + j], a, pf[n][x][0], pf[n][x][1]);
              }
            }
          }
        }
      }
      __syncwarp();
      // (the first step of a tile that has fewer than four arrives for the others)
      if (lane == 0) {
        const int lo = max(b & ~3, b0), hi = min((b & ~3) + 4, b1);
        mbar_arrive_n(&empty[place], b == lo ? 5 - (hi - lo) : 1);
      }
    }
    // the next item's first step and tile
    turn -= (b1 - b0) % W;
    if (turn < 0) turn += W;
    from += b0 < b1 ? ((b1 + 3) >> 2) - tile0 : 0;
    par ^= from / NS & 1;
    from %= NS;
    if (next) store_q(cur + 1);
    // ------------------------------------------------- join the warps' parts
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[n][j];
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) x += __shfl_xor_sync(0xffffffffu, x, q);
        if (g8 == 0) mls[warp * C::ROWS + 8 * n + 2 * c4 + j] = make_float2(mref[n][j], x);
      }
    if (lane == 0) atomicMax(&bars->unit, etop);
    meet();
    // O stays over the values' largest power of two that a warp met until it is divided:
    // what it is before may not be a float.
    const int unit = *(volatile int*)&bars->unit;
    if (threadIdx.x < rows) {
      float M = -INFINITY, L = 0.f;
      for (int w = 0; w < W; ++w) M = fmaxf(M, mls[w * C::ROWS + threadIdx.x].x);
      for (int w = 0; w < W; ++w) {
        const float2 ml = mls[w * C::ROWS + threadIdx.x];
        L = fmaf(ml.x == M ? 1.f : ex2_approx(ml.x - M), ml.y, L);
      }
      stat[threadIdx.x] = make_float2(M, L);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float M = -INFINITY;
        for (int w = 0; w < W; ++w) M = fmaxf(M, mls[w * C::ROWS + 8 * n + 2 * c4 + j].x);
        const float a = (mref[n][j] == M ? 1.f : ex2_approx(mref[n][j] - M)) * pow2_cut(eref - unit);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          o[n][t][j] *= a;
          o[n][t][2 + j] *= a;
        }
      }
    const int part = s.ib > 0 ? 1 : s.ie < s.k.kt ? 2 : 0;
    const long long prow = (long long)(2 * (int)blockIdx.x + part - 1) * p.part_rows;
    const bool f32 = part || p.o_f32;                  // a part is float32, not divided
    const int kept = part && unit >= -127 ? part_power(unit, -7) : 0;
    const float opow = pow2_any(unit - 7 - kept);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {                 // 64 columns at a time
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * n + 2 * c4 + j;
          if (r < rows) {
            float* at = red + (warp * C::ROWS + r) * C::RED_STRIDE + 8 * g8;
#pragma unroll
            for (int q = 0; q < 2; ++q)
              *reinterpret_cast<float4*>(at + 4 * q) = make_float4(o[n][4 * c + 2 * q][j], o[n][4 * c + 2 * q][2 + j],
                                                                   o[n][4 * c + 2 * q + 1][j], o[n][4 * c + 2 * q + 1][2 + j]);
          }
        }
      meet();
      const bool lost = s.lost != 0;
      if (lost && part && threadIdx.x == 0) bars->part_lost[part - 1] = 1;
      if (threadIdx.x == 0) bars->unit = -1000;        // (read by all)
      for (int i = threadIdx.x; i < rows * 16 && !lost; i += 32 * W) {
        const int r = i >> 4, x = (i & 15) * 4;        // four columns of row r
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < W; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(red + (w * C::ROWS + r) * C::RED_STRIDE + x);
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
        const float2 ml = stat[r];
        const int tok = r / p.group, hq = s.g * p.group + r % p.group;
        const int col = (x >> 3) * (D / 8) + 8 * c + (x & 7);
        if (part == 0) {
          const float inv = ml.y > 0.f ? 1.f / ml.y : 0.f;
          v.x *= inv;
          v.y *= inv;
          v.z *= inv;
          v.w *= inv;
        }
        v.x *= opow;
        v.y *= opow;
        v.z *= opow;
        v.w *= opow;
        const long long at = part ? (prow + r) * D + col : ((long long)(s.tok + tok) * p.Hq + hq) * D + col;
        if (f32) {
          *reinterpret_cast<float4*>((part ? p.part_o : static_cast<float*>(p.o)) + at) = v;
        } else {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
        if (c == 0 && x == 0) {
          if (part)
            *reinterpret_cast<float4*>(p.part_ml + (prow + r) * 4) = make_float4(ml.x, ml.y, ml.y, __int_as_float(kept));
          else
            p.lse[(long long)hq * p.T + s.tok + tok] = ml.y == 0.f ? -INFINITY : (ml.x + lg2_approx(ml.y)) * kLn2;
        }
      }
      meet();
    }
    if (lane == 0) mbar_arrive(&bars->seg_empty[cur % kSegs]);
    go = next && known(cur + 1);
  }
  __syncthreads();
  // The call's other kernel may still run; what follows this one must find both
  // at their end.
  grid_dependency_wait();
}

template <int D, int NR>
int launch_few(const PagedParams& p, int grid, bool after, cudaStream_t stream) {
  using C = Few<D, NR>;
  auto kern = p.alibi ? fwd_paged_few_kernel<D, NR, true> : fwd_paged_few_kernel<D, NR, false>;
  if (const int e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return e;
  CUtensorMap tk, tv;
  const long long slots = (long long)p.num_pages * p.page_size;
  if (const int e = make_tmap_codes_3d(&tk, p.k, D, p.Hkv, slots, 1, std::min(p.page_size, 128))) return e;
  if (const int e = make_tmap_codes_3d(&tv, p.v, D, p.Hkv, slots, 1, std::min(p.page_size, 128))) return e;
  if (after) return launch_dependent(kern, dim3(grid), dim3(C::NT), C::SMEM_BYTES, stream, tk, tv, p);
  kern<<<grid, C::NT, C::SMEM_BYTES, stream>>>(tk, tv, p);
  return (int)cudaGetLastError();
}

}  // namespace

#ifdef FA_PAGED_STOP
extern "C" int fa_selftest_paged_few_stop(int warp, int cta, int item) {
  const int at[3] = {warp, cta, item};
  return (int)cudaMemcpyToSymbol(g_stop, at, sizeof(at));
}
#endif

int launch_fwd_paged_few(PagedParams p, int grid, bool after, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (p.few_rows <= 8) return p.d == 128 ? launch_few<128, 1>(p, grid, after, stream) : launch_few<64, 1>(p, grid, after, stream);
  if (p.few_rows <= 16) return p.d == 128 ? launch_few<128, 2>(p, grid, after, stream) : launch_few<64, 2>(p, grid, after, stream);
  if (p.few_rows <= 24) return p.d == 128 ? launch_few<128, 3>(p, grid, after, stream) : launch_few<64, 3>(p, grid, after, stream);
  return p.d == 128 ? launch_few<128, 4>(p, grid, after, stream) : launch_few<64, 4>(p, grid, after, stream);
}

}  // namespace fa
