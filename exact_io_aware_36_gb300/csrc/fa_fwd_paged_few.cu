// fa_fwd_paged_few.cu -- attention over pages of e4m3 codes where a sequence
// brings few rows (new tokens x query heads of a kv head: at most 32), as in
// decoding: bound by the bytes of the cache.
//
//     S = scale Q K^T (+ ALiBi),   O = softmax(S) V,   k = 2^ek ck,  v = 2^ev cv
// with codes c and one pair of exponents for every 16 slots of a kv head.
//
// A warp takes such a block of 16 keys by itself: its codes come from HBM by
// cp.async into a ring of its own, several blocks ahead and on into the next
// items, and no warp waits for another until an item ends.  The codes become
// fp16 in registers (exact) and go straight into matrix instructions of 16 rows:
// their order along d (and along the keys, for P V) is free as long as both
// operands agree, so each lane's operands are whole 16-byte reads.  The
// exponents stay out of the products: 2^ek multiplies a block's scores, and
// 2^(ev - eref) its P, with O held in units of 2^eref.
//   Q  is scaled by a power of two per row to at most 2^15 and rounded to fp16:
//      exact for elements down to 2^-22 of the row's largest, and what the
//      others lose is below 2^-39 of that one.
//   P  is rounded to fp16 once (11 bits); m is a reference that a row's scores
//      exceed by at most 2^8, and 2^7 P at most 2^15, so that P's normal range
//      reaches down to 2^-21 and its smallest step is 2^-31.
// What a 16-row instruction leaves unused does not matter: 128 keys cost an SM
// some 130 cycles of the matrix pipe and 1500 of its share of HBM at d = 128.
//
// The work is cut as in fa_fwd_paged.cuh (equal runs of the line of key tiles,
// parts joined in a fixed order), so nothing depends on timing.  There is no
// wait that could run out.
#include <cuda_fp16.h>

#include "fa_fwd_paged.cuh"

namespace fa {
namespace {

template <int D, int MT>
struct Few {
  static constexpr int ROWS = 16 * MT;
  // Warps: as many as the registers of O (D MT / 2 of a lane), Q and the codes
  // leave room for.
  static constexpr int W = D == 128 ? (MT == 1 ? 12 : 8) : (MT == 1 ? 16 : 12);
  static constexpr int NT = 32 * W;
  static constexpr int RD = D == 128 && MT == 1 ? 3 : 4;    // blocks of a warp's ring
  static constexpr int POOL = 16 * D;                       // codes of a block in one pool
  static constexpr int BLOCK_BYTES = 2 * POOL + 16;
  static constexpr int RED_STRIDE = 68;                     // floats per row of 64 columns
  static constexpr int RING_OFF = 0;
  static constexpr int RED_OFF = RING_OFF + W * RD * BLOCK_BYTES;
  static constexpr int ML_OFF = RED_OFF + W * ROWS * RED_STRIDE * 4;
  static constexpr int STAT_OFF = ML_OFF + W * ROWS * 8;
  static constexpr int SEG_OFF = STAT_OFF + ROWS * 8;
  static constexpr int PAR_OFF = SEG_OFF + 4 * 96;
  static constexpr int BAR_OFF = PAR_OFF + 256;
  static constexpr int SMEM_BYTES = BAR_OFF + 512 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(kPagedMaxBatch * 8 <= W * RD * BLOCK_BYTES, "plan");
  static_assert(SEG_OFF % 16 == 0 && RED_OFF % 16 == 0, "alignment");
};

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two codes (four) as fp16.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^e, the exponent cut to what a float holds.
__device__ __forceinline__ float pow2_cut(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }

__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

template <int D, int MT, bool ALIBI>
__global__ void __launch_bounds__(Few<D, MT>::NT, 1) fwd_paged_few_kernel(const __grid_constant__ PagedParams p) {
  using C = Few<D, MT>;
  constexpr int W = C::W;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedParams& ps = *reinterpret_cast<const PagedParams*>(smem + C::PAR_OFF);
  if (threadIdx.x < sizeof(PagedParams) / 4)
    reinterpret_cast<uint32_t*>(smem + C::PAR_OFF)[threadIdx.x] = reinterpret_cast<const uint32_t*>(&p)[threadIdx.x];
  if (threadIdx.x == 0) bars->part_lost[0] = bars->part_lost[1] = 0;
  __syncthreads();
  make_plan<C::NT, true>(ps, bars, reinterpret_cast<unsigned long long*>(smem + C::RING_OFF), kMinRunOne);
  grid_launch_dependents();

  // The run's items: segs[n % 4] is item n (ie < 0: the end).  Warp 0 finds them,
  // two ahead; each is published by the barrier of an item's end.
  Seg* segs = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  Walk walk;
  int cont = 0;
  int4 begun = make_int4(0, 0, 0, 0);
  bool more = true;
  auto find = [&](int n) {
    if (!more) return;
    Seg s;
    s.lost = 0;
    more = walk_next<true>(p, walk, s);
    if (more) {
      if (s.ib > 0) cont = s.ie == s.k.kt ? 2 : 1;
      else if (s.ie < s.k.kt) begun = make_int4(1, s.tok, s.ntok, s.g);
    } else {
      s.ie = -1;
    }
    if (lane == 0) segs[n & 3] = s;
  };
  if (warp == 0) {
    walk_begin<true>(p, bars, walk);
    find(0);
    find(1);
  }
  __syncthreads();

  // ---- this warp's blocks on their way: block kb of item it is the next
  const uint32_t ring = smem_u32(smem + C::RING_OFF + warp * C::RD * C::BLOCK_BYTES);
  constexpr int CPR = D / 16;                          // 16-byte pieces of a row
  constexpr int RPL = 32 / CPR;                        // rows per load
  constexpr int LOADS = 16 / RPL;
  const int lr = lane / CPR, lc = lane % CPR;
  const long long scale_bytes = (long long)p.num_pages * (p.page_size >> 4) * p.Hkv;
  auto first_block = [&](const Seg& s) { return max((s.k.hi_all - s.ie + 1) * 8, s.k.vlo >> 4); };
  auto end_block = [&](const Seg& s) { return min((s.k.hi_all - s.ib + 1) * 8, (s.k.vhi + 15) >> 4); };
  int it = 0, kb = 0, kb_end = 0, page = 0, fetched = 0;
  bool any = false;                                    // block kb exists, its page is in `page`
  int cur = 0;                                         // the item being worked on
  auto settle = [&] {                                  // on to the next block that exists
    any = true;
    while (kb >= kb_end) {
      // (items behind the next one are not known yet)
      if (it > cur || segs[(it + 1) & 3].ie < 0) {
        any = false;
        break;
      }
      ++it;
      kb = first_block(segs[it & 3]) + warp;
      kb_end = end_block(segs[it & 3]);
    }
    if (any) page = __ldg(p.block_table + (long long)segs[it & 3].b * p.max_pages + ((kb << 4) >> p.page_shift));
  };
  auto fetch = [&] {
    const uint32_t at = ring + fetched % C::RD * C::BLOCK_BYTES;
    ++fetched;
    const Seg& s = segs[it & 3];
    const bool good = page >= 0 && page < p.num_pages;
    if (!good && lane == 0) {
      // nothing is read, and the item's rows are not written
      record_status(p.status, FA_ERR_PAGE);
      segs[it & 3].lost = 1;
    }
    const long long row = good ? (long long)page * p.page_size + ((kb << 4) & (p.page_size - 1)) : 0;
    const long long off = ((row + lr) * p.Hkv + s.g) * D + lc * 16;
    const long long step = (long long)RPL * p.Hkv * D;
    const int lo = good ? s.k.vlo - (kb << 4) : 16, hi = s.k.vhi - (kb << 4);
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int r = u * RPL + lr;
      const bool seen = r >= lo && r < hi;
      const long long from = seen ? off + u * step : 0;
      const int kc = D == 128 ? lc ^ (r & 7) : lc, vc = D == 128 ? lc ^ 2 * (r & 3) : lc ^ 2 * (r >> 1 & 1);
      copy_async16(at + r * D + kc * 16, static_cast<const uint8_t*>(p.k) + from, seen ? 16 : 0);
      copy_async16(at + C::POOL + r * D + vc * 16, static_cast<const uint8_t*>(p.v) + from, seen ? 16 : 0);
    }
    if (lane == 0) {
      const long long j = good ? (row >> 4) * p.Hkv + s.g : 0;
      const int n = good ? (int)min(4ll, scale_bytes - (j & ~3ll)) : 0;
      copy_async4(at + 2 * C::POOL, p.k_scales + (j & ~3ll), n);
      copy_async4(at + 2 * C::POOL + 4, p.v_scales + (j & ~3ll), n);
      sts32(at + 2 * C::POOL + 8, (uint32_t)(j & 3) * 8);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    kb += W;
    settle();
  };
  if (segs[0].ie >= 0) {
    kb = first_block(segs[0]) + warp;
    kb_end = end_block(segs[0]);
  }

  const int g8 = lane >> 2, c4 = lane & 3;
  constexpr int X = D == 64 ? 1 : 0;
  // the keys of a lane's columns 2 c4 and 2 c4 + 1 of eight (even columns: rows
  // 0 .. 3 of the block's half, odd ones 4 .. 7; so that eight lanes' reads of
  // keys and of values take eight different places of a line)
  const int key_even = c4, key_odd = 4 + (c4 ^ X);
  const int krow = g8 & 1 ? 4 + ((g8 >> 1) ^ X) : g8 >> 1;    // the key of column g8
  int used = 0;                                        // blocks taken from the ring
  float* red = reinterpret_cast<float*>(smem + C::RED_OFF);
  float2* mls = reinterpret_cast<float2*>(smem + C::ML_OFF);
  float2* stat = reinterpret_cast<float2*>(smem + C::STAT_OFF);

#pragma unroll 1
  for (;; ++cur) {
    const Seg& s = segs[cur & 3];
    if (s.ie < 0) break;
    if (!any) settle();
    while (any && fetched - used < C::RD) fetch();
    if (warp == 0) find(cur + 2);
    const int rows = s.ntok * p.group;
    const int f = s.k.f[0];
    // rows beyond `diag` or below `low`: keys that some row does not see
    const int diag = p.causal ? f : s.L - 1, low = f + s.ntok - 1 - p.window;
    // ------------------------------------------------- Q, as fp16 fragments
    uint32_t qf[MT][D / 16][4];
    float slope2[MT][2];
    int kend[MT][2], qup[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * m + 8 * h + g8, tok = r / p.group, head = s.g * p.group + r % p.group;
        const bool valid = r < rows;
        uint4 x[D / 32];                               // 16 elements of each 64: two pieces
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + ((long long)(s.tok + tok) * p.Hq + head) * D + 16 * c4;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          x[i] = valid ? __ldg(reinterpret_cast<const uint4*>(src + 64 * (i >> 1)) + (i & 1)) : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(w[j] << 16 & 0x7fff0000u, w[j] & 0x7fff0000u));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest element to [2^14, 2^15)
        const int up = min(14 - (max((int)(top >> 23), 1) - 127), 127);
        const float mul = pow2_cut(up);
        qup[m][h] = up;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qf[m][2 * i + (j >> 1)][h + 2 * (j & 1)] =
                pack_f16x2(__uint_as_float(w[j] << 16) * mul, __uint_as_float(w[j] & 0xFFFF0000u) * mul);
        }
        kend[m][h] = !valid ? -1 : p.causal ? f + tok : s.L - 1;
        slope2[m][h] = ALIBI && valid ? __ldg(p.alibi + head) * kLog2e : 0.f;
      }
    float mref[MT][2], l[MT][2];
    float o[MT][D / 8][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mref[m][0] = mref[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][t][i] = 0.f;
    }
    int eref = -1000, etop = -1000;                    // O's unit, the largest it had
    // ------------------------------------------------------------- blocks
    const int kb1 = end_block(s);
#pragma unroll 1
    for (int b = first_block(s) + warp; b < kb1; b += W) {
      if (fetched - used == C::RD) asm volatile("cp.async.wait_group %0;" :: "n"(C::RD - 1) : "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      const uint32_t at = ring + used % C::RD * C::BLOCK_BYTES;
      ++used;
      const uint4 hd = lds128(at + 2 * C::POOL);
      const int ek = (int)min(hd.x >> hd.z & 0xffu, (uint32_t)kScaleHigh + 127) - 127;
      const int ev = (int)min(hd.y >> hd.z & 0xffu, (uint32_t)kScaleHigh + 127) - 127;
      // S of 16 rows x 8 keys, twice
      float sc[MT][2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = 8 * t + krow;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[m][t][i] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 kw = lds128(at + r * D + (D == 128 ? ((c4 + 4 * h) ^ (r & 7)) : c4) * 16);
          const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            codes_f16(w[i], b0, b1);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(sc[m][t], qf[m][4 * h + i], b0, b1);
          }
        }
      }
      // scores in log2 units; -inf where a row does not see a key
      const int k0 = b << 4;
      const bool masked = k0 + 15 > diag || k0 < low;
      bool raise = false;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float cs = p.scale_log2 * pow2_cut(ek - qup[m][h]);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float& x = sc[m][t][2 * h + j];
              const int key = k0 + 8 * t + (j ? key_odd : key_even);
              x = ALIBI ? fmaf(x, cs, slope2[m][h] * (float)(key - kend[m][h])) : x * cs;
              if (masked && (key > kend[m][h] || (p.causal && key < kend[m][h] - p.window))) x = -INFINITY;
              raise |= x > mref[m][h] + kTau;
            }
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(fmaxf(sc[m][0][2 * h], sc[m][0][2 * h + 1]), fmaxf(sc[m][1][2 * h], sc[m][1][2 * h + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const bool up = mx > mref[m][h] + kTau;
            const float alpha = up ? ex2_approx(mref[m][h] - mx) : 1.f;
            if (up) mref[m][h] = mx;
            l[m][h] *= alpha;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
              o[m][t][2 * h] *= alpha;
              o[m][t][2 * h + 1] *= alpha;
            }
          }
      }
      if (ev > eref || ev < eref - 8) {
        // O's unit follows the values' exponent, at most 2^80 below the largest
        // so far (which O's float32 holds)
        etop = max(etop, ev);
        const int e = max(ev, etop - 80);
        const float alpha = pow2_cut(eref - e);
        eref = e;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < D / 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][t][i] *= alpha;
      }
      const float sv = pow2_cut(ev - eref + 7);
      uint32_t pf[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mb = mref[m][h] == -INFINITY ? 0.f : mref[m][h];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float p0 = ex2_approx(sc[m][t][2 * h] - mb), p1 = ex2_approx(sc[m][t][2 * h + 1] - mb);
            l[m][h] += p0 + p1;
            pf[m][2 * t + h] = pack_f16x2(p0 * sv, p1 * sv);
          }
        }
      // O of 16 rows x 8 columns, D / 8 times: column g8 of product t is element
      // g8 D / 8 + t
      {
        const uint32_t vat = at + C::POOL;
        uint32_t w[4][D / 32];                         // of the keys 2 c4, 2 c4 + 1, 8 + 2 c4, 9 + 2 c4
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * (i >> 1) + (i & 1 ? key_odd : key_even);
          if (D == 128) {
            const uint4 v = lds128(vat + r * 128 + (g8 ^ 2 * (r & 3)) * 16);
            w[i][0] = v.x;
            w[i][1] = v.y;
            w[i][D / 32 - 2] = v.z;
            w[i][D / 32 - 1] = v.w;
          } else {
            const uint2 v = lds64(vat + r * 64 + ((g8 >> 1) ^ 2 * (r >> 1 & 1)) * 16 + (g8 & 1) * 8);
            w[i][0] = v.x;
            w[i][1] = v.y;
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
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(o[m][4 * i + j], pf[m], b0[j], b1[j]);
        }
      }
      __syncwarp();
      if (any) fetch();
    }
    // ------------------------------------------------- join the warps' parts
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[m][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c4 == 0) mls[warp * C::ROWS + 16 * m + 8 * h + g8] = make_float2(mref[m][h], x);
      }
    __syncthreads();
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
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float M = -INFINITY;
        for (int w = 0; w < W; ++w) M = fmaxf(M, mls[w * C::ROWS + 16 * m + 8 * h + g8].x);
        const float a = (mref[m][h] == M ? 1.f : ex2_approx(mref[m][h] - M)) * pow2_cut(eref - 7);
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          o[m][t][2 * h] *= a;
          o[m][t][2 * h + 1] *= a;
        }
      }
    const int part = s.ib > 0 ? 1 : s.ie < s.k.kt ? 2 : 0;
    const long long prow = (long long)(2 * (int)blockIdx.x + part - 1) * p.part_rows;
    const bool f32 = part || p.o_f32;                  // a part is float32, not divided
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {                 // 64 columns at a time
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * m + 8 * h + g8;
          if (r < rows) {
            float* to = red + (warp * C::ROWS + r) * C::RED_STRIDE + 16 * c4;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int q = 0; q < 2; ++q)
                *reinterpret_cast<float4*>(to + 8 * j + 4 * q) =
                    make_float4(o[m][8 * c + 4 * q][2 * h + j], o[m][8 * c + 4 * q + 1][2 * h + j],
                                o[m][8 * c + 4 * q + 2][2 * h + j], o[m][8 * c + 4 * q + 3][2 * h + j]);
          }
        }
      __syncthreads();
      const bool lost = s.lost != 0;
      if (lost && part && threadIdx.x == 0) bars->part_lost[part - 1] = 1;
      for (int i = threadIdx.x; i < rows * 16 && !lost; i += C::NT) {
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
        const int tok = r / p.group, head = s.g * p.group + r % p.group;
        const int col = (x >> 3) * (D / 8) + 8 * c + (x & 7);
        if (part == 0) {
          const float inv = ml.y > 0.f ? 1.f / ml.y : 0.f;
          v.x *= inv;
          v.y *= inv;
          v.z *= inv;
          v.w *= inv;
        }
        const long long at = part ? (prow + r) * D + col : ((long long)(s.tok + tok) * p.Hq + head) * D + col;
        if (f32) {
          *reinterpret_cast<float4*>((part ? p.part_o : static_cast<float*>(p.o)) + at) = v;
        } else {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
        if (c == 0 && x == 0) {
          if (part)
            *reinterpret_cast<float4*>(p.part_ml + (prow + r) * 4) = make_float4(ml.x, ml.y, ml.y, 0.f);
          else
            p.lse[(long long)head * p.T + s.tok + tok] = ml.y == 0.f ? -INFINITY : (ml.x + lg2_approx(ml.y)) * kLn2;
        }
      }
      __syncthreads();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (threadIdx.x == 0) {
    p.part_meta[2 * blockIdx.x] = bars->part_lost[0] ? make_int4(0, 0, 0, 0) : make_int4(cont, 0, 0, 0);
    p.part_meta[2 * blockIdx.x + 1] = bars->part_lost[1] ? make_int4(0, 0, 0, 0) : begun;
  }
}

template <int D, int MT>
int launch_few(const PagedParams& p, int grid, cudaStream_t stream) {
  using C = Few<D, MT>;
  auto kern = p.alibi ? fwd_paged_few_kernel<D, MT, true> : fwd_paged_few_kernel<D, MT, false>;
  if (const int e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return e;
  kern<<<grid, C::NT, C::SMEM_BYTES, stream>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_fwd_paged_few(const PagedParams& p, int grid, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (p.few_rows <= 16) return p.d == 128 ? launch_few<128, 1>(p, grid, stream) : launch_few<64, 1>(p, grid, stream);
  return p.d == 128 ? launch_few<128, 2>(p, grid, stream) : launch_few<64, 2>(p, grid, stream);
}

}  // namespace fa
