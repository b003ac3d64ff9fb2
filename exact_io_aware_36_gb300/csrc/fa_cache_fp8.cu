// fa_cache_fp8.cu -- new tokens' keys and values quantized into the pages of a
// cache held in 8 bits, plain and with the norm and rotation of q and k.
//
// A block is 16 slots of a page, one head, of the keys or of the values: e4m3
// codes c and one power of two 2^e, x = c 2^e.  For the tokens that a call
// writes into a block
//     e = min { e >= -100 : max |x| <= 448 2^e } (at most 119),
//     c = e4m3(x 2^-e), nearest even, saturated;
// where older tokens lie before them in the block, e does not fall below the
// block's own, and where it rises the older codes become e4m3(c 2^(e_old - e)).
// A power of two costs a code no precision (e4m3 is a floating format), makes
// the rescaling of older codes exact but for the smallest, and leaves c 2^e a
// bf16 value, so that the attention reads what was written without rounding.
//
// Bound by HBM: rows are read once (2 bytes) and written once (1 byte).  One
// warp has one block: its up to 16 rows are in registers, 4 KB at d = 128 all
// on their way at once, so the maximum and the codes come from one read and no
// other warp has to be asked.  Rows of a block lie next to each other in time,
// and the warps of a CTA have the heads of one block, so they share its angles
// in L1.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fa_host_util.h"
#include "fa_internal.h"
#include "fa_norm_rope.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------ norm, rotation

// A lane's 8 elements of a row, normed and rotated: z = r (x wc + x' ws), wc and
// ws the angles times the weights, x' the pair's other member.
struct Turn {
  uint64_t wc[4], ws[4];
};

template <bool INTER>
__device__ __forceinline__ void make_turn(const Angles& ang, const float* weight, int l, int mate, Turn& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.wc[i] = ang.c[i];
    f.ws[i] = ang.s[i];
  }
  if (weight) {
    uint64_t a[4], b[4];
    load_weights(weight, l, a);
    load_weights(weight, mate, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.wc[i] = fmul2(f.wc[i], a[i]);
      f.ws[i] = fmul2(f.ws[i], INTER ? swap_pair(b[i]) : b[i]);
    }
  }
}

// Warp-collective.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rope_row(const NormRopeParams& p, const Vec8<__nv_bfloat16>& x, const Turn& f, bool norm,
                                              int src_lane, bool on, uint64_t* z) {
  float r = 1.f;
  if (norm) {
    uint64_t ss = fmul2(x.pair(0), x.pair(0));
#pragma unroll
    for (int i = 1; i < 4; ++i) ss = ffma2(x.pair(i), x.pair(i), ss);
    r = rsqrtf(row_sum<D / 8>(pair_sum(ss)) * (1.f / D) + p.eps);
  }
  const uint64_t r2 = f2(r, r);
  const Partners<__nv_bfloat16, INTER> y(p, x, src_lane, on);
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = fmul2(ffma2(x.pair(i), f.wc[i], fmul2(y.pair(i), f.ws[i])), r2);
}

// This warp's sets of its token's query heads.
template <int D, bool INTER, int AHEAD>
__device__ __forceinline__ void query_rows(const NormRopeParams& p, const Unit& u, int lane) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;                // rows per set
  const int l = lane & (LPR - 1), sub = lane / LPR;
  int pos;
  long long row;
  if (!locate(p, u.t, lane, &pos, &row)) return;
  if (p.rot && pos >= p.max_pos) {
    if (lane == 0) record_status(p.status, FA_ERR_POSITION);
    return;
  }
  Angles ang;
  load_angles(p, pos, l, false, ang);
  const bool on = 8 * l < p.rot;
  const int ml = mate_lane(p, l);
  const Heads hd = heads_of<RPS>(u, 0, p.sets_q, sub);
  Turn f;
  make_turn<INTER>(ang, p.q_weight, l, ml, f);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + u.t * p.q_stride + hd.h * D + 8 * l;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + (u.t * p.Hq + hd.h) * D + 8 * l;
  int left = p.Hq - hd.h;                      // the lane's heads: every RPS-th
  for (int k = 0; k < hd.sets; k += AHEAD) {
    Vec8<__nv_bfloat16> x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (k + i < hd.sets && left > i * RPS) x[i].load(src + i * RPS * D);
      else x[i].zero();
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (k + i >= hd.sets) break;
      uint64_t z[4];
      norm_rope_row<D, INTER>(p, x[i], f, p.q_weight != nullptr, sub * LPR + ml, on, z);
      if (left > i * RPS) {
        Vec8<__nv_bfloat16> v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v.set(j, z[j]);
        v.store(dst + i * RPS * D);
      }
    }
    src += AHEAD * RPS * D;
    dst += AHEAD * RPS * D;
    left -= AHEAD * RPS;
  }
}

// -------------------------------------------------------------------- blocks

// A block of a sequence's slots that the call writes: positions [p0 + lo,
// p0 + hi), p0 its first slot's; tokens t0 .. t0 + hi - lo - 1.
struct Block {
  int b, p0, lo, hi;
  long long t0;
};

// Block number `at` of the batch; false: there is none (numbers are dealt out
// with gaps), or its sequence is malformed, which is recorded.  With
// `report` the warp speaks for its sequence.  Warp-collective, warp-uniform.
__device__ __forceinline__ bool block_at(const QuantAppendParams& q, int at, int lane, bool report, Block& k) {
  const NormRopeParams& p = q.n;
  int j;
  if (q.per_seq) {
    k.b = at / q.per_seq;
    j = at - k.b * q.per_seq;
  } else {
    // Sequence b's blocks begin at number cu[b] / 16 + 3 b: n new tokens lie in
    // at most n / 16 + 1.875 blocks, and the next sequence begins more than
    // n / 16 + 2 numbers on.  The last b whose blocks begin at or before `at`,
    // 32 probes at a time.
    int lo = 0, len = p.B;
    while (len > 1) {
      const int step = (len + 31) / 32;
      const int i = lo + lane * step;
      const bool le = lane * step < len && (long long)__ldg(p.cu_seqlens + i) / 16 + 3ll * i <= at;
      const int cnt = __popc(__ballot_sync(0xffffffffu, le));
      if (cnt == 0) return false;              // malformed: reported by the sequence's own warp
      const int on = (cnt - 1) * step;
      lo += on;
      len = min(step, len - on);
    }
    k.b = lo;
    const long long first = (long long)__ldg(p.cu_seqlens + lo) / 16 + 3ll * lo;
    if (at < first || at - first > (1 << 30)) return false;
    j = (int)(at - first);
  }
  if (k.b >= p.B) return false;
  int c0, n;
  if (p.cu_seqlens) {
    c0 = __ldg(p.cu_seqlens + k.b);
    const int c1 = __ldg(p.cu_seqlens + k.b + 1);
    if (c0 < 0 || c1 < c0 || (long long)c1 > p.T || c1 - c0 > p.N || __ldg(p.cu_seqlens) != 0) {
      if (report && lane == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
      return false;
    }
    n = c1 - c0;
  } else {
    c0 = k.b * p.N;
    n = p.N;
  }
  if (n == 0) return false;
  const int L = __ldg(p.cache_seqlens + k.b);
  if (L < n || (long long)L > (long long)p.max_pages * p.page_size) {
    if (report && lane == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
    return false;
  }
  const int start = L - n;
  const int block = start / 16 + j;
  if (block > (L - 1) / 16) return false;
  k.p0 = 16 * block;
  k.lo = max(start - k.p0, 0);
  k.hi = min(L - k.p0, 16);
  k.t0 = (long long)c0 + (k.p0 + k.lo - start);
  return true;
}

// Two floats as e4m3 codes, a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ void e4m3x2_floats(uint32_t c, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a = f.x;
  b = f.y;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// 16 bytes from global to shared memory, asynchronously; zeros without `bytes`.
__device__ __forceinline__ void copy_async16(uint4* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One head of a block, of the keys or the values.  `mine`: TURN's 8 KB (4 at d =
// 64) of shared memory of this warp, 32 bytes per lane and load.
template <int D, bool TURN, bool INTER>
__device__ __forceinline__ void write_block(const QuantAppendParams& q, const Block& k, int lane, int h, bool values,
                                            [[maybe_unused]] uint4* mine) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;                // rows per load
  constexpr int NL = 16 / RPS;                 // loads of a block
  const NormRopeParams& p = q.n;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  const int page = __ldg(p.block_table + (long long)k.b * p.max_pages + (k.p0 >> p.page_shift));
  const long long stride = values ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(values ? p.v : p.k) + k.t0 * stride + h * D + 8 * l;
  int hi = k.hi;
  if (TURN && p.rot && k.p0 + hi > p.max_pos) {
    if (lane == 0) record_status(p.status, FA_ERR_POSITION);
    hi = max(p.max_pos - k.p0, 0);
  }
  const bool turn = TURN && !values;
  // Values: the rows are in registers.  Keys that are normed and turned: in shared
  // memory, each lane's own pieces, first as they came and then as floats; so the
  // work on a row is one loop's body and not one per row, and the kernel's registers
  // leave room for twice the warps.
  Vec8<__nv_bfloat16> x[NL];
  if (turn) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = i * RPS + sub;
      const bool in = r >= k.lo && r < hi;
      copy_async16(mine + 64 * i + lane, in ? src + (r - k.lo) * stride : src, in ? 16 : 0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = i * RPS + sub;
      if (r >= k.lo && r < hi) x[i].load(src + (r - k.lo) * stride);
      else x[i].zero();
    }
  }
  if (page < 0 || page >= p.num_pages || k.lo >= hi) {
    if (turn) copies_wait();
    if (lane == 0 && (page < 0 || page >= p.num_pages)) record_status(p.status, FA_ERR_PAGE);
    return;
  }
  const long long row = ((long long)page << p.page_shift) + (k.p0 & (p.page_size - 1));
  uint8_t* scale = (values ? q.v_scales : q.k_scales) + (row >> 4) * p.Hkv + h;
  uint8_t* dst = static_cast<uint8_t*>(values ? p.v_out : p.k_out) + (row * p.Hkv + h) * D + 8 * l;
  const int was = k.lo > 0 ? min(max((int)*scale, kScaleLow + 127), kScaleHigh + 127) - 127 : kScaleLow;

  const int first = k.lo / RPS, last = (hi - 1) / RPS;     // loads with a row that is written
  float top = 0.f;
  uint64_t none = 0;                           // becomes NaN by what is not finite
  auto take = [&](const uint64_t* z) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      f2split(z[j], a, b);
      top = fmax3(top, fabsf(a), fabsf(b));
      none = ffma2(z[j], 0, none);
    }
  };
  if (turn) {
    const bool on = 8 * l < p.rot;
    const int ml = mate_lane(p, l);
    copies_wait();
#pragma unroll 2
    for (int i = first; i <= last; ++i) {
      Vec8<__nv_bfloat16> y;
      y.from(mine + 64 * i + lane);
      Angles ang;
      load_angles(p, k.p0 + min(max(i * RPS + sub, k.lo), hi - 1), l, false, ang);
      Turn f;
      make_turn<INTER>(ang, p.k_weight, l, ml, f);
      uint64_t z[4];
      norm_rope_row<D, INTER>(p, y, f, p.k_weight != nullptr, sub * LPR + ml, on, z);
      take(z);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<ulonglong2*>(mine)[64 * i + 32 * j + lane] = make_ulonglong2(z[2 * j], z[2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint64_t z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = x[i].pair(j);
      take(z);
    }
  }
  // A value's floats are made anew each time: kept, they would take twice the registers.
  auto again = [&] {
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+r"(x[i].w[j]));
  };
  auto turned = [&](int i, uint64_t* z) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const ulonglong2 v = reinterpret_cast<const ulonglong2*>(mine)[64 * i + 32 * j + lane];
      z[2 * j] = v.x;
      z[2 * j + 1] = v.y;
    }
  };
  float na, nb;
  f2split(none, na, nb);
  const bool some = __any_sync(0xffffffffu, !(na + nb == 0.f));
  if (!turn) again();
  if (some) {                                  // the maximum of the others
    top = 0.f;
    auto take_finite = [&](const uint64_t* z) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a, b;
        f2split(z[j], a, b);
        top = fmax3(top, finite(a) ? fabsf(a) : 0.f, finite(b) ? fabsf(b) : 0.f);
      }
    };
    if (turn) {
#pragma unroll 1
      for (int i = first; i <= last; ++i) {
        uint64_t z[4];
        turned(i, z);
        take_finite(z);
      }
    } else {
#pragma unroll 1
      for (int n = 0; n < NL; ++n)
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        if (i != n) continue;
        uint64_t z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = x[i].pair(j);
        take_finite(z);
      }
    }
  }
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  // 448 = 1.75 2^8
  int e = (int)(m >> 23) - 127 - 8 + ((m & 0x7fffffu) > 0x600000u);
  e = max(min(max(e, kScaleLow), kScaleHigh), was);
  const float inv = pow2(-e);
  auto put = [&](int i, const uint64_t* z) {
    const int r = i * RPS + sub;
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      f2split(z[j], a, b);
      if (some) {                              // (e4m3 has no infinity)
        if (!finite(a)) a = NAN;
        if (!finite(b)) b = NAN;
      }
      c[j] = e4m3x2(a * inv, b * inv);
    }
    if (r >= k.lo && r < hi)
      *reinterpret_cast<uint2*>(dst + r * p.Hkv * D) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  };
  if (turn) {
#pragma unroll 2
    for (int i = first; i <= last; ++i) {
      uint64_t z[4];
      turned(i, z);
      put(i, z);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint64_t z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = x[i].pair(j);
      put(i, z);
    }
  }
  if (k.lo > 0 && e > was) {                   // the older codes under the new scale
    const float down = pow2(max(was - e, -126));
#pragma unroll 1
    for (int r = sub; r < k.lo; r += RPS) {
      uint2* at = reinterpret_cast<uint2*>(dst + r * p.Hkv * D);
      uint2 w = *at;
      uint32_t* ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a, b, c, d;
        e4m3x2_floats(ws[j] & 0xffffu, a, b);
        e4m3x2_floats(ws[j] >> 16, c, d);
        ws[j] = e4m3x2(a * down, b * down) | e4m3x2(c * down, d * down) << 16;
      }
      *at = w;
    }
  }
  if (lane == 0) *scale = (uint8_t)(e + 127);
}

// TURN: with q, norm and rotation; q.block_ctas CTAs, every q.block_every-th, have
// the blocks, the others the query heads: those wait for memory where these take
// all that it gives (8000 tokens of 32 heads on 8: one after the other 49 us,
// mixed MIX_US).
template <int D, bool TURN, bool INTER>
__global__ void __launch_bounds__(kThreads, TURN ? 3 : 4) append_fp8_kernel(const QuantAppendParams q) {
  const NormRopeParams& p = q.n;
  extern __shared__ uint4 rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned nth = TURN ? blockIdx.x / q.block_every : blockIdx.x;
  if (TURN && (nth * q.block_every != blockIdx.x || nth >= q.block_ctas)) {
    Unit u;
    if (unit_at(p, (blockIdx.x - min(nth + 1, q.block_ctas)) * kWarps + warp, u)) query_rows<D, INTER, 4>(p, u, lane);
    return;
  }
  const unsigned w = nth * kWarps + warp;
  const unsigned per = 2 * p.Hkv;              // warps of a block
  const int at = (int)(w / per), rest = (int)(w - at * per);
  if (at >= q.blocks) return;
  // One warp per sequence reports a malformed one.
  if (p.cu_seqlens && rest == 0 && at < p.B && lane == 0) {
    const int c0 = __ldg(p.cu_seqlens + at), c1 = __ldg(p.cu_seqlens + at + 1);
    bool bad = c0 < 0 || c1 < c0 || (long long)c1 > p.T || c1 - c0 > p.N || (at == 0 && c0 != 0);
    if (!bad && c1 > c0) {
      const int L = __ldg(p.cache_seqlens + at);
      bad = L < c1 - c0 || (long long)L > (long long)p.max_pages * p.page_size;
    }
    if (bad) record_status(p.status, FA_ERR_CU_SEQLENS);
  }
  Block k;
  if (!block_at(q, at, lane, rest == 0, k)) return;
  write_block<D, TURN, INTER>(q, k, lane, rest % p.Hkv, rest >= p.Hkv, rows + warp * (4 * D));
}

template <int D>
int launch_d(QuantAppendParams q, bool turn, cudaStream_t stream) {
  NormRopeParams& p = q.n;
  // numbers for the blocks: as many for every sequence, or by its place in
  // cu_seqlens, whichever takes fewer
  const long long per_seq = (p.N + 14) / 16 + 1;
  const long long even = per_seq * p.B, by_place = p.T / 16 + 3ll * p.B + 1;
  q.per_seq = !p.cu_seqlens || even <= by_place ? (int)per_seq : 0;
  const long long blocks = q.per_seq ? even : by_place;
  const long long ctas = (blocks * 2 * p.Hkv + kWarps - 1) / kWarps;
  long long units = 0;
  if (turn) {
    constexpr int RPS = 32 / (D / 8);
    p.sets_q = (p.Hq + RPS - 1) / RPS;
    p.sets_k = p.sets_v = 0;
    p.sets_per_unit = (int)std::min<long long>(p.sets_q, std::max(2ll, p.T * p.sets_q / kNormRopeWarps));
    p.units_per_token = (p.sets_q + p.sets_per_unit - 1) / p.sets_per_unit;
    units = p.T * p.units_per_token;
  }
  const long long grid = ctas + (units + kWarps - 1) / kWarps;
  if (grid >= (1ll << 31) / kWarps || blocks >= (1ll << 31) / (2 * p.Hkv)) return (int)cudaErrorInvalidConfiguration;
  q.blocks = (int)blocks;
  q.block_ctas = (unsigned)ctas;
  q.block_every = (unsigned)(grid / ctas);
  auto kern = !turn ? append_fp8_kernel<D, false, false>
                    : p.interleaved ? append_fp8_kernel<D, true, true> : append_fp8_kernel<D, true, false>;
  const int smem = turn ? kWarps * 64 * D : 0;
  if (turn)
    if (const int e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return e;
  kern<<<(unsigned)grid, kThreads, smem, stream>>>(q);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_append_fp8(const QuantAppendParams& q, bool turn, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return q.n.d == 128 ? launch_d<128>(q, turn, stream) : launch_d<64>(q, turn, stream);
}

}  // namespace fa
