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
// other warp has to be asked.  The registers are kept low (values' floats are made
// twice, keys to be turned wait in shared memory), because the chain lengths -> page ->
// rows asks for many warps: 8 prompts of 4096 tokens, 8 heads of 128, 33.2 us, 6.07
// TB/s, 91 % of the copy rate (51.4 us with 16 warps per SM, 33.2 with 32); one token
// each of 64 sequences with norm and rotation 3.8 us; 8000 tokens of 32 heads on 8 with
// them 42 us, 4.2 TB/s: there the warps that norm and turn keys wait for their angles
// and shuffles, 24 us, and the query heads' 26 us come after them.
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

// The same of many rows, of which each has its own angles: the weights of a lane's
// elements, and of their partners with the sign of the sine.
struct Weights {
  uint64_t a[4], b[4];
};

template <bool INTER>
__device__ __forceinline__ void make_weights(const NormRopeParams& p, const float* weight, int l, int mate, Weights& w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w.a[i] = w.b[i] = f2(1.f, 1.f);
  if (weight) {
    load_weights(weight, l, w.a);
    load_weights(weight, mate, w.b);
  }
  const float sg = 8 * l < p.rot / 2 ? -1.f : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) w.b[i] = INTER ? fmul2(swap_pair(w.b[i]), f2(-1.f, 1.f)) : fmul2(w.b[i], f2(sg, sg));
}

template <bool INTER>
__device__ __forceinline__ void turn_of(const NormRopeParams& p, int pos, int l, const Weights& w, Turn& f) {
  if (8 * l >= p.rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.wc[i] = w.a[i];
      f.ws[i] = 0;
    }
    return;
  }
  const int half = p.rot / 2, at = INTER ? 4 * l : 8 * l < half ? 8 * l : 8 * l - half;
  const float4* cs = reinterpret_cast<const float4*>(p.cos + (long long)pos * half + at);
  const float4* sn = reinterpret_cast<const float4*>(p.sin + (long long)pos * half + at);
  const float4 c = __ldg(cs), s = __ldg(sn);
  if (INTER) {
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.wc[i] = fmul2(f2(cv[i], cv[i]), w.a[i]);
      f.ws[i] = fmul2(f2(sv[i], sv[i]), w.b[i]);
    }
  } else {
    const float4 d = __ldg(cs + 1), t = __ldg(sn + 1);
    f.wc[0] = fmul2(f2(c.x, c.y), w.a[0]);
    f.wc[1] = fmul2(f2(c.z, c.w), w.a[1]);
    f.wc[2] = fmul2(f2(d.x, d.y), w.a[2]);
    f.wc[3] = fmul2(f2(d.z, d.w), w.a[3]);
    f.ws[0] = fmul2(f2(s.x, s.y), w.b[0]);
    f.ws[1] = fmul2(f2(s.z, s.w), w.b[1]);
    f.ws[2] = fmul2(f2(t.x, t.y), w.b[2]);
    f.ws[3] = fmul2(f2(t.z, t.w), w.b[3]);
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
    const float v = row_sum<D / 8>(pair_sum(ss)) * (1.f / D) + p.eps;
    r = rsqrtf(v);
    // one step of Newton's method: a code next to its rounding's border shows the
    // last bit of r
    const float off = fmaf(-v * r, r, 1.f);
    if (fabsf(off) < 1.f) r = fmaf(0.5f * r, off, r);
  }
  const uint64_t r2 = f2(r, r);
  const Partners<__nv_bfloat16, INTER> y(p, x, src_lane, on);
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = fmul2(ffma2(x.pair(i), f.wc[i], fmul2(y.pair(i), f.ws[i])), r2);
}

// This warp's sets of its token's query heads, AHEAD of them at a time while the
// next are on their way; the first before the token's place is known.
template <int D, bool INTER, int AHEAD>
__device__ __forceinline__ void query_rows(const NormRopeParams& p, const Unit& u, int lane) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;                // rows per set
  const int l = lane & (LPR - 1), sub = lane / LPR;
  const Heads hd = heads_of<RPS>(u, 0, p.sets_q, sub);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + u.t * p.q_stride + hd.h * D + 8 * l;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + (u.t * p.Hq + hd.h) * D + 8 * l;
  const int left = p.Hq - hd.h;                // the lane's heads: every RPS-th
  Vec8<__nv_bfloat16> x[AHEAD], y[AHEAD];
  auto fetch = [&](int k, Vec8<__nv_bfloat16>* v) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (k + i < hd.sets && left > (k + i) * RPS) v[i].load(src + (k + i) * RPS * D);
      else v[i].zero();
    }
  };
  fetch(0, x);
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
  Turn f;
  make_turn<INTER>(ang, p.q_weight, l, ml, f);
  for (int k = 0; k < hd.sets; k += AHEAD) {
    fetch(k + AHEAD, y);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (k + i >= hd.sets) break;
      uint64_t z[4];
      norm_rope_row<D, INTER>(p, x[i], f, p.q_weight != nullptr, sub * LPR + ml, on, z);
      if (left > (k + i) * RPS) {
        Vec8<__nv_bfloat16> v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v.set(j, z[j]);
        v.store(dst + (k + i) * RPS * D);
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) x[i] = y[i];
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
  // (all loads before the first of their checks)
  const int L = __ldg(p.cache_seqlens + k.b);
  int c0 = k.b * p.N, n = p.N;
  if (p.cu_seqlens) {
    const int begin = __ldg(p.cu_seqlens), c1 = __ldg(p.cu_seqlens + k.b + 1);
    c0 = __ldg(p.cu_seqlens + k.b);
    if (begin != 0 || c0 < 0 || c1 < c0 || (long long)c1 > p.T || c1 - c0 > p.N) {
      if (report && lane == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
      return false;
    }
    n = c1 - c0;
  }
  if (n == 0) return false;
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

// One head of a block, of the keys or the values.  TURN: keys that are normed and
// turned; `mine`: their 8 KB (4 at d = 64) of shared memory of this warp, 32 bytes
// per lane and load.
template <int D, bool TURN, bool INTER, bool ROPE>
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
  if (ROPE && p.rot && k.p0 + hi > p.max_pos) {
    if (lane == 0) record_status(p.status, FA_ERR_POSITION);
    hi = max(p.max_pos - k.p0, 0);
  }
  // The rows are in registers; those to be normed and turned in shared memory, each lane's own pieces, first as they came and then as floats; so the
  // work on a row is one loop's body and not one per row, and the kernel's registers
  // leave room for twice the warps.
  Vec8<__nv_bfloat16> x[NL];
  if constexpr (TURN) {
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
    if (TURN) copies_wait();
    if (lane == 0 && (page < 0 || page >= p.num_pages)) record_status(p.status, FA_ERR_PAGE);
    return;
  }
  const long long row = ((long long)page << p.page_shift) + (k.p0 & (p.page_size - 1));
  uint8_t* scale = (values ? q.v_scales : q.k_scales) + (row >> 4) * p.Hkv + h;
  uint8_t* dst = static_cast<uint8_t*>(values ? p.v_out : p.k_out) + (row * p.Hkv + h) * D + 8 * l;
  // (a block's own scale, of another writer, may lie below the least that is written)
  const int was = k.lo > 0 ? min((int)*scale, kScaleHigh + 127) - 127 : kScaleLow;

  const int first = k.lo / RPS, last = (hi - 1) / RPS;     // loads with a row that is written
  float top = 0.f;
  bool some;                                   // something is not finite
  if constexpr (TURN) {
    const bool on = 8 * l < p.rot;
    const int ml = mate_lane(p, l);
    Weights w;
    make_weights<INTER>(p, p.k_weight, l, ml, w);
    copies_wait();
    uint64_t none = 0;                         // becomes NaN by what is not finite
#pragma unroll 2
    for (int i = first; i <= last; ++i) {
      Vec8<__nv_bfloat16> y;
      y.from(mine + 64 * i + lane);
      Turn f;
      turn_of<INTER>(p, k.p0 + min(max(i * RPS + sub, k.lo), hi - 1), l, w, f);
      uint64_t z[4];
      norm_rope_row<D, INTER>(p, y, f, p.k_weight != nullptr, sub * LPR + ml, on, z);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a, b;
        f2split(z[j], a, b);
        top = fmax3(top, fabsf(a), fabsf(b));
        none = ffma2(z[j], 0, none);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<ulonglong2*>(mine)[64 * i + 32 * j + lane] = make_ulonglong2(z[2 * j], z[2 * j + 1]);
    }
    float na, nb;
    f2split(none, na, nb);
    some = !(na + nb == 0.f);
  } else {
    // absolute values of bf16 are in the order of their bits
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) most = __vmaxu2(most, x[i].w[j] & 0x7fff7fffu);
    most = max(most >> 16, most & 0xffffu);
    top = __uint_as_float(most << 16);
    some = most >= 0x7f80u;
  }
  auto turned = [&](int i, uint64_t* z) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const ulonglong2 v = reinterpret_cast<const ulonglong2*>(mine)[64 * i + 32 * j + lane];
      z[2 * j] = v.x;
      z[2 * j + 1] = v.y;
    }
  };
  if (__any_sync(0xffffffffu, some)) {         // the maximum of the others; these become NaN (e4m3 has no infinity)
    top = 0.f;
    if constexpr (TURN) {
#pragma unroll 1
      for (int n = 64 * first; n < 64 * (last + 1); n += 32) {
        float4 z = reinterpret_cast<const float4*>(mine)[n + lane];
        float* v = &z.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (finite(v[j])) top = fmaxf(top, fabsf(v[j]));
          else v[j] = NAN;
        }
        reinterpret_cast<float4*>(mine)[n + lane] = z;
      }
    } else {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < NL; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a = x[i].w[j] & 0x7fff7fffu;
          const uint32_t odd = __vcmpgeu2(a, 0x7f807f80u);
          most = __vmaxu2(most, a & ~odd);
          x[i].w[j] |= odd & 0x7fff7fffu;
        }
      top = __uint_as_float(max(most >> 16, most & 0xffffu) << 16);
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
      f2split(fmul2(z[j], f2(inv, inv)), a, b);
      c[j] = e4m3x2(a, b);
    }
    if (r >= k.lo && r < hi)
      *reinterpret_cast<uint2*>(dst + r * p.Hkv * D) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  };
  if constexpr (TURN) {
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

// TURN: with q, norm and rotation; the first q.block_ctas CTAs have the blocks,
// the others the query heads.
template <int D, bool TURN, bool INTER>
__global__ void __launch_bounds__(kThreads, TURN ? 3 : 4) append_fp8_kernel(const QuantAppendParams q) {
  const NormRopeParams& p = q.n;
  extern __shared__ uint4 rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (TURN && blockIdx.x >= q.block_ctas) {
    Unit u;
    if (unit_at(p, (blockIdx.x - q.block_ctas) * kWarps + warp, u)) query_rows<D, INTER, 4>(p, u, lane);
    return;
  }
  const unsigned w = blockIdx.x * kWarps + warp;
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
  const int h = rest < p.Hkv ? rest : rest - p.Hkv;
  if (TURN && rest < p.Hkv) write_block<D, TURN, INTER, TURN>(q, k, lane, h, false, rows + warp * (4 * D));
  else write_block<D, false, false, TURN>(q, k, lane, h, rest >= p.Hkv, nullptr);
}

template <int D>
int launch_d(QuantAppendParams q, bool turn, cudaStream_t stream) {
  NormRopeParams& p = q.n;
  // numbers for the blocks: as many for every sequence, or by its place in
  // cu_seqlens, whichever takes fewer
  const long long per_seq = ((long long)p.N + 14) / 16 + 1;
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
