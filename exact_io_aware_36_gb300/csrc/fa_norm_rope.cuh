// fa_norm_rope.cuh -- pieces of the kernels that norm, rotate and write rows of
// query, key and value heads: 8 elements of a row per lane, the angles of a
// position, the place of a new token in its sequence's pages, and how a token's
// rows are dealt out to warps.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

// 8 consecutive elements of a row as stored; as 4 float32 pairs; swapped within
// their pairs; and another lane's.
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ __forceinline__ void from(const uint4* a) { w[0] = a->x; w[1] = a->y; w[2] = a->z; w[3] = a->w; }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
  __device__ __forceinline__ uint64_t pair(int i) const {
    return f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ uint64_t swapped(int i) const {
    return f2(__uint_as_float(w[i] & 0xFFFF0000u), __uint_as_float(w[i] << 16));
  }
  __device__ __forceinline__ Vec8 from_lane(int src) const {
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], src);
    return r;
  }
  __device__ __forceinline__ void set(int i, uint64_t v) {
    float a, b;
    f2split(v, a, b);
    w[i] = pack_bf16x2(a, b);
  }
};

template <>
struct Vec8<float> {
  float w[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void from(const uint4* a) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[4 * i] = __uint_as_float(a[i].x); w[4 * i + 1] = __uint_as_float(a[i].y);
      w[4 * i + 2] = __uint_as_float(a[i].z); w[4 * i + 3] = __uint_as_float(a[i].w);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.f;
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = make_float4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ uint64_t pair(int i) const { return f2(w[2 * i], w[2 * i + 1]); }
  __device__ __forceinline__ uint64_t swapped(int i) const { return f2(w[2 * i + 1], w[2 * i]); }
  __device__ __forceinline__ Vec8 from_lane(int src) const {
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], src);
    return r;
  }
  __device__ __forceinline__ void set(int i, uint64_t v) { f2split(v, w[2 * i], w[2 * i + 1]); }
};

// Sum over the LPR lanes that share a row; every one of them gets it.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  f2split(v, a, b);
  return a + b;
}

// The angles of a lane's 8 elements at one position, as 4 pairs of (c, c) and
// (s, s), s signed so that z = y c + y' s.  Not interleaved: the lane's elements
// are all first or all second members of their pairs (rot is a multiple of
// 16), and the other members are those of lane `mate` of the row.  Lanes
// without rotation have c = 1, s = 0 and must not use y'.
struct Angles {
  uint64_t c[4], s[4];
};

// The lane whose elements are this lane's partners (itself without rotation or
// interleaved).
__device__ __forceinline__ int mate_lane(const NormRopeParams& p, int l) {
  if (8 * l >= p.rot || p.interleaved) return l;
  return 16 * l < p.rot ? l + p.rot / 16 : l - p.rot / 16;
}

// `inv`: the transposed rotation.
__device__ __forceinline__ void load_angles(const NormRopeParams& p, int pos, int l, bool inv, Angles& g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g.c[i] = f2(1.f, 1.f);
    g.s[i] = f2(0.f, 0.f);
  }
  if (8 * l >= p.rot) return;
  const int half = p.rot / 2;
  const float* cs = p.cos + (long long)pos * half;
  const float* sn = p.sin + (long long)pos * half;
  if (p.interleaved) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + 4 * l));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(sn + 4 * l));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g.c[i] = f2(c[i], c[i]);
      g.s[i] = inv ? f2(s[i], -s[i]) : f2(-s[i], s[i]);
    }
  } else {
    const bool first = 8 * l < half;
    const int i0 = first ? 8 * l : 8 * l - half;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(cs + i0));
    const float4 c1 = __ldg(reinterpret_cast<const float4*>(cs + i0) + 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(sn + i0));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(sn + i0) + 1);
    const float sg = first != inv ? -1.f : 1.f;
    g.c[0] = f2(c0.x, c0.y); g.c[1] = f2(c0.z, c0.w); g.c[2] = f2(c1.x, c1.y); g.c[3] = f2(c1.z, c1.w);
    g.s[0] = f2(sg * s0.x, sg * s0.y); g.s[1] = f2(sg * s0.z, sg * s0.w);
    g.s[2] = f2(sg * s1.x, sg * s1.y); g.s[3] = f2(sg * s1.z, sg * s1.w);
  }
}

// The partners of a lane's elements.  Warp-collective; zero where there is no
// rotation, so that an infinity there meets no 0.
template <typename T, bool INTER>
struct Partners {
  Vec8<T> v;
  __device__ __forceinline__ Partners(const NormRopeParams& p, const Vec8<T>& x, int src, bool on) {
    v = x;
    if (!INTER && p.rot) v = x.from_lane(src);
    if (!on) v.zero();
  }
  __device__ __forceinline__ uint64_t pair(int i) const { return INTER ? v.swapped(i) : v.pair(i); }
};

__device__ __forceinline__ void load_weights(const float* w, int l, uint64_t* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + 8 * l));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w + 8 * l) + 1);
  f[0] = f2(a.x, a.y); f[1] = f2(a.z, a.w); f[2] = f2(b.x, b.y); f[3] = f2(b.z, b.w);
}

__device__ __forceinline__ uint64_t swap_pair(uint64_t v) {
  float a, b;
  f2split(v, a, b);
  return f2(b, a);
}

// The sequence that token t belongs to, its position there and its row in the
// pages (page * page_size + slot).  Warp-collective and warp-uniform.  False:
// the token has none (it lies behind the last sequence), or a length or page
// is out of range, which is recorded.
__device__ __forceinline__ bool locate(const NormRopeParams& p, long long t, int lane, int* pos, long long* row) {
  int b, n, i;
  if (p.cu_seqlens) {
    // The last b with cu[b] <= t, 32 probes at a time.
    int lo = 0, len = p.B + 1;                 // the answer lies in [lo, lo + len), or nowhere
    while (len > 1) {
      const int step = (len + 31) / 32;
      const int at = lo + lane * step;
      const bool le = lane * step < len && (long long)__ldg(p.cu_seqlens + at) <= t;
      const int cnt = __popc(__ballot_sync(0xffffffffu, le));
      if (cnt == 0) break;                     // t < cu[lo]: malformed
      lo += (cnt - 1) * step;
      len = min(step, p.B + 1 - lo);
    }
    b = lo;
    const int c0 = __ldg(p.cu_seqlens + b);
    if (b == p.B) {                            // behind the last sequence: no work
      if (c0 > t && lane == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
      return false;
    }
    const int c1 = __ldg(p.cu_seqlens + b + 1);
    n = c1 - c0;
    if (c0 < 0 || c0 > t || t >= c1 || c1 > p.T || n > p.N || __ldg(p.cu_seqlens) != 0) {
      if (lane == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
      return false;
    }
    i = (int)(t - c0);
  } else {
    b = (int)(t / p.N);
    n = p.N;
    i = (int)(t - (long long)b * p.N);
  }
  const int L = __ldg(p.cache_seqlens + b);
  if (L < n || (long long)L > (long long)p.max_pages * p.page_size) {
    if (lane == 0) record_status(p.status, FA_ERR_CU_SEQLENS);
    return false;
  }
  *pos = L - n + i;
  const int page = __ldg(p.block_table + (long long)b * p.max_pages + (*pos >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_status(p.status, FA_ERR_PAGE);
    return false;
  }
  *row = ((long long)page << p.page_shift) + (*pos & (p.page_size - 1));
  return true;
}

// What one warp does: sets [sa, sb) of token t.  A token's sets are those of its
// query heads, of its key heads and, with pages, of its value heads.
struct Unit {
  long long t;
  int sa, sb;
};

__device__ __forceinline__ bool unit_at(const NormRopeParams& p, unsigned unit, Unit& u) {
  const unsigned t = unit / (unsigned)p.units_per_token;
  if (t >= (unsigned long long)p.T) return false;
  u.t = t;
  u.sa = (int)(unit - t * p.units_per_token) * p.sets_per_unit;
  u.sb = min(u.sa + p.sets_per_unit, p.sets_q + p.sets_k + p.sets_v);
  return true;
}

// This warp's sets [s0, s1) of the kind whose sets are [from, from + n), as
// heads: the lane's first, and behind the last set.
struct Heads {
  int h, sets;
};

template <int RPS>
__device__ __forceinline__ Heads heads_of(const Unit& u, int from, int n, int sub) {
  const int s0 = max(u.sa, from), s1 = min(u.sb, from + n);
  return Heads{(s0 - from) * RPS + sub, max(s1 - s0, 0)};
}

}  // namespace
}  // namespace fa
