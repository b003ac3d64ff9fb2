// fa_norm_rope.cu -- RMS norm of every query and key head and the rotation by
// position in one pass, its gradient, and the serving form that writes the new
// tokens' k and v into the pages of a cache.
//
// Row x (d elements of one head of one token), weight w, angle table at the
// token's position:
//     r = (mean(x^2) + eps)^-1/2,   y = x r w,   z = R y,
// R rotating rot / 2 pairs of elements: (i, i + rot / 2), or (2 i, 2 i + 1)
// when interleaved; elements from rot on pass unrotated.  Gradient of z -> x, w:
//     dy = R^T dz,   dw = sum over rows of dy x r,
//     dx = r (dy w - xh mean(dy w xh)),   xh = x r.
// All arithmetic is float32; each output is rounded once.  r is recomputed in
// the backward: x has to be read anyway, so saving r would only add bytes.
//
// Bound by HBM: a row is read and written once (twice read in the backward)
// against about 10 operations per element.  A lane holds 8 consecutive
// elements (16 bytes of bf16), so d / 8 lanes share a row and a warp holds
// 32 * 8 / d rows at a time, two such sets per unit of work: the loads of both
// are in flight before the first is used.  A unit's rows belong to one token,
// so its angles are loaded once for all of them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fa_host_util.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSets = 2;                      // row sets of one unit of work

// 8 consecutive elements of a row, as stored and as float32.
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Sum over the LPR lanes that share a row; every one of them gets it.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The angles of a lane's 8 elements at one position.  Not interleaved: the
// lane's elements 8 l .. 8 l + 7 are all first or all second members of their
// pairs (rot is a multiple of 16), the other members sit 8 elements per lane
// at lane `mate`, and c / s hold 8 angles (s negated for first members, so
// z = y c + y' s for both).  Interleaved: 4 pairs within the lane.
struct Angles {
  float c[8], s[8];
  int mate;
  bool on;                                    // the lane's elements are rotated
};

// INV: the transposed rotation.
template <int LPR>
__device__ __forceinline__ void load_angles(const NormRopeParams& p, int pos, int l, bool inv, Angles& g) {
  g.on = 8 * l < p.rot;
  g.mate = l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g.c[i] = 1.f;
    g.s[i] = 0.f;
  }
  if (!g.on) return;
  const int half = p.rot / 2;
  const float* cs = p.cos + (long long)pos * half;
  const float* sn = p.sin + (long long)pos * half;
  if (p.interleaved) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + 4 * l));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(sn + 4 * l));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g.c[2 * i] = g.c[2 * i + 1] = c[i];
      g.s[2 * i] = inv ? s[i] : -s[i];
      g.s[2 * i + 1] = inv ? -s[i] : s[i];
    }
  } else {
    const bool first = 8 * l < half;
    const int i0 = first ? 8 * l : 8 * l - half;
    g.mate = first ? l + half / 8 : l - half / 8;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(cs + i0));
    const float4 c1 = __ldg(reinterpret_cast<const float4*>(cs + i0) + 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(sn + i0));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(sn + i0) + 1);
    const float sg = first != inv ? -1.f : 1.f;
    g.c[0] = c0.x; g.c[1] = c0.y; g.c[2] = c0.z; g.c[3] = c0.w;
    g.c[4] = c1.x; g.c[5] = c1.y; g.c[6] = c1.z; g.c[7] = c1.w;
    g.s[0] = sg * s0.x; g.s[1] = sg * s0.y; g.s[2] = sg * s0.z; g.s[3] = sg * s0.w;
    g.s[4] = sg * s1.x; g.s[5] = sg * s1.y; g.s[6] = sg * s1.z; g.s[7] = sg * s1.w;
  }
}

// f <- rotated f.  Warp-collective (the pair's other member may sit in another
// lane of the row); lanes without rotation keep f.
template <int LPR>
__device__ __forceinline__ void rotate(const NormRopeParams& p, const Angles& g, int lane, float* f) {
  if (p.rot == 0) return;
  float o[8];
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = f[i ^ 1];
  } else {
    const int src = (lane & ~(LPR - 1)) + g.mate;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, f[i], src);
  }
  if (g.on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf(f[i], g.c[i], o[i] * g.s[i]);
  }
}

__device__ __forceinline__ void load_weights(const float* w, int l, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + 8 * l));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w + 8 * l) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
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

// Rows of a token, in this order: Hq query heads, Hkv key heads and, with
// PAGES, Hkv value heads (copied).  One warp per unit: kSets sets of
// 32 / LPR rows of one token.
template <int D, typename T, bool PAGES>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;                // rows per set
  const int lane = threadIdx.x & 31;
  const int l = lane & (LPR - 1);
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int per_token = p.units_per_token;
  const long long t = unit / per_token;
  if (t >= p.T) return;
  const int h0 = (int)(unit - t * per_token) * (kSets * RPS);
  const int nrow = p.Hq + (PAGES ? 2 : 1) * p.Hkv;

  Vec8<T> x[kSets];
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int h = h0 + s * RPS + lane / LPR;
    const T* src = h < p.Hq ? static_cast<const T*>(p.q) + t * p.q_stride + (long long)h * D
                 : h < p.Hq + p.Hkv
                     ? static_cast<const T*>(p.k) + t * p.k_stride + (long long)(h - p.Hq) * D
                     : static_cast<const T*>(p.v) + t * p.v_stride + (long long)(h - p.Hq - p.Hkv) * D;
    if (h < nrow) x[s].load(src + 8 * l);
    else x[s].zero();
  }
  int pos = 0;
  long long page_row = 0;
  if constexpr (PAGES) {
    if (!locate(p, t, lane, &pos, &page_row)) return;
  } else if (p.rot) {
    pos = __ldg(p.positions + t);
  }
  if (p.rot && (pos < 0 || pos >= p.max_pos)) {
    if (lane == 0) record_status(p.status, FA_ERR_POSITION);
    return;
  }
  Angles ang;
  load_angles<LPR>(p, pos, l, false, ang);
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int h = h0 + s * RPS + lane / LPR;
    const bool is_q = h < p.Hq, is_v = PAGES && h >= p.Hq + p.Hkv;
    float f[8];
    x[s].get(f);
    if (p.q_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
      float w[8];
      load_weights(is_q ? p.q_weight : p.k_weight, l, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
    }
    rotate<LPR>(p, ang, lane, f);
    if (!is_v) x[s].set(f);                    // value rows pass as they are
    if (h < nrow) {
      T* dst;
      if (is_q) dst = static_cast<T*>(p.q_out) + (t * p.Hq + h) * D;
      else if constexpr (PAGES)
        dst = is_v ? static_cast<T*>(p.v_out) + (page_row * p.Hkv + (h - p.Hq - p.Hkv)) * D
                   : static_cast<T*>(p.k_out) + (page_row * p.Hkv + (h - p.Hq)) * D;
      else dst = static_cast<T*>(p.k_out) + (t * p.Hkv + (h - p.Hq)) * D;
      x[s].store(dst + 8 * l);
    }
  }
}

// Gradient.  A warp walks units with a fixed stride and keeps the weights'
// sums of its columns in registers; a block writes its sum to the workspace
// (float32 [blocks][2][D]) and norm_rope_dw_kernel adds the blocks up, both in
// a fixed order, so the result is the same from run to run.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;
  __shared__ float red[kWarps][2][D];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int l = lane & (LPR - 1);
  const int per_token = p.units_per_token;
  const long long units = p.T * per_token;
  const int nrow = p.Hq + p.Hkv;
  float dwq[8], dwk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;

  for (long long unit = (long long)blockIdx.x * kWarps + warp; unit < units; unit += (long long)gridDim.x * kWarps) {
    const long long t = unit / per_token;
    const int h0 = (int)(unit - t * per_token) * (kSets * RPS);
    Vec8<T> x[kSets], z[kSets];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int h = h0 + s * RPS + lane / LPR;
      const bool is_q = h < p.Hq;
      const int hk = h - p.Hq;
      if (h < nrow) {
        x[s].load((is_q ? static_cast<const T*>(p.q) + t * p.q_stride + (long long)h * D
                        : static_cast<const T*>(p.k) + t * p.k_stride + (long long)hk * D) + 8 * l);
        z[s].load((is_q ? static_cast<const T*>(p.dq_out) + (t * p.Hq + h) * D
                        : static_cast<const T*>(p.dk_out) + (t * p.Hkv + hk) * D) + 8 * l);
      } else {
        x[s].zero();
        z[s].zero();
      }
    }
    const int pos = p.rot ? __ldg(p.positions + t) : 0;
    if (p.rot && (pos < 0 || pos >= p.max_pos)) {
      if (lane == 0) record_status(p.status, FA_ERR_POSITION);
      continue;
    }
    Angles ang;
    load_angles<LPR>(p, pos, l, true, ang);
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int h = h0 + s * RPS + lane / LPR;
      const bool is_q = h < p.Hq;
      float f[8], dy[8];
      x[s].get(f);
      z[s].get(dy);
      rotate<LPR>(p, ang, lane, dy);
      if (p.q_weight) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        float w[8];
        load_weights(is_q ? p.q_weight : p.k_weight, l, w);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] *= r;                           // xh
          const float dw = h < nrow ? dy[i] * f[i] : 0.f;
          dwq[i] += is_q ? dw : 0.f;
          dwk[i] += is_q ? 0.f : dw;
          dy[i] *= w[i];
          dot = fmaf(dy[i], f[i], dot);
        }
        const float m = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[i] = r * fmaf(-f[i], m, dy[i]);
      }
      if (h < nrow) {
        x[s].set(dy);
        T* dst = is_q ? static_cast<T*>(p.dq) + t * p.dq_stride + (long long)h * D
                      : static_cast<T*>(p.dk) + t * p.dk_stride + (long long)(h - p.Hq) * D;
        x[s].store(dst + 8 * l);
      }
    }
  }
  if (p.q_weight) {
    // the warp's row groups, then the block's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
        dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
      }
      if (lane < LPR) {
        red[warp][0][8 * l + i] = dwq[i];
        red[warp][1][8 * l + i] = dwk[i];
      }
    }
    __syncthreads();
    if (threadIdx.x < 2 * D) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += (&red[w][0][0])[threadIdx.x];
      p.dw_part[(long long)blockIdx.x * 2 * D + threadIdx.x] = s;
    }
  }
  grid_launch_dependents();
}

// Sum of the blocks' parts: one block per 32 of the 2 D columns, 8 strips of
// blocks per column, added in a fixed order.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* part, int nblocks, int D, float* dwq, float* dwk) {
  __shared__ float red[8][32];
  grid_dependency_wait();
  const int c = threadIdx.x & 31;
  const int strip = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.f;
#pragma unroll 4
  for (int b = strip; b < nblocks; b += 8) s += part[(long long)b * 2 * D + col];
  red[strip][c] = s;
  __syncthreads();
  if (strip == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][c];
    if (col < D) dwq[col] = s;
    else dwk[col - D] = s;
  }
}

template <int D, typename T, bool PAGES>
int launch_fwd(NormRopeParams p, cudaStream_t stream) {
  constexpr int rows = kSets * (32 / (D / 8));
  p.units_per_token = (p.Hq + (PAGES ? 2 : 1) * p.Hkv + rows - 1) / rows;
  const long long grid = (p.T * p.units_per_token + kWarps - 1) / kWarps;
  norm_rope_kernel<D, T, PAGES><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  return (int)cudaGetLastError();
}

template <int D, typename T>
int launch_bwd(NormRopeParams p, cudaStream_t stream) {
  constexpr int rows = kSets * (32 / (D / 8));
  p.units_per_token = (p.Hq + p.Hkv + rows - 1) / rows;
  const int grid = (int)std::min<long long>((p.T * p.units_per_token + kWarps - 1) / kWarps, kNormRopeBwdBlocks);
  norm_rope_bwd_kernel<D, T><<<grid, kThreads, 0, stream>>>(p);
  if (const cudaError_t e = cudaGetLastError()) return (int)e;
  if (!p.q_weight) return 0;
  return launch_dependent(norm_rope_dw_kernel, dim3(2 * D / 32), dim3(256), 0, stream,
                          (const float*)p.dw_part, grid, D, p.dq_weight, p.dk_weight);
}

}  // namespace

int launch_norm_rope(const NormRopeParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (p.f32) return p.d == 128 ? launch_fwd<128, float, false>(p, stream) : launch_fwd<64, float, false>(p, stream);
  return p.d == 128 ? launch_fwd<128, __nv_bfloat16, false>(p, stream) : launch_fwd<64, __nv_bfloat16, false>(p, stream);
}

int launch_norm_rope_pages(const NormRopeParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return p.d == 128 ? launch_fwd<128, __nv_bfloat16, true>(p, stream) : launch_fwd<64, __nv_bfloat16, true>(p, stream);
}

int launch_norm_rope_bwd(const NormRopeParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (p.f32) return p.d == 128 ? launch_bwd<128, float>(p, stream) : launch_bwd<64, float>(p, stream);
  return p.d == 128 ? launch_bwd<128, __nv_bfloat16>(p, stream) : launch_bwd<64, __nv_bfloat16>(p, stream);
}

}  // namespace fa
