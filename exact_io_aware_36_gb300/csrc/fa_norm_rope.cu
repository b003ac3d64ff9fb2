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
// Bound by HBM: a row is read and written once (two are read in the backward).
// A lane holds 8 consecutive elements (16 bytes of bf16), so d / 8 lanes share
// a row and a warp holds a set of 32 * 8 / d rows of one kind (query, key or
// value heads) of one token.  A warp takes several sets of its token, a few
// loaded at a time, so that a token's angles, multiplied by the weights, are
// made once:
//     z = r (x (w c) + x' (w' s)),   x', w': the pair's other member.
// With these packed in float32 pairs a set costs some 120 instructions (170 in
// the backward), which leaves issue slots idle at HBM's rate; the first form,
// at twice as many, was bound by them.  One GB300, 16384 tokens of 32 + 8 heads
// of 128 in bf16: 58.3 us, 5.79 TB/s, 85 % of the measured copy rate; backward
// 87.6 us, 5.77 TB/s, 85 %.  The order of the rotation's pairs is a template
// argument: chosen at run time the two cost 58.6 and 91.5 us.
#include <cuda.h>
#include <cuda_bf16.h>
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
// Sets that the forward loads before it uses the first, and the blocks per SM
// that leaves room for (registers).  Both cover HBM's latency: 16384 tokens of
// 32 + 8 heads of 128 took 67 us with two bf16 sets ahead, 59 with four, 61 with
// six and three blocks; fetching a warp's first rows ahead of its angles cost
// registers or time (67 by loads, 60 by a prefetch into L2).  The bf16 forms do
// not quite fit their 64 registers: they spill 84 bytes (96 into pages, 24-32
// with neighbouring pairs).  Float32 sets are twice as large (four: 7.9 us for
// 3001 tokens of 16 heads of 64, two: 6.4, without spills).
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;
template <typename T>
constexpr int kBlocksPerSm = sizeof(T) == 2 ? 4 : 3;

// Rows that pass as they are: this warp's sets of [from, from + n), H heads at
// src and dst, AHEAD sets loaded before the first is stored.
template <int D, int AHEAD>
__device__ __forceinline__ void copy_rows(const Unit& u, int lane, const void* src_, void* dst_, int H, int from, int n) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;
  const Heads hd = heads_of<RPS>(u, from, n, lane / LPR);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(src_) + hd.h * D + 8 * (lane & (LPR - 1));
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(dst_) + hd.h * D + 8 * (lane & (LPR - 1));
  int left = H - hd.h;                         // the lane's heads: every RPS-th
  for (int k = 0; k < hd.sets; k += AHEAD) {
    Vec8<__nv_bfloat16> x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (k + i < hd.sets && left > i * RPS) x[i].load(src + i * RPS * D);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (k + i < hd.sets && left > i * RPS) x[i].store(dst + i * RPS * D);
    src += AHEAD * RPS * D;
    dst += AHEAD * RPS * D;
    left -= AHEAD * RPS;
  }
}

// New tokens' keys and values into the pages, bit for bit (the arithmetic of
// norm_rope_kernel with a weight of 1 and no angle would lose the sign of zero
// and a NaN's payload).  Bound by HBM: 8 x 4096 tokens of 8 heads of 128 take
// 40.9 us, 6.56 TB/s, 97 % of the measured copy rate.
template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const NormRopeParams p) {
  const int lane = threadIdx.x & 31;
  Unit u;
  if (!unit_at(p, blockIdx.x * kWarps + (threadIdx.x >> 5), u)) return;
  int pos;
  long long row;
  if (!locate(p, u.t, lane, &pos, &row)) return;
  auto rows = [&](const void* x, long long stride, void* pool, int from, int n) {
    copy_rows<D, 4>(u, lane, static_cast<const __nv_bfloat16*>(x) + u.t * stride,
                    static_cast<__nv_bfloat16*>(pool) + row * p.Hkv * D, p.Hkv, from, n);
  };
  rows(p.k, p.k_stride, p.k_out, 0, p.sets_k);
  rows(p.v, p.v_stride, p.v_out, p.sets_k, p.sets_v);
}

// INTER: the pairs of the rotation are neighbours (p.interleaved).
template <int D, typename T, bool PAGES, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<T>) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;                // rows per set
  const int lane = threadIdx.x & 31;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  Unit u;
  if (!unit_at(p, blockIdx.x * kWarps + (threadIdx.x >> 5), u)) return;
  const long long t = u.t;
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
  load_angles(p, pos, l, false, ang);
  const bool on = 8 * l < p.rot;
  const int ml = mate_lane(p, l), src_lane = sub * LPR + ml;

  // H heads at src and dst (this token's), sets [from, from + n)
  auto rows = [&](const T* src, T* dst, int H, int from, int n, const float* weight) {
    const Heads hd = heads_of<RPS>(u, from, n, sub);
    if (hd.sets == 0) return;
    uint64_t wc[4], ws[4];                     // angles times weights
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wc[i] = ang.c[i];
      ws[i] = ang.s[i];
    }
    if (weight) {
      uint64_t a[4], b[4];
      load_weights(weight, l, a);
      load_weights(weight, ml, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wc[i] = fmul2(wc[i], a[i]);
        ws[i] = fmul2(ws[i], INTER ? swap_pair(b[i]) : b[i]);
      }
    }
    src += hd.h * D + 8 * l;
    dst += hd.h * D + 8 * l;
    const int left0 = H - hd.h;                // the lane's heads: every RPS-th
    auto one = [&](const Vec8<T>& x, T* at, bool live) {
      float r = 1.f;
      if (weight) {
        uint64_t ss = fmul2(x.pair(0), x.pair(0));
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = ffma2(x.pair(i), x.pair(i), ss);
        r = rsqrtf(row_sum<LPR>(pair_sum(ss)) * (1.f / D) + p.eps);
      }
      const uint64_t r2 = f2(r, r);
      const Partners<T, INTER> y(p, x, src_lane, on);
      Vec8<T> z;
#pragma unroll
      for (int i = 0; i < 4; ++i) z.set(i, fmul2(ffma2(x.pair(i), wc[i], fmul2(y.pair(i), ws[i])), r2));
      if (live) z.store(at);
    };
    int left = left0;
    for (int k = 0; k < hd.sets; k += kAhead<T>) {
      Vec8<T> x[kAhead<T>];
#pragma unroll
      for (int i = 0; i < kAhead<T>; ++i) {
        if (k + i < hd.sets && left > i * RPS) x[i].load(src + i * RPS * D);
        else x[i].zero();
      }
#pragma unroll
      for (int i = 0; i < kAhead<T>; ++i) {
        if (k + i >= hd.sets) break;
        one(x[i], dst + i * RPS * D, left > i * RPS);
      }
      src += kAhead<T> * RPS * D;
      dst += kAhead<T> * RPS * D;
      left -= kAhead<T> * RPS;
    }
  };
  const bool norm = p.q_weight != nullptr;
  rows(static_cast<const T*>(p.q) + t * p.q_stride, static_cast<T*>(p.q_out) + t * p.Hq * D, p.Hq, 0, p.sets_q,
       norm ? p.q_weight : nullptr);
  rows(static_cast<const T*>(p.k) + t * p.k_stride, static_cast<T*>(p.k_out) + (PAGES ? page_row : t) * p.Hkv * D, p.Hkv,
       p.sets_q, p.sets_k, norm ? p.k_weight : nullptr);
  if constexpr (PAGES)
    copy_rows<D, 2>(u, lane, static_cast<const T*>(p.v) + t * p.v_stride, static_cast<T*>(p.v_out) + page_row * p.Hkv * D,
                    p.Hkv, p.sets_q + p.sets_k, p.sets_v);
}

// 16 bytes from global to shared memory, asynchronously; zeros where `bytes`
// is 0 (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Sets of x and of dz that a warp of the gradient has on their way (bf16, 16384
// tokens: four 87.6 us, six 87.6, eight 88.5).
template <typename T>
constexpr int kDepth = sizeof(T) == 2 ? 6 : 3;

template <typename T>
constexpr int kBwdSmem = kWarps * kDepth<T> * 2 * 32 * 8 * sizeof(T);

// Gradient.  A warp walks units with a fixed stride and keeps the weights'
// sums of its columns in registers; a block writes its sum to the workspace
// (float32 [blocks][2][D]) and norm_rope_dw_kernel adds the blocks up, both in
// a fixed order, so the result is the same from run to run.  All of it is
// float32: a weight's sum of N = tokens x heads terms passes through a chain of
// about 2 N / 4864 + 95 additions at most, each off by 2^-24 of the sum so far.
// The registers this takes leave 16 warps per SM, too few for HBM's latency
// with loads into registers (102 us for 16384 tokens of 32 + 8 heads of 128,
// 94 this way, when this was built).  So the loads go to shared memory, kDepth
// sets ahead and on into the warp's next units: each lane fetches the 8
// elements that it will itself use, so no lane waits for another.
template <int D, typename T, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const NormRopeParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPS = 32 / LPR;
  constexpr int DEPTH = kDepth<T>;
  constexpr int PARTS = 8 * sizeof(T) / 16;    // 16-byte pieces of a lane's elements
  extern __shared__ uint4 ring_smem[];         // [warp][DEPTH][x, z][PARTS][lane]
  __shared__ float red[kWarps][2][D];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  const bool on = 8 * l < p.rot;
  const int src = sub * LPR + mate_lane(p, l);
  uint4* ring = ring_smem + warp * DEPTH * 2 * PARTS * 32 + lane;
  uint64_t dwq[4], dwk[4];                     // of the query and the key weight
#pragma unroll
  for (int i = 0; i < 4; ++i) dwq[i] = dwk[i] = f2(0.f, 0.f);

  // The set to be fetched next: this lane's place in x and dz, the heads and
  // the sets left of its kind, whether keys follow; and its place in the ring.
  Unit lu;
  unsigned lunit = blockIdx.x * kWarps + warp;
  const T *lx = nullptr, *lz = nullptr;
  int lheads = 0, lsets = 0;
  bool lkeys = false;
  auto begin_kind = [&](bool keys) {
    const int H = keys ? p.Hkv : p.Hq;
    const Heads hd = keys ? heads_of<RPS>(lu, p.sets_q, p.sets_k, sub) : heads_of<RPS>(lu, 0, p.sets_q, sub);
    lx = (keys ? static_cast<const T*>(p.k) + lu.t * p.k_stride : static_cast<const T*>(p.q) + lu.t * p.q_stride) + hd.h * D + 8 * l;
    lz = (keys ? static_cast<const T*>(p.dk_out) : static_cast<const T*>(p.dq_out)) + lu.t * H * D + hd.h * D + 8 * l;
    lheads = H - hd.h;
    lsets = hd.sets;
    lkeys = keys;
  };
  bool more = unit_at(p, lunit, lu);
  if (more) begin_kind(false);
  uint32_t lring = smem_u32(ring);
  const uint32_t ring_end = lring + DEPTH * 2 * PARTS * 32 * 16;
  auto fetch = [&] {
    if (more) {
      while (lsets == 0) {                     // on to the next kind or unit
        if (!lkeys) {
          begin_kind(true);
        } else {
          lunit += gridDim.x * kWarps;
          if (!(more = unit_at(p, lunit, lu))) break;
          begin_kind(false);
        }
      }
    }
    if (more) {
      const uint32_t bytes = lheads > 0 ? 16 : 0;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        copy16(lring + i * 512, lx + i * (16 / sizeof(T)), bytes);
        copy16(lring + (PARTS + i) * 512, lz + i * (16 / sizeof(T)), bytes);
      }
      lx += RPS * D;
      lz += RPS * D;
      lheads -= RPS;
      --lsets;
    }
    lring += 2 * PARTS * 512;
    if (lring == ring_end) lring = smem_u32(ring);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < DEPTH - 1; ++i) fetch();

  const uint4* oldest = ring;
  auto take = [&](Vec8<T>& x, Vec8<T>& z) {    // the oldest set of the ring
    fetch();
    asm volatile("cp.async.wait_group %0;" :: "n"(DEPTH - 1) : "memory");
    uint4 v[2 * PARTS];
#pragma unroll
    for (int i = 0; i < 2 * PARTS; ++i) v[i] = oldest[i * 32];
    x.from(v);
    z.from(v + PARTS);
    oldest += 2 * PARTS * 32;
    if (oldest == ring + DEPTH * 2 * PARTS * 32) oldest = ring;
  };

  Unit u;
  for (unsigned unit = blockIdx.x * kWarps + warp; unit_at(p, unit, u); unit += gridDim.x * kWarps) {
    const long long t = u.t;
    const int pos = p.rot ? __ldg(p.positions + t) : 0;
    const bool bad = p.rot && (pos < 0 || pos >= p.max_pos);
    if (bad && lane == 0) record_status(p.status, FA_ERR_POSITION);
    Angles ang = {};
    if (!bad) load_angles(p, pos, l, true, ang);
    auto rows = [&](T* d_at, int H, int from, int n, const float* weight, uint64_t* dw) {
      const Heads hd = heads_of<RPS>(u, from, n, sub);
      uint64_t w[4];
      if (weight && hd.sets) load_weights(weight, l, w);
      d_at += hd.h * D + 8 * l;
      int left = bad ? 0 : H - hd.h;           // the lane's heads: every RPS-th
#pragma unroll 1
      for (int k = 0; k < hd.sets; ++k, d_at += RPS * D, left -= RPS) {
        Vec8<T> x, z;
        take(x, z);
        const bool live = left > 0;
        uint64_t dy[4];
        {
          const Partners<T, INTER> y(p, z, src, on);
#pragma unroll
          for (int i = 0; i < 4; ++i) dy[i] = ffma2(z.pair(i), ang.c[i], fmul2(y.pair(i), ang.s[i]));
        }
        if (weight) {
          uint64_t g[4], ss = f2(0.f, 0.f), dot = f2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[i] = fmul2(dy[i], w[i]);
            ss = ffma2(x.pair(i), x.pair(i), ss);
            dot = ffma2(g[i], x.pair(i), dot);
          }
          float a = pair_sum(ss), b = pair_sum(dot);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
          }
          const float r = rsqrtf(a * (1.f / D) + p.eps);
          // xh = x r, dw += dy xh, dx = r (dy w - xh mean(dy w xh)); a row
          // that is not there adds nothing, whatever its r
          const float m = -(b * r * (1.f / D)) * r;
          const uint64_t r2 = f2(r, r), m2 = f2(m, m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t xh = fmul2(x.pair(i), r2);
            if (live) dw[i] = ffma2(dy[i], xh, dw[i]);
            dy[i] = ffma2(xh, m2, fmul2(g[i], r2));
          }
        }
        if (live) {
          Vec8<T> d;
#pragma unroll
          for (int i = 0; i < 4; ++i) d.set(i, dy[i]);
          d.store(d_at);
        }
      }
    };
    const bool norm = p.q_weight != nullptr;
    rows(static_cast<T*>(p.dq) + t * p.dq_stride, p.Hq, 0, p.sets_q, norm ? p.q_weight : nullptr, dwq);
    rows(static_cast<T*>(p.dk) + t * p.dk_stride, p.Hkv, p.sets_q, p.sets_k, norm ? p.k_weight : nullptr, dwk);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (p.q_weight) {
    // the warp's row groups, then the block's warps, in a fixed order
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        f2split(k ? dwk[i] : dwq[i], a, b);
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (lane < LPR) *reinterpret_cast<float2*>(&red[warp][k][8 * l + 2 * i]) = make_float2(a, b);
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

// Sum of the blocks' parts: one block per 32 of the 2 D columns, 32 strips of
// blocks per column (ten loads each, all on their way at once), added in a
// fixed order.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int nblocks, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  grid_dependency_wait();
  const int c = threadIdx.x & 31;
  const int strip = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  constexpr int kLoads = (kNormRopeBwdBlocks + 31) / 32;
  float x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) x[i] = strip + 32 * i < nblocks ? part[(long long)(strip + 32 * i) * 2 * D + col] : 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) s += x[i];
  red[strip][c] = s;
  __syncthreads();
  // warp `strip` adds up column `strip`
  s = red[c][strip];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (c == 0) {
    const int out = blockIdx.x * 32 + strip;
    if (out < D) dwq[out] = s;
    else dwk[out - D] = s;
  }
}

// Cuts a token's sets into units: as many sets per warp as still leave a GPU
// of GB300's size `want` warps, at least two (the loads of both overlap).
template <int D>
long long cut_units(NormRopeParams& p, bool values, int want) {
  constexpr int RPS = 32 / (D / 8);
  p.sets_q = (p.Hq + RPS - 1) / RPS;
  p.sets_k = (p.Hkv + RPS - 1) / RPS;
  p.sets_v = values ? p.sets_k : 0;
  const long long sets = p.sets_q + p.sets_k + p.sets_v;
  p.sets_per_unit = (int)std::min(sets, std::max(2ll, p.T * sets / want));
  p.units_per_token = (int)((sets + p.sets_per_unit - 1) / p.sets_per_unit);
  return p.T * p.units_per_token;
}

template <int D, typename T, bool PAGES>
int launch_fwd(NormRopeParams p, cudaStream_t stream) {
  const long long units = cut_units<D>(p, PAGES, kNormRopeWarps);
  auto kern = p.interleaved ? norm_rope_kernel<D, T, PAGES, true> : norm_rope_kernel<D, T, PAGES, false>;
  kern<<<(unsigned)((units + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
  return (int)cudaGetLastError();
}

template <int D>
int launch_append(NormRopeParams p, cudaStream_t stream) {
  const long long units = cut_units<D>(p, true, kNormRopeWarps);
  append_kernel<D><<<(unsigned)((units + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
  return (int)cudaGetLastError();
}

template <int D, typename T>
int launch_bwd(NormRopeParams p, cudaStream_t stream) {
  const long long units = cut_units<D>(p, false, kNormRopeWarps);
  const int grid = (int)std::min<long long>((units + kWarps - 1) / kWarps, kNormRopeBwdBlocks);
  auto kern = p.interleaved ? norm_rope_bwd_kernel<D, T, true> : norm_rope_bwd_kernel<D, T, false>;
  if (const int e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kBwdSmem<T>)) return e;
  kern<<<grid, kThreads, kBwdSmem<T>, stream>>>(p);
  if (const cudaError_t e = cudaGetLastError()) return (int)e;
  if (!p.q_weight) return 0;
  return launch_dependent(norm_rope_dw_kernel, dim3(2 * D / 32), dim3(1024), 0, stream,
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
  if (!p.q_weight && p.rot == 0) return p.d == 128 ? launch_append<128>(p, stream) : launch_append<64>(p, stream);
  return p.d == 128 ? launch_fwd<128, __nv_bfloat16, true>(p, stream) : launch_fwd<64, __nv_bfloat16, true>(p, stream);
}

int launch_norm_rope_bwd(const NormRopeParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (p.f32) return p.d == 128 ? launch_bwd<128, float>(p, stream) : launch_bwd<64, float>(p, stream);
  return p.d == 128 ? launch_bwd<128, __nv_bfloat16>(p, stream) : launch_bwd<64, __nv_bfloat16>(p, stream);
}

}  // namespace fa
