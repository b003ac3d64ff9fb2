// fa_fwd_paged_fp8.cu -- attention of each sequence's newest tokens over a cache
// in pages of e4m3 codes with a power of two for every 16 slots and head.
//
// Two kernels share a call: sequences that bring few rows (fa_fwd_paged_few.cu)
// and the others (fa_fwd_paged.cuh).  The one for few rows begins on the SMs that
// the other leaves.  Where the largest number of new tokens says that all
// sequences are of one kind, only that kernel runs: all of up to 32 rows, where the
// one for few is the faster (16 caches of 1k-32k tokens, one token each, 107-115 us by
// the box against 172 with the other; five tokens of 32 sequences, 20 rows, 123 against
// 139).  In a batch of both kinds it has the sequences of one token (up to their rows,
// in eights): 171 us against 187 with the other alone.
//
// For the others the products with the keys take the codes as they are, at twice
// the rate of bf16, so q has to be e4m3 too: times a power of two that brings a
// row's largest element to [2^7, 2^8) it is the sum of two e4m3 parts,
//     q 2^up = hi + lo,   hi = e4m3(q 2^up),  lo = e4m3(q 2^up - hi).
// bf16 has 8 bits, hi takes 4 of them and lo the others: exact for elements down
// to 2^-9 of the row's largest, and what the others lose is at most 2^-10, 2^-17
// of that one.  Both products go into one accumulator and cost what one in bf16
// does.  split_rows_kernel makes the parts, bound by HBM: 4 bytes per element.
#include "fa_fwd_paged.cuh"

namespace fa {
namespace {

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// A lane has 8 elements, D / 8 lanes a row.
template <int D>
__global__ void __launch_bounds__(256) split_rows_kernel(const PagedParams p) {
  constexpr int LPR = D / 8;
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x, rows = p.T * p.Hq;
  const long long row = at / LPR;
  const bool in = row < rows;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (in) x = __ldg(static_cast<const uint4*>(p.q) + at);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] << 16 & 0x7fff0000u, w[i] & 0x7fff0000u));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int up = min(7 - (max((int)(top >> 23), 1) - 127), 127);
  const float mul = pow2_cut(up);
  uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __uint_as_float(w[i] << 16) * mul, b = __uint_as_float(w[i] & 0xFFFF0000u) * mul;
    // an infinity is no e4m3 value; as NaN it makes the row NaN, as it would be
    if (!(fabsf(a) < INFINITY)) a = NAN;
    if (!(fabsf(b) < INFINITY)) b = NAN;
    const uint32_t h = e4m3x2(a, b);
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)h));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    hi[i / 2] |= h << (16 * (i & 1));
    lo[i / 2] |= e4m3x2(a - f.x, b - f.y) << (16 * (i & 1));
  }
  if (in) {
    reinterpret_cast<uint2*>(p.q_codes)[at] = make_uint2(hi[0], hi[1]);
    reinterpret_cast<uint2*>(p.q_codes + rows * D)[at] = make_uint2(lo[0], lo[1]);
    if (threadIdx.x % LPR == 0) p.q_exps[row] = up;
  }
  grid_launch_dependents();
}

template <int D>
int launch_two(const PagedParams& few, const PagedParams& many, cudaStream_t stream) {
  int nsm = 0;
  if (const int e = sm_count(&nsm)) return e;
  const int grid = std::min(nsm, kPagedCtas);
  const int ym = many.B ? (many.part_rows + 31) / 32 : 0, yf = few.B ? std::max(1, (few.part_rows + 7) / 8) : 0;
  if (many.B) {
    const long long blocks = (many.T * many.Hq * (D / 8) + 255) / 256;
    if (blocks >= (1ll << 31)) return (int)cudaErrorInvalidConfiguration;
    split_rows_kernel<D><<<(unsigned)blocks, 256, 0, stream>>>(many);
    if (const cudaError_t e = cudaGetLastError()) return (int)e;
    if (const int e = launch_d<D, true>(many, stream)) return e;
  }
  if (few.B)
    if (const int e = launch_fwd_paged_few(few, grid, many.B != 0, stream)) return e;
  return launch_dependent(paged_merge_two_kernel<D>, dim3(grid, ym + yf), dim3(256), 0, stream, few, many, ym, grid);
}

}  // namespace

#ifdef FA_PAGED_STOP
extern "C" int fa_selftest_paged_fp8_stop(int warp, int cta, int item) {
  const int at[3] = {warp, cta, item};
  return (int)cudaMemcpyToSymbol(g_stop, at, sizeof(at));
}
#endif

int launch_fwd_paged_fp8(const PagedParams& few, const PagedParams& many, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return (few.B ? few.d : many.d) == 128 ? launch_two<128>(few, many, stream) : launch_two<64>(few, many, stream);
}

}  // namespace fa
