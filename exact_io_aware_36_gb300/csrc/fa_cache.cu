// fa_cache.cu -- copies of whole pages of a key / value cache.
//
// Pair i copies page src[i] to page dst[i], in the key pool and in the value
// pool.  A page is page_size * Hkv * d bf16 elements in one run, so a copy is
// bound by HBM: every byte read once and written once.  One block moves up to
// kChunk bytes of one page in both pools, all its loads in flight before its
// first store (one GB300: 4096 pages of 32 + 32 KB in 82 us, 6.5 TB/s, 96 % of
// the measured copy rate).
//
// The pairs run in no order, so a page written by one pair must not be read
// or written by another.  Each block looks for such pairs itself, while its
// loads are in flight: it compares its pair with all n, 8 n bytes out of L1
// and L2 beside the 4 * min(page bytes, kChunk) that it moves.  So the check
// grows with n^2, again for every chunk of a page: with pages of 32 KB it reads
// as much as the copy moves at 16384 pairs, with pages of 2 KB (16 tokens of
// one head of 64) at 1024, and at the limit of 131072 pairs 8 and 128 times as
// much.  A page below kChunk also leaves part of its block idle.  A pair in such a conflict copies
// nothing and is recorded, and so is one with a page outside the pool.
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                              // 16-byte pieces per thread and pool
constexpr int kChunk = kThreads * kPer * 16;         // bytes per block and pool

// SCALES: the pages hold codes, and their scales go with them (scale_bytes of
// each page, a few at a time by the block of the page's first chunk).
template <bool SCALES>
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const CachePagesCopy p) {
  const int i = (int)(blockIdx.x / p.chunks);
  const long long off = (long long)(blockIdx.x % p.chunks) * kChunk;
  const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
  if (s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages) {
    if (threadIdx.x == 0) record_status(p.status, FA_ERR_PAGE);
    return;
  }
  if (s == d) return;
  const long long from = (long long)s * p.page_bytes + off, to = (long long)d * p.page_bytes + off;
  const int n16 = (int)(min((long long)kChunk, p.page_bytes - off) / 16);
  uint4 x[2][kPer];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(v ? p.v : p.k) + from);
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (u * kThreads + threadIdx.x < n16) x[v][u] = __ldcs(at + u * kThreads + threadIdx.x);
  }
  uint8_t sc[2] = {0, 0};
  const bool scales = SCALES && off == 0;
  if (scales && threadIdx.x < p.scale_bytes) {
    sc[0] = p.k_scales[(long long)s * p.scale_bytes + threadIdx.x];
    sc[1] = p.v_scales[(long long)s * p.scale_bytes + threadIdx.x];
  }
  bool clash = false;
  for (int j = threadIdx.x; j < p.n; j += kThreads) {
    const int sj = __ldg(p.src + j), dj = __ldg(p.dst + j);
    if (j != i && sj != dj) clash |= dj == d || sj == d || dj == s;
  }
  if (__syncthreads_or(clash)) {
    if (threadIdx.x == 0) record_status(p.status, FA_ERR_PAGE);
    return;
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint4* at = reinterpret_cast<uint4*>(static_cast<char*>(v ? p.v : p.k) + to);
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (u * kThreads + threadIdx.x < n16) __stcs(at + u * kThreads + threadIdx.x, x[v][u]);
  }
  if (scales)
    for (int i = threadIdx.x; i < p.scale_bytes; i += kThreads) {
      if (i >= kThreads) {
        sc[0] = p.k_scales[(long long)s * p.scale_bytes + i];
        sc[1] = p.v_scales[(long long)s * p.scale_bytes + i];
      }
      p.k_scales[(long long)d * p.scale_bytes + i] = sc[0];
      p.v_scales[(long long)d * p.scale_bytes + i] = sc[1];
    }
}

}  // namespace

int launch_copy_pages(CachePagesCopy p, void* stream) {
  p.chunks = (unsigned)((p.page_bytes + kChunk - 1) / kChunk);
  const long long grid = (long long)p.n * p.chunks;
  if (grid >= (1ll << 31)) return (int)cudaErrorInvalidConfiguration;
  auto kern = p.k_scales ? copy_pages_kernel<true> : copy_pages_kernel<false>;
  kern<<<(unsigned)grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace fa
