// fa_fwd_paged_fp8.cu -- attention of each sequence's newest tokens over a cache
// in pages of e4m3 codes with a power of two for every 16 slots and head.
//
// Two kernels share a call: sequences that bring few rows (fa_fwd_paged_few.cu)
// and the others (fa_fwd_paged.cuh).  The second begins on the SMs that the
// first leaves.  Where the largest number of new tokens says that all sequences
// are of one kind, only that kernel runs.
#include "fa_fwd_paged.cuh"

namespace fa {
namespace {

template <int D>
int launch_two(const PagedParams& few, const PagedParams& many, cudaStream_t stream) {
  int nsm = 0;
  if (const int e = sm_count(&nsm)) return e;
  const int grid = std::min(nsm, kPagedCtas);
  if (few.B == 0) return launch_d<D, true>(many, stream);
  if (const int e = launch_fwd_paged_few(few, grid, stream)) return e;
  const int rows = std::max(1, few.part_rows);
  if (many.B == 0)
    return launch_dependent(paged_merge_kernel<D>, dim3(grid, (rows + 7) / 8), dim3(256), 0, stream, few, grid);
  if (const int e = launch_d<D, true>(many, stream, true)) return e;
  return launch_dependent(paged_merge_two_kernel<D>, dim3(grid, (std::max(rows, many.part_rows) + 7) / 8, 2), dim3(256), 0,
                          stream, few, many, grid);
}

}  // namespace

int launch_fwd_paged_fp8(const PagedParams& few, const PagedParams& many, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return (few.B ? few.d : many.d) == 128 ? launch_two<128>(few, many, stream) : launch_two<64>(few, many, stream);
}

}  // namespace fa
