// fa_fwd_paged_fp8.cu -- attention of each sequence's newest tokens over a cache
// in pages of e4m3 codes with a power of two for every 16 slots and head.
#include "fa_fwd_paged.cuh"

namespace fa {

int launch_fwd_paged_fp8(const PagedParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return p.d == 128 ? launch_d<128, true>(p, stream) : launch_d<64, true>(p, stream);
}

}  // namespace fa
