// fa_fwd_paged.cu -- attention of each sequence's newest tokens over a cache in
// pages of bf16 (the kernel is in fa_fwd_paged.cuh).
#include "fa_fwd_paged.cuh"

namespace fa {

#ifdef FA_PAGED_STOP
extern "C" int fa_selftest_paged_stop(int warp, int cta, int item) {
  const int at[3] = {warp, cta, item};
  return (int)cudaMemcpyToSymbol(g_stop, at, sizeof(at));
}
#endif

int launch_fwd_paged(const PagedParams& p, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return p.d == 128 ? launch_d<128, false>(p, stream) : launch_d<64, false>(p, stream);
}

}  // namespace fa
