// delta_f16.cu -- the gated delta rule's chunked kernels for float16 elements.
#include "delta.cuh"

namespace emb {

template <>
cudaError_t run_delta<__half>(const emb_delta_s* h, const DeltaArgs& a, const DeltaViews& w, bool backward,
                          cudaStream_t s) {
  return launch_delta<__half>(h, a, w, backward, s);
}

}  // namespace emb
