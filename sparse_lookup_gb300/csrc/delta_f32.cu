// delta_f32.cu -- the gated delta rule's chunked kernels for float32 elements.
#include "delta.cuh"

namespace emb {

template <>
cudaError_t run_delta<float>(const emb_delta_s* h, const DeltaArgs& a, const DeltaViews& w, bool backward,
                          cudaStream_t s) {
  return launch_delta<float>(h, a, w, backward, s);
}

}  // namespace emb
