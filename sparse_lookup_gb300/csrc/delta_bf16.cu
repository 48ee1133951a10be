// delta_bf16.cu -- the gated delta rule's chunked kernels for bfloat16 elements.
#include "delta.cuh"

namespace emb {

template <>
cudaError_t run_delta<__nv_bfloat16>(const emb_delta_s* h, const DeltaArgs& a, const DeltaViews& w, bool backward,
                          cudaStream_t s) {
  return launch_delta<__nv_bfloat16>(h, a, w, backward, s);
}

}  // namespace emb
