// moe.cuh -- the handle that the router's sources share (library-internal).
#pragma once

#include "rows.cuh"

struct emb_moe_s {
  int32_t n_experts = 0, top_k = 0, align = 1;
  int64_t max_tokens = 0;
  int sm_count = 0, device = 0;
  uint32_t* part = nullptr;   // [SMs][n_experts]
  void* gate = nullptr;       // the gate's sums (gate.cu)
};

namespace emb {

constexpr int kMaxExperts = 2048;

// Bytes of the gate's sums, and what they must hold before the first call.
size_t gate_bytes(int sm_count, int n_experts);
cudaError_t gate_clear(void* gate, int sm_count, int n_experts);

}  // namespace emb
