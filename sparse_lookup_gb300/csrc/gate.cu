// gate.cu -- the gate in front of the router: choices, weights, counts and
// losses from a batch's logits, and the logits' gradient (moe_gate* in emb.h).
#include "moe.cuh"

namespace emb {

constexpr int kGateThreads = 256;
constexpr int kGateWarps = kGateThreads / 32;
constexpr int kGateCtas = 3;      // CTAs on an SM: as many as a token's 16 experts a lane leave registers for
constexpr int kGradCtas = 4;      // of the backward
constexpr int kSumCols = 8;       // experts of a CTA of the last reduction
constexpr int kSumRows = 64;      // CTAs' rows that it takes side by side

// What the CTAs of one call leave for the reduction.
struct GateSums {
  float* p;          // [CTAs][E] sums of the probabilities
  uint32_t* chosen;  // [CTAs][E]
  double* z;         // [CTAs] sums of lse^2
  uint32_t* live;    // [CTAs]
  double* share;     // [E / kSumCols] sums of counts * p of so many experts
  uint32_t* done;    // reducing CTAs that are through: 0 between calls
};

struct GateArgs {
  int64_t n;
  int32_t n_experts, top_k;
  int64_t stride;          // of logits' rows
  const uint8_t* live;     // NULL: all
  int normalize;
  int32_t *experts, *counts, *live_count;
  float *weights, *losses;
  float2* stats;
  GateSums sums;
};

// Sums, largest and smallest over the 2^k lanes of a token.
__device__ __forceinline__ float group_sum(float x, int L) {
  for (int o = 1; o < L; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
__device__ __forceinline__ float group_max(float x, int L) {
  for (int o = 1; o < L; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ int group_min(int x, int L) {
  for (int o = 1; o < L; o <<= 1) x = min(x, __shfl_xor_sync(kFull, x, o));
  return x;
}

// A token's logits in its lanes: element m of a lane is expert
// ((m / V) * L + lane) * V + m % V, so a lane's experts ascend with m.
template <class T, int V, int M>
__device__ __forceinline__ void load_logits(const T* row, int sub, int L, int E, bool live, float (&v)[M]) {
#pragma unroll
  for (int i = 0; i < M / V; ++i) {
    const int e = (i * L + sub) * V;
    if (live && e < E) {
      const Vec<T, V> x = load_vec<T, V>(row + e);
#pragma unroll
      for (int u = 0; u < V; ++u) v[i * V + u] = to_f32(x.e[u]);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u) v[i * V + u] = -INFINITY;
    }
  }
}
template <int V>
__device__ __forceinline__ int expert_of(int m, int sub, int L) {
  return ((m / V) * L + sub) * V + m % V;
}

// The balance and z losses from the whole batch's sums.
__device__ __forceinline__ void write_losses(const GateArgs& a, double share, double z, uint32_t live) {
  const double n = live ? (double)live : 1.0;
  a.losses[0] = (float)(share * a.n_experts / (n * n * a.top_k));
  a.losses[1] = (float)(z / n);
  *a.live_count = (int32_t)live;
}

// One pass over the logits.  A token's row stays in its lanes' registers: the
// largest, the sum of exponentials, then top_k rounds of (largest that is left,
// lowest expert of equals).  Few lanes a token (16 experts each where there are
// up to 512): a round's scan of the lane's own is cheaper than shuffles that
// every token pays.  Column sums of the probabilities stay in registers too, and
// leave as one row a CTA.  ONE: a single CTA, which writes the losses itself.  131072
// tokens of 128 fp32 logits, four choices: 47 us (67 MB), 285 instructions a token on two
// thirds of the issue slots.
template <class T, int V, int M, bool ONE>
__global__ void __launch_bounds__(kGateThreads, M <= 16 ? kGateCtas : 1) k_gate(GateArgs a, const T* __restrict__ logits, int glog) {
  extern __shared__ float held[];   // [warps][E] probabilities; [E] choices
  __shared__ double zs[kGateWarps];
  __shared__ uint32_t ns[kGateWarps];
  const int E = a.n_experts, K = a.top_k, L = 1 << glog, sub = threadIdx.x & (L - 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* chosen = (uint32_t*)(held + kGateWarps * E);
  for (int e = threadIdx.x; e < E; e += kGateThreads) chosen[e] = 0;
  __syncthreads();
  float psum[M];
#pragma unroll
  for (int m = 0; m < M; ++m) psum[m] = 0.f;
  float z32 = 0.f, lost = 0.f;   // a lane's sum of lse^2, and what its additions rounded off
  uint32_t count = 0;
  const int per = kGateThreads >> glog;
  const int64_t step = (int64_t)gridDim.x * per;
  // every lane of a warp makes the same number of rounds: the sums are joint
  for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.n; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> glog);
    const bool in = t < a.n;
    const bool live = in && (!a.live || a.live[t]);
    float v[M];
    load_logits<T, V, M>(logits + t * a.stride, sub, L, E, live, v);
    float top = v[0];
#pragma unroll
    for (int m = 1; m < M; ++m) top = fmaxf(top, v[m]);
    top = group_max(top, L);
    const bool some = top > -INFINITY;
    // the row's exponentials; an all -inf row has none
    const float base = some ? top : 0.f;
    float total = 0.f, e[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      e[m] = expf(v[m] - base);
      total += e[m];
    }
    total = group_sum(total, L);
    const float lse = some ? base + logf(total) : total > 0.f || total != total ? total : -INFINITY;
    const float inv = some ? 1.f / total : total;
#pragma unroll
    for (int m = 0; m < M; ++m) psum[m] += e[m] * inv;
    if (sub == 0 && in) {
      a.stats[t] = make_float2(top, total);
      if (lse != -INFINITY) {
        const float x = __fsub_rn(__fmul_rn(lse, lse), lost), s = __fadd_rn(z32, x);
        lost = __fsub_rn(__fsub_rn(s, z32), x);
        z32 = s;
        ++count;
      }
    }
    float kept = 0.f;   // of the chosen: their exponentials
    float mine_e = 0.f; // of the lane's last choice
    float best = top;
    for (int k = 0; k < K; ++k) {
      if (k) {
        best = v[0];
#pragma unroll
        for (int m = 1; m < M; ++m) best = fmaxf(best, v[m]);
        best = group_max(best, L);
      }
      int own = -1;   // the lane's first of the largest
#pragma unroll
      for (int m = M - 1; m >= 0; --m)
        if (v[m] == best) own = m;
      const bool any = best > -INFINITY;
      const int mine = own >= 0 ? expert_of<V>(own, sub, L) : 1 << 30, at = group_min(mine, L);
      if (mine != at) own = -1;
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (m == own) v[m] = -INFINITY;
      const float each = any ? expf(best - base) : 0.f;
      kept += each;
      if (in && sub == (k & (L - 1))) {
        a.experts[t * K + k] = any ? at : -1;
        mine_e = each;
        if (K > L) a.weights[t * K + k] = each;
        if (any) atomicAdd(&chosen[at], 1u);
      }
    }
    if (in) {
      // of the row, or over the chosen alone: where there are more choices than lanes, of what this lane wrote
      const float scale = !a.normalize ? inv : total != total ? total : kept > 0.f ? 1.f / kept : 0.f;
      if (K > L) {
        for (int k = sub; k < K; k += L) a.weights[t * K + k] *= scale;
      } else if (sub < K) {
        a.weights[t * K + sub] = mine_e * scale;
      }
    }
  }
  // a warp's tokens, then the warps in their order
  for (int o = L; o < 32; o <<= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) psum[m] += __shfl_xor_sync(kFull, psum[m], o);
  if (lane < L)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int e = expert_of<V>(m, sub, L);
      if (e < E) held[warp * E + e] = psum[m];
    }
  double z = z32;
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(kFull, z, o);
    count += __shfl_xor_sync(kFull, count, o);
  }
  if (lane == 0) zs[warp] = z, ns[warp] = count;
  __syncthreads();
  pdl_trigger();
  double share = 0.0;
  for (int e = threadIdx.x; e < E; e += kGateThreads) {
    float s = 0.f;
    for (int w = 0; w < kGateWarps; ++w) s += held[w * E + e];
    if constexpr (ONE) {
      a.counts[e] = (int32_t)chosen[e];
      share += (double)chosen[e] * s;
    } else {
      a.sums.p[(int64_t)blockIdx.x * E + e] = s;
      a.sums.chosen[(int64_t)blockIdx.x * E + e] = chosen[e];
    }
  }
  if constexpr (ONE) {
    for (int o = 16; o > 0; o >>= 1) share += __shfl_xor_sync(kFull, share, o);
    __shared__ double ss[kGateWarps];
    if (lane == 0) ss[warp] = share;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kGateWarps; ++w) share += ss[w], z += zs[w], count += ns[w];
      write_losses(a, share, z, count);
    }
  } else if (threadIdx.x == 0) {
    for (int w = 1; w < kGateWarps; ++w) z += zs[w], count += ns[w];
    a.sums.z[blockIdx.x] = z;
    a.sums.live[blockIdx.x] = count;
  }
}

// The CTAs' sums, kSumCols experts a CTA; the last one through adds up the parts, in
// their order.
__global__ void __launch_bounds__(kSumCols* kSumRows) k_gate_sum(GateArgs a, int ctas) {
  __shared__ float ps[kSumRows][kSumCols + 1];
  __shared__ uint32_t cs[kSumRows][kSumCols + 1];
  __shared__ uint32_t last;
  pdl_wait();
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols, e = blockIdx.x * kSumCols + col;
  const int E = a.n_experts, lane = threadIdx.x & 31;
  float p = 0.f;
  uint32_t c = 0;
  if (e < E)
#pragma unroll 4
    for (int i = row; i < ctas; i += kSumRows) {
      p += a.sums.p[(int64_t)i * E + e];
      c += a.sums.chosen[(int64_t)i * E + e];
    }
  ps[row][col] = p, cs[row][col] = c;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // four lanes an expert
  p = 0.f, c = 0;
  for (int i = lane / kSumCols; i < kSumRows; i += 32 / kSumCols) p += ps[i][col], c += cs[i][col];
  for (int o = kSumCols; o < 32; o <<= 1) {
    p += __shfl_xor_sync(kFull, p, o);
    c += __shfl_xor_sync(kFull, c, o);
  }
  if (e < E && lane < kSumCols) a.counts[e] = (int32_t)c;
  double share = (double)c * p;
  for (int o = kSumCols / 2; o > 0; o >>= 1) share += __shfl_xor_sync(kFull, share, o);
  if (lane == 0) {
    a.sums.share[blockIdx.x] = share;
    __threadfence();
    last = atomicAdd(a.sums.done, 1u) == gridDim.x - 1;
  }
  __syncwarp();
  if (!last) return;
  __threadfence();
  double z = 0.0;
  uint32_t n = 0;
  for (int i = lane; i < ctas; i += 32) z += a.sums.z[i], n += a.sums.live[i];
  share = 0.0;
  for (int i = lane; i < (int)gridDim.x; i += 32) share += ((volatile double*)a.sums.share)[i];
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(kFull, z, o);
    n += __shfl_xor_sync(kFull, n, o);
    share += __shfl_xor_sync(kFull, share, o);
  }
  if (lane == 0) {
    write_losses(a, share, z, n);
    *a.sums.done = 0;
  }
}

struct GateGrad {
  int64_t n;
  int32_t n_experts, top_k;
  int64_t stride, grad_stride;
  int normalize;
  const int32_t *experts, *counts, *live_count;
  const float* weights;
  const float2* stats;
  const float *grad_weights, *grad_losses;
};

// With c_e the balance loss' gradient of p_e, every logit gets
//   p_e (c_e - sum p c + 2 gz lse / n - [not normalised] sum w gw)
// and a chosen one w gw more (normalised: w (gw - sum w gw)).  One pass; the
// chosen are written over the row once it is there, by a lane each.  131072 x 128 fp32
// 35 us (4.0 TB/s).
template <class T, int V, int M>
__global__ void __launch_bounds__(kGateThreads) k_gate_bwd(GateGrad a, const T* __restrict__ logits,
                                                           T* __restrict__ grad, int glog) {
  extern __shared__ float held[];   // [E] c
  const int E = a.n_experts, K = a.top_k, L = 1 << glog, sub = threadIdx.x & (L - 1);
  const float n = fmaxf((float)*a.live_count, 1.f);
  const float gb = a.grad_losses ? a.grad_losses[0] : 0.f, gz = a.grad_losses ? a.grad_losses[1] : 0.f;
  const float each = gb * (float)E / (n * (float)K) / n;
  for (int e = threadIdx.x; e < E; e += kGateThreads) held[e] = each * (float)a.counts[e];
  __syncthreads();
  const int per = kGateThreads >> glog;
  const int64_t step = (int64_t)gridDim.x * per;
  for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.n; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> glog);
    const bool in = t < a.n;
    // the largest logit and the sum beside it, not their lse: that rounds off what a sum is beside a large logit
    const float2 st = in ? a.stats[t] : make_float2(-INFINITY, 0.f);
    const bool live = st.x != -INFINITY;
    const float inv = 1.f / st.y, lse = st.x + logf(st.y);
    float v[M];
    load_logits<T, V, M>(logits + t * a.stride, sub, L, E, live, v);
    float along = 0.f, mean = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int e = expert_of<V>(m, sub, L);
      v[m] = live ? expf(v[m] - st.x) * inv : 0.f;
      if (e < E) along += v[m] * held[e];
    }
    along = group_sum(along, L);
    if (live && a.grad_weights)
      for (int k = sub; k < K; k += L)
        if (a.experts[t * K + k] >= 0) mean += a.weights[t * K + k] * a.grad_weights[t * K + k];
    mean = group_sum(mean, L);
    const float off = (2.f * gz / n) * lse - along - (a.normalize ? 0.f : mean);
    if (in) {
      T* to = grad + t * a.grad_stride;
#pragma unroll
      for (int i = 0; i < M / V; ++i) {
        const int e = (i * L + sub) * V;
        if (e >= E) continue;
        Vec<T, V> o;
#pragma unroll
        for (int u = 0; u < V; ++u) o.e[u] = from_f32<T>(v[i * V + u] != 0.f ? v[i * V + u] * (held[e + u] + off) : 0.f);
        store_vec(to + e, o);
      }
    }
    __syncwarp();
    if (live && a.grad_weights)
      for (int k = sub; k < K; k += L) {
        const int e = a.experts[t * K + k];
        if (e < 0 || e >= E) continue;
        const float w = a.weights[t * K + k], gw = a.grad_weights[t * K + k];
        const float p = expf(to_f32(logits[t * a.stride + e]) - st.x) * inv;
        grad[t * a.grad_stride + e] = from_f32<T>(p * (held[e] + off) + w * (gw - (a.normalize ? mean : 0.f)));
      }
    __syncwarp();
  }
}

namespace {

GateSums sums_at(void* gate, int sm_count, int n_experts) {
  const size_t ctas = (size_t)sm_count * kGateCtas, E = n_experts;
  GateSums s;
  s.z = (double*)gate;
  s.share = s.z + ctas;
  s.p = (float*)(s.share + (E + kSumCols - 1) / kSumCols);
  s.chosen = (uint32_t*)(s.p + ctas * E);
  s.live = s.chosen + ctas * E;
  s.done = s.live + ctas;
  return s;
}
GateSums sums_of(const emb_moe_s* h) { return sums_at(h->gate, h->sm_count, h->n_experts); }

// Calls f with (T*, V, M) and the log of the lanes of a token.
template <class F>
cudaError_t with_gate(int32_t dtype, int E, bool wide, F f) {
  return with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    using std::integral_constant;
    const auto of = [&](auto width) {
      const auto lanes = [&](int m) {
        int g = 0;
        while ((m << g) < E) ++g;
        return g;
      };
      constexpr int V = decltype(width)::value, least = V > 4 ? V : 4;
      if (E <= 4 * least) return f(t, width, integral_constant<int, least>(), lanes(least));
      if (E <= 512) return f(t, width, integral_constant<int, 16>(), lanes(16));
      return f(t, width, integral_constant<int, 64>(), lanes(64));
    };
    constexpr int V = 16 / sizeof(T);
    return wide ? of(integral_constant<int, V>()) : of(integral_constant<int, 1>());
  });
}

bool gate_wide(int32_t dtype, int32_t E, int64_t stride, const void* p, int64_t stride2, const void* p2) {
  const int v = 16 / dtype_size(dtype);
  return E % v == 0 && stride % v == 0 && stride2 % v == 0 && aligned16(p) && aligned16(p2);
}

unsigned gate_grid(const emb_moe_s* h, int64_t n, int glog, int ctas) {
  const int per = kGateThreads >> glog;
  const int64_t need = (n + per - 1) / per, most = (int64_t)h->sm_count * ctas;
  return (unsigned)(need < most ? need : most);
}

}  // namespace

size_t gate_bytes(int sm_count, int n_experts) {
  return (size_t)((char*)(sums_at(nullptr, sm_count, n_experts).done + 1) - (char*)nullptr);
}
cudaError_t gate_clear(void* gate, int sm_count, int n_experts) {
  const cudaError_t e = cudaMemset(sums_at(gate, sm_count, n_experts).done, 0, sizeof(uint32_t));
  return e == cudaSuccess ? cudaDeviceSynchronize() : e;
}

}  // namespace emb

using namespace emb;

extern "C" emb_status moe_gate(emb_moe h, int64_t n, int32_t dtype, const void* logits, int64_t logits_stride,
                               const uint8_t* live, int32_t normalize, int32_t* experts, float* weights,
                               int32_t* counts, float* losses, float* stats, int32_t* live_count, void* stream) {
  if (!h || n < 0 || n > h->max_tokens || !on_device(h->device) || dtype_size(dtype) == 0 || logits_stride < 0 ||
      !counts || !losses || !live_count || (n > 0 && (!logits || !experts || !weights || !stats)) ||
      !aligned_to(logits, dtype_size(dtype)) || !aligned_to(stats, 8))
    return EMB_ERR_INVALID_ARG;
  for (const void* p : {(const void*)experts, (const void*)weights, (const void*)counts, (const void*)losses,
                        (const void*)live_count})
    if (!aligned_to(p, 4)) return EMB_ERR_INVALID_ARG;
  const int E = h->n_experts;
  const GateArgs a{n,      E,          h->top_k, logits_stride, live, normalize != 0, experts,
                   counts, live_count, weights,  losses,        (float2*)stats, sums_of(h)};
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(with_gate(dtype, E, gate_wide(dtype, E, logits_stride, logits, 0, nullptr),
                               [&](auto* t, auto width, auto count, int glog) {
    using T = std::remove_pointer_t<decltype(t)>;
    constexpr int V = decltype(width)::value, M = decltype(count)::value;
    const unsigned ctas = n ? gate_grid(h, n, glog, kGateCtas) : 1;
    const size_t smem = sizeof(float) * (kGateWarps + 1) * E;
    const auto kernel = ctas == 1 ? k_gate<T, V, M, true> : k_gate<T, V, M, false>;
    if (smem > 48 << 10) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    kernel<<<ctas, kGateThreads, smem, s>>>(a, (const T*)logits, glog);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || ctas == 1) return e;
    return launch_dependent(k_gate_sum, (unsigned)((E + kSumCols - 1) / kSumCols), kSumCols * kSumRows, 0, s, a,
                            (int)ctas);
  }));
}

extern "C" emb_status moe_gate_backward(emb_moe h, int64_t n, int32_t dtype, const void* logits,
                                        int64_t logits_stride, int32_t normalize, const int32_t* experts,
                                        const float* weights, const int32_t* counts, const float* stats,
                                        const int32_t* live_count, const float* grad_weights,
                                        const float* grad_losses, void* grad_logits, int64_t grad_stride,
                                        void* stream) {
  if (!h || n < 0 || n > h->max_tokens || !on_device(h->device) || dtype_size(dtype) == 0 || logits_stride < 0)
    return EMB_ERR_INVALID_ARG;
  if (n == 0) return EMB_OK;
  const int size = dtype_size(dtype), E = h->n_experts;
  if (!logits || !experts || !weights || !counts || !stats || !aligned_to(stats, 8) || !live_count || !grad_logits ||
      !aligned_to(logits, size) || !aligned_to(grad_logits, size) || (n > 1 && grad_stride < E) || grad_stride < 0)
    return EMB_ERR_INVALID_ARG;
  for (const void* p : {(const void*)experts, (const void*)weights, (const void*)counts, (const void*)live_count,
                        (const void*)grad_weights, (const void*)grad_losses})
    if (!aligned_to(p, 4)) return EMB_ERR_INVALID_ARG;
  const GateGrad a{n,      E,          h->top_k, logits_stride, grad_stride, normalize != 0, experts,
                   counts, live_count, weights,  (const float2*)stats, grad_weights, grad_losses};
  return cuda_status(with_gate(dtype, E, gate_wide(dtype, E, logits_stride, logits, grad_stride, grad_logits),
                               [&](auto* t, auto width, auto count, int glog) {
    using T = std::remove_pointer_t<decltype(t)>;
    const auto kernel = k_gate_bwd<T, decltype(width)::value, decltype(count)::value>;
    kernel<<<gate_grid(h, n, glog, kGradCtas), kGateThreads, sizeof(float) * E, (cudaStream_t)stream>>>(
        a, (const T*)logits, (T*)grad_logits, glog);
    return cudaGetLastError();
  }));
}
