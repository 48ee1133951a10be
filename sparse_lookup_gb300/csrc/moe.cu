// moe.cu -- tokens sorted by expert and back, with their gradients (moe_* in
// emb.h).
#include <new>

#include "rows.cuh"

namespace emb {

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMinSpan = 4096;   // choices a CTA takes at least
constexpr int kMaxExperts = 2048;
constexpr int kRowThreads = 256;

struct RouteArgs {
  const int32_t* experts;
  int64_t n;             // choices
  int32_t n_experts, align;
  int64_t rows;          // R: rows of the expert-ordered arrays
  int64_t span;          // choices per CTA
  uint32_t* part;        // [CTAs][n_experts] choices of each expert in a CTA's span
  int32_t *offsets, *counts, *pos, *src;
};

__device__ __forceinline__ int expert_at(const RouteArgs& a, int64_t i) {
  const int e = a.experts[i];
  return e >= 0 && e < a.n_experts ? e : -1;
}

__global__ void __launch_bounds__(kRouteThreads) k_route_count(RouteArgs a) {
  extern __shared__ uint32_t hist[];
  for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * a.span, hi = min(a.n, lo + a.span);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kRouteThreads) {
    const int e = expert_at(a, i);
    if (e >= 0) atomicAdd(&hist[e], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads)
    a.part[(int64_t)blockIdx.x * a.n_experts + e] = hist[e];
}

// Exclusive sum over the CTA of one value per thread; every thread calls.
__device__ __forceinline__ uint32_t cta_exclusive(uint32_t x, uint32_t* wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  __syncthreads();
  return base + s - x;
}

// Places a CTA's span.  Shared: cnt [warps][experts] -- next row of each
// expert for each warp's part of the span.
__global__ void __launch_bounds__(kRouteThreads) k_route_place(RouteArgs a) {
  extern __shared__ uint32_t cnt[];
  __shared__ uint32_t wsum[kRouteWarps];
  const int E = a.n_experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* mine = cnt + warp * E;
  const int64_t lo = blockIdx.x * a.span, hi = min(a.n, lo + a.span);
  const int64_t part = (a.span / kRouteWarps + 31) / 32 * 32;
  const int64_t wlo = min(hi, lo + warp * part), whi = min(hi, wlo + part);
  for (int i = threadIdx.x; i < kRouteWarps * E; i += kRouteThreads) cnt[i] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 32) {
    const int e = expert_at(a, i);
    if (e >= 0) atomicAdd(&mine[e], 1u);
  }
  __syncthreads();
  // starts of the segments, then of each warp's share of them
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += kRouteThreads) {
    const int e = e0 + threadIdx.x;
    uint32_t before = 0, total = 0;
    if (e < E)
      for (unsigned c = 0; c < gridDim.x; ++c) {
        const uint32_t k = a.part[(int64_t)c * E + e];
        if (c < blockIdx.x) before += k;
        total += k;
      }
    const uint32_t room = (total + a.align - 1) / a.align * a.align;
    const uint32_t start = carry + cta_exclusive(room, wsum);
    if (e < E) {
      uint32_t row = start + before;
      for (int w = 0; w < kRouteWarps; ++w) {
        const uint32_t k = cnt[w * E + e];
        cnt[w * E + e] = row;
        row += k;
      }
      if (blockIdx.x == 0) {
        a.offsets[e] = (int32_t)start;
        a.counts[e] = (int32_t)total;
        if (e == E - 1) a.offsets[E] = (int32_t)(start + room);
      }
      if (e % gridDim.x == blockIdx.x)
        for (uint32_t r = start + total; r < start + room; ++r) a.src[r] = -1;
    }
    if (threadIdx.x == kRouteThreads - 1) wsum[0] = start + room;
    __syncthreads();
    carry = wsum[0];
    __syncthreads();
  }
  for (int64_t r = carry + blockIdx.x * (int64_t)kRouteThreads + threadIdx.x; r < a.rows;
       r += (int64_t)gridDim.x * kRouteThreads)
    a.src[r] = -1;
  const unsigned lt = (1u << lane) - 1u;
  for (int64_t i0 = wlo; i0 < whi; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < whi ? expert_at(a, i) : -1;
    const unsigned peers = __match_any_sync(kFull, e);
    uint32_t row = 0;
    if (e >= 0) row = mine[e] + __popc(peers & lt);
    __syncwarp();
    if (e >= 0 && (peers & lt) == 0) mine[e] += __popc(peers);
    __syncwarp();
    if (i < whi) {
      a.pos[i] = e >= 0 ? (int32_t)row : -1;
      if (e >= 0) a.src[row] = (int32_t)i;
    }
  }
}

// Rows are moved by groups of 2^GLOG lanes, V elements per access.
struct RowArgs {
  int64_t n, rows;       // tokens; rows of the expert-ordered arrays
  int32_t top_k, vecs;   // accesses per row
  const int32_t *pos, *src;
};

// -1 is a dropped choice; no position reaches outside the arrays.
__device__ __forceinline__ bool live_row(const RowArgs& a, int64_t p) { return p >= 0 && p < a.rows; }

template <class T, int V>
__device__ __forceinline__ void zero_padding(const RowArgs& a, T* xs, int glog) {
  const int sub = threadIdx.x & ((1 << glog) - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  Vec<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) z.e[i] = from_f32<T>(0.f);
  for (int64_t r = group; r < a.rows; r += groups)
    if (a.src[r] < 0)
      for (int j = sub; j < a.vecs; j += 1 << glog) store_vec(xs + (r * a.vecs + j) * V, z);
}

template <class T, int V>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(RowArgs a, const T* __restrict__ x, int64_t stride,
                                                          T* __restrict__ xs, int glog) {
  const int sub = threadIdx.x & ((1 << glog) - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  for (int64_t t = group; t < a.n; t += groups)
    for (int j = sub; j < a.vecs; j += 1 << glog) {
      const Vec<T, V> r = load_vec<T, V>(x + t * stride + (int64_t)j * V);
      for (int k = 0; k < a.top_k; ++k) {
        const int64_t p = a.pos[t * a.top_k + k];
        if (live_row(a, p)) store_vec(xs + (p * a.vecs + j) * V, r);
      }
    }
  zero_padding<T, V>(a, xs, glog);
}

template <class T, int V>
__global__ void __launch_bounds__(kRowThreads) k_combine(RowArgs a, const T* __restrict__ ys,
                                                         const float* __restrict__ w, T* __restrict__ y,
                                                         int64_t stride, int glog) {
  const int sub = threadIdx.x & ((1 << glog) - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  for (int64_t t = group; t < a.n; t += groups)
    for (int j = sub; j < a.vecs; j += 1 << glog) {
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
      for (int k = 0; k < a.top_k; ++k) {
        const int64_t p = a.pos[t * a.top_k + k];
        if (!live_row(a, p)) continue;
        const float wk = w ? w[t * a.top_k + k] : 1.f;
        const Vec<T, V> r = load_vec<T, V>(ys + (p * a.vecs + j) * V);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += wk * to_f32(r.e[i]);
      }
      Vec<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(acc[i]);
      store_vec(y + t * stride + (int64_t)j * V, o);
    }
}

template <class T, int V>
__global__ void __launch_bounds__(kRowThreads) k_combine_bwd(RowArgs a, const T* __restrict__ gy, int64_t stride,
                                                             const T* __restrict__ ys, const float* __restrict__ w,
                                                             T* __restrict__ gys, float* __restrict__ gw, int glog) {
  const int sub = threadIdx.x & ((1 << glog) - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  // every lane of a warp makes the same number of rounds (the sums shuffle)
  for (int64_t t0 = group - (group & ((32 >> glog) - 1)); t0 < a.n; t0 += groups) {
    const int64_t t = t0 + (group & ((32 >> glog) - 1));
    for (int k = 0; k < a.top_k; ++k) {
      const int64_t p = t < a.n ? a.pos[t * a.top_k + k] : -1;
      float dot = 0.f;
      if (live_row(a, p)) {
        const float wk = w ? w[t * a.top_k + k] : 1.f;
        for (int j = sub; j < a.vecs; j += 1 << glog) {
          const Vec<T, V> g = load_vec<T, V>(gy + t * stride + (int64_t)j * V);
          if (gw) {
            const Vec<T, V> r = load_vec<T, V>(ys + (p * a.vecs + j) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) dot += to_f32(g.e[i]) * to_f32(r.e[i]);
          }
          Vec<T, V> o;
#pragma unroll
          for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(wk * to_f32(g.e[i]));
          store_vec(gys + (p * a.vecs + j) * V, o);
        }
      }
      if (gw) {
        for (int o = (1 << glog) >> 1; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        if (sub == 0 && t < a.n) gw[t * a.top_k + k] = dot;
      }
    }
  }
  zero_padding<T, V>(a, gys, glog);
}

}  // namespace emb

struct emb_moe_s {
  int32_t n_experts = 0, top_k = 0, align = 1;
  int64_t max_tokens = 0;
  int sm_count = 0;
  uint32_t* part = nullptr;
};

using namespace emb;

namespace {

int64_t rows_of(const emb_moe_s* h, int64_t n) {
  const int64_t r = n * h->top_k + (int64_t)h->n_experts * (h->align - 1);
  return (r + h->align - 1) / h->align * h->align;
}

bool rows_ok(emb_moe h, int64_t n, int32_t dim, int32_t dtype) {
  return h && n >= 0 && n <= h->max_tokens && dim >= 1 && dim <= (1 << 20) && dtype_size(dtype) != 0;
}

// Largest access, in elements, that divides the row, both strides and every
// pointer (1 at the least: pointers are aligned to their element).
int access_width(int size, int32_t dim, int64_t stride, const void* a, const void* b, const void* c) {
  int v = 16 / size;
  while (v > 1 && (dim % v || stride % v || !aligned_to(a, v * size) || !aligned_to(b, v * size) ||
                   !aligned_to(c, v * size)))
    v >>= 1;
  return v;
}

// Lanes per row: the smallest power of two that covers a row's accesses, at
// most a warp.
int lanes_log(int vecs) {
  int g = 0;
  while (g < 5 && (1 << g) < vecs) ++g;
  return g;
}

unsigned row_grid(const emb_moe_s* h, int64_t groups, int glog) {
  const int64_t need = ((groups << glog) + kRowThreads - 1) / kRowThreads, most = (int64_t)h->sm_count * 8;
  return (unsigned)(need < 1 ? 1 : need < most ? need : most);
}

// Calls f with null pointers of the element type and of Vec<T, V> for the
// access width v.
template <class F>
void with_access(int32_t dtype, int v, F f) {
  with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    switch (v) {
      case 8:
        if constexpr (sizeof(T) == 2) f(t, (Vec<T, 8>*)nullptr, std::integral_constant<int, 8>());
        break;
      case 4: f(t, (Vec<T, 4>*)nullptr, std::integral_constant<int, 4>()); break;
      case 2: f(t, (Vec<T, 2>*)nullptr, std::integral_constant<int, 2>()); break;
      default: f(t, (Vec<T, 1>*)nullptr, std::integral_constant<int, 1>()); break;
    }
  });
}

}  // namespace

extern "C" emb_status moe_create(int32_t n_experts, int32_t top_k, int64_t max_tokens, int32_t align, emb_moe* out) {
  if (!out) return EMB_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_experts < 1 || top_k < 1 || max_tokens < 1 || align < 1) return EMB_ERR_INVALID_ARG;
  if (n_experts > kMaxExperts || top_k > 64 || align > 65536 || max_tokens >= (int64_t(1) << 31) ||
      max_tokens * top_k + (int64_t)n_experts * align >= (int64_t(1) << 31))
    return EMB_ERR_UNSUPPORTED;
  emb_moe_s* h = new (std::nothrow) emb_moe_s();
  if (!h) return EMB_ERR_OOM;
  h->n_experts = n_experts;
  h->top_k = top_k;
  h->align = align;
  h->max_tokens = max_tokens;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = dev_alloc((void**)&h->part, sizeof(uint32_t) * h->sm_count * n_experts);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_route_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRouteWarps * kMaxExperts * (int)sizeof(uint32_t));
  if (e != cudaSuccess) {
    dev_free(h->part);
    delete h;
    return cuda_status(e);
  }
  *out = h;
  return EMB_OK;
}

extern "C" emb_status moe_destroy(emb_moe h) {
  if (!h) return EMB_ERR_INVALID_ARG;
  const cudaError_t e = cudaDeviceSynchronize();
  dev_free(h->part);
  delete h;
  return cuda_status(e);
}

extern "C" emb_status moe_route(emb_moe h, int64_t n, const int32_t* experts, int32_t* offsets, int32_t* counts,
                                int32_t* pos, int32_t* src, void* stream) {
  if (!h || n < 0 || n > h->max_tokens || !offsets || !counts || (n > 0 && (!experts || !pos)) ||
      (rows_of(h, n) > 0 && !src))
    return EMB_ERR_INVALID_ARG;
  for (const void* p : {(const void*)experts, (const void*)offsets, (const void*)counts, (const void*)pos, (const void*)src})
    if (!aligned_to(p, 4)) return EMB_ERR_INVALID_ARG;
  RouteArgs a{experts, n * h->top_k, h->n_experts, h->align, rows_of(h, n), 0, h->part, offsets, counts, pos, src};
  int64_t ctas = (a.n + kRouteMinSpan - 1) / kRouteMinSpan;
  ctas = ctas < 1 ? 1 : ctas > h->sm_count ? h->sm_count : ctas;
  a.span = ((a.n + ctas - 1) / ctas + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
  cudaStream_t s = (cudaStream_t)stream;
  k_route_count<<<(unsigned)ctas, kRouteThreads, sizeof(uint32_t) * a.n_experts, s>>>(a);
  EMB_CUDA_TRY(cudaGetLastError());
  k_route_place<<<(unsigned)ctas, kRouteThreads, sizeof(uint32_t) * a.n_experts * kRouteWarps, s>>>(a);
  return cuda_status(cudaGetLastError());
}

extern "C" emb_status moe_dispatch(emb_moe h, int64_t n, int32_t dim, int32_t dtype, const void* x, int64_t x_stride,
                                   const int32_t* pos, const int32_t* src, void* xs, void* stream) {
  if (!rows_ok(h, n, dim, dtype) || x_stride < 0) return EMB_ERR_INVALID_ARG;
  const int size = dtype_size(dtype);
  const int64_t R = rows_of(h, n);
  if (R == 0) return EMB_OK;
  if ((n > 0 && (!x || !pos)) || !src || !xs || !aligned_to(x, size) || !aligned_to(xs, size) || !aligned_to(pos, 4) ||
      !aligned_to(src, 4))
    return EMB_ERR_INVALID_ARG;
  const int v = access_width(size, dim, x_stride, x, xs, nullptr);
  const RowArgs a{n, R, h->top_k, dim / v, pos, src};
  const int glog = lanes_log(a.vecs);
  with_access(dtype, v, [&](auto* t, auto*, auto V) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_dispatch<T, decltype(V)::value><<<row_grid(h, R, glog), kRowThreads, 0, (cudaStream_t)stream>>>(
        a, (const T*)x, x_stride, (T*)xs, glog);
  });
  return cuda_status(cudaGetLastError());
}

extern "C" emb_status moe_combine(emb_moe h, int64_t n, int32_t dim, int32_t dtype, const void* ys,
                                  const float* weights, const int32_t* pos, void* y, int64_t y_stride, void* stream) {
  if (!rows_ok(h, n, dim, dtype)) return EMB_ERR_INVALID_ARG;
  if (n == 0) return EMB_OK;
  const int size = dtype_size(dtype);
  if (!ys || !pos || !y || !aligned_to(ys, size) || !aligned_to(y, size) || !aligned_to(pos, 4) ||
      !aligned_to(weights, 4) || (n > 1 && y_stride < dim))
    return EMB_ERR_INVALID_ARG;
  const int v = access_width(size, dim, y_stride, ys, y, nullptr);
  const RowArgs a{n, rows_of(h, n), h->top_k, dim / v, pos, nullptr};
  const int glog = lanes_log(a.vecs);
  with_access(dtype, v, [&](auto* t, auto*, auto V) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_combine<T, decltype(V)::value><<<row_grid(h, n, glog), kRowThreads, 0, (cudaStream_t)stream>>>(
        a, (const T*)ys, weights, (T*)y, y_stride, glog);
  });
  return cuda_status(cudaGetLastError());
}

extern "C" emb_status moe_combine_backward(emb_moe h, int64_t n, int32_t dim, int32_t dtype, const void* grad_y,
                                           int64_t grad_y_stride, const void* ys, const float* weights,
                                           const int32_t* pos, const int32_t* src, void* grad_ys,
                                           float* grad_weights, void* stream) {
  if (!rows_ok(h, n, dim, dtype) || grad_y_stride < 0) return EMB_ERR_INVALID_ARG;
  const int size = dtype_size(dtype);
  const int64_t R = rows_of(h, n);
  if (R == 0) return EMB_OK;
  if ((n > 0 && (!grad_y || !pos || (grad_weights && !ys))) || !src || !grad_ys || !aligned_to(grad_y, size) ||
      !aligned_to(ys, size) || !aligned_to(grad_ys, size) || !aligned_to(pos, 4) || !aligned_to(src, 4) ||
      !aligned_to(weights, 4) || !aligned_to(grad_weights, 4))
    return EMB_ERR_INVALID_ARG;
  const int v = access_width(size, dim, grad_y_stride, grad_y, grad_weights ? ys : nullptr, grad_ys);
  const RowArgs a{n, R, h->top_k, dim / v, pos, src};
  const int glog = lanes_log(a.vecs);
  with_access(dtype, v, [&](auto* t, auto*, auto V) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_combine_bwd<T, decltype(V)::value><<<row_grid(h, R, glog), kRowThreads, 0, (cudaStream_t)stream>>>(
        a, (const T*)grad_y, grad_y_stride, (const T*)ys, weights, (T*)grad_ys, grad_weights, glog);
  });
  return cuda_status(cudaGetLastError());
}
