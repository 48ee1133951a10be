// moe.cu -- tokens sorted by expert and back, with their gradients (moe_* in
// emb.h).
#include <new>

#include "moe.cuh"

namespace emb {

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteOne = 8192;       // choices that one CTA places alone
constexpr int kRouteMinSpan = 2048;   // choices of a CTA at least, where there are more
constexpr int kRowThreads = 128;
constexpr int kBwdCtas = 8;           // its CTAs on an SM: at 64 registers a lane only single fp32 columns spill (8 bytes)
constexpr int kInFlight = 4;          // accesses of a lane that the combine's backward keeps in flight

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

// How often each expert occurs in a CTA's span: counted in shared memory, so
// the choices (2 MB for 524288 of them) are all that is read.
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
  pdl_trigger();
  for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads) a.part[blockIdx.x * a.n_experts + e] = hist[e];
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
// expert for each warp's part of the span; of the experts' choices, those
// ahead of the span and all.  One CTA (ONE) counts for itself, without
// k_route_count: one launch in place of two pays up to kRouteOne choices.
// A warp ranks 32 choices at a time by matching lanes, so rows follow the
// choices' order.  Both kernels take 12 us for 524288 choices of 128 experts and
// 31 for 1.6 M of 512 (a floor of 1 and 3 us): latency bounds them, of the
// ranking's shared memory and of the spans' counts; more choices loaded ahead
// changed nothing.  16 choices of 16 experts take 2.8 us, a launch.
template <bool ONE>
__global__ void __launch_bounds__(kRouteThreads) k_route_place(RouteArgs a) {
  extern __shared__ uint32_t cnt[];
  __shared__ uint32_t wsum[kRouteWarps];
  const int E = a.n_experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t *mine = cnt + warp * E, *ahead = cnt + kRouteWarps * E, *all = ahead + E;
  if constexpr (!ONE) pdl_wait();
  const int64_t lo = blockIdx.x * a.span, hi = min(a.n, lo + a.span);
  const int64_t part = (a.span / kRouteWarps + 31) / 32 * 32;
  const int64_t wlo = min(hi, lo + warp * part), whi = min(hi, wlo + part);
  for (int i = threadIdx.x; i < (kRouteWarps + 2) * E; i += kRouteThreads) cnt[i] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 32) {
    const int e = expert_at(a, i);
    if (e >= 0) atomicAdd(&mine[e], 1u);
  }
  if constexpr (!ONE) {
    // the spans' counts, a row of E for each CTA: a thread sums its part of one
    // expert's column in registers, many loads in flight (65536 x 2 choices of
    // 1500 experts: 20 us in all, with eight in flight 31)
    const int wide = min(E, kRouteThreads), parts = kRouteThreads / wide, first = threadIdx.x / wide;
    for (int e = threadIdx.x % wide; first < parts && e < E; e += wide) {
      uint32_t total = 0, before = 0;
#pragma unroll 32
      for (int r = first; r < (int)gridDim.x; r += parts) {
        const uint32_t k = a.part[r * E + e];
        total += k;
        before += r < (int)blockIdx.x ? k : 0u;
      }
      if (total) atomicAdd(&all[e], total);
      if (before) atomicAdd(&ahead[e], before);
    }
  }
  __syncthreads();
  // starts of the segments, then of each warp's share of them
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += kRouteThreads) {
    const int e = e0 + threadIdx.x;
    uint32_t total = 0;
    if (e < E) {
      if constexpr (ONE)
        for (int w = 0; w < kRouteWarps; ++w) total += cnt[w * E + e];
      else
        total = all[e];
    }
    const uint32_t room = (total + a.align - 1) / a.align * a.align;
    const uint32_t start = carry + cta_exclusive(room, wsum);
    if (e < E) {
      uint32_t row = start + ahead[e];
#pragma unroll
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
  int e = wlo + lane < whi ? expert_at(a, wlo + lane) : -1;
  for (int64_t i0 = wlo; i0 < whi; i0 += 32) {
    const int64_t i = i0 + lane;
    const int next = i + 32 < whi ? expert_at(a, i + 32) : -1;
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
    e = next;
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

// Rows whose src is -1 become 0.  A warp looks at up to 32 neighbouring rows
// at once, at fewer where there are not enough to go round: padding comes in
// stretches, which few warps would otherwise fill.
template <class T, int V>
__device__ __forceinline__ void zero_padding(const RowArgs& a, T* xs) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> 5;
  const int64_t warps = ((int64_t)gridDim.x * kRowThreads) >> 5;
  int look = 1;
  while (look < 32 && look * warps < a.rows) look <<= 1;
  Vec<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) z.e[i] = from_f32<T>(0.f);
  for (int64_t r0 = warp * look; r0 < a.rows; r0 += warps * look) {
    unsigned empty = __ballot_sync(kFull, lane < look && r0 + lane < a.rows && a.src[r0 + lane] < 0);
    while (empty) {
      const int64_t r = r0 + __ffs(empty) - 1;
      empty &= empty - 1;
      for (int j = lane; j < a.vecs; j += 32) store_vec(xs + (r * a.vecs + j) * V, z);
    }
  }
}

// A token's rows, KU of them at a time: -1 where there is none.
template <int KU>
__device__ __forceinline__ void load_rows(const RowArgs& a, int64_t t, int k0, int32_t (&p)[KU]) {
#pragma unroll
  for (int u = 0; u < KU; ++u) {
    p[u] = k0 + u < a.top_k ? a.pos[t * a.top_k + k0 + u] : -1;
    if (!live_row(a, p[u])) p[u] = -1;
  }
}
template <int KU>
__device__ __forceinline__ void load_weights(const RowArgs& a, const float* w, int64_t t, int k0, float (&x)[KU]) {
#pragma unroll
  for (int u = 0; u < KU; ++u) x[u] = w && k0 + u < a.top_k ? w[t * a.top_k + k0 + u] : 1.f;
}

// Each row of x is read once and written to its top_k places, which no other
// kernel reads soon: they leave the caches first.  Bound by memory: 131072 x 4
// x 1024 bf16 with padding to 128 rows 211 us, 6.5 TB/s.
template <class T, int V, int KU>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(RowArgs a, const T* __restrict__ x, int64_t stride,
                                                          T* __restrict__ xs, int glog) {
  const int L = 1 << glog, sub = threadIdx.x & (L - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  for (int64_t t = group; t < a.n; t += groups)
    for (int k0 = 0; k0 < a.top_k; k0 += KU) {
      int32_t p[KU];
      load_rows<KU>(a, t, k0, p);
      const T* from = x + t * stride;
#pragma unroll 4
      for (int j = sub; j < a.vecs; j += L) {
        const Vec<T, V> r = load_vec<T, V>(from + (int64_t)j * V);
#pragma unroll
        for (int u = 0; u < KU; ++u)
          if (p[u] >= 0) store_last(xs + ((int64_t)p[u] * a.vecs + j) * V, r);
      }
    }
  zero_padding<T, V>(a, xs);
}

// Each row of ys is read once; a lane sums its columns of a token's rows in
// registers, in the order of k, with the rows' loads in flight together.
// Bound by memory: 131072 x 4 x 1024 bf16 198 us, 6.8 TB/s.
template <class T, int V, int KU>
__global__ void __launch_bounds__(kRowThreads) k_combine(RowArgs a, const T* __restrict__ ys,
                                                         const float* __restrict__ w, T* __restrict__ y,
                                                         int64_t stride, int glog) {
  const int L = 1 << glog, sub = threadIdx.x & (L - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  for (int64_t t = group; t < a.n; t += groups) {
    int32_t p[KU];
    float wk[KU];
    load_rows<KU>(a, t, 0, p);
    load_weights<KU>(a, w, t, 0, wk);
    for (int j = sub; j < a.vecs; j += L) {
      Pairs<V> acc;
#pragma unroll
      for (int i = 0; i < (V + 1) / 2; ++i) acc.p[i] = make_float2(0.f, 0.f);
      for (int k0 = 0;;) {
        Vec<T, V> r[KU];
#pragma unroll
        for (int u = 0; u < KU; ++u)
          if (p[u] >= 0) r[u] = load_vec<T, V>(ys + ((int64_t)p[u] * a.vecs + j) * V);
#pragma unroll
        for (int u = 0; u < KU; ++u)
          if (p[u] >= 0) {
            const Pairs<V> x = pairs_of(r[u]);
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) acc.p[i] = __ffma2_rn(make_float2(wk[u], wk[u]), x.p[i], acc.p[i]);
          }
        if (a.top_k <= KU) break;   // more choices than KU: their rows are looked up for every column
        k0 = k0 + KU < a.top_k ? k0 + KU : 0;
        load_rows<KU>(a, t, k0, p);
        load_weights<KU>(a, w, t, k0, wk);
        if (k0 == 0) break;
      }
      store_vec(y + t * stride + (int64_t)j * V, vec_of<T>(acc));
    }
  }
}

// Each row of ys is read once, each row of grad_ys written once, grad_y's row
// once where C accesses of a lane hold it (again from the caches for each k
// where it is wider).  4 / C choices go together, so that four accesses of a
// lane are in flight whatever the width; the lanes' partial dot products are
// joined by shuffles.  Bound by memory: 131072 x 4 x 1024 bf16 378 us, 6.5 TB/s
// (one product after the other bound it to 650).
template <class T, int V, int C>
__global__ void __launch_bounds__(kRowThreads, kBwdCtas) k_combine_bwd(RowArgs a, const T* __restrict__ gy, int64_t stride,
                                                             const T* __restrict__ ys, const float* __restrict__ w,
                                                             T* __restrict__ gys, float* __restrict__ gw, int glog) {
  constexpr int KB = kInFlight / C;
  const int L = 1 << glog, sub = threadIdx.x & (L - 1);
  const int64_t group = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) >> glog;
  const int64_t groups = ((int64_t)gridDim.x * kRowThreads) >> glog;
  const int in_warp = (int)(group & ((32 >> glog) - 1));
  // every lane of a warp makes the same number of rounds (the sums shuffle)
  for (int64_t t0 = group - in_warp; t0 < a.n; t0 += groups) {
    const int64_t t = t0 + in_warp;
    const bool ok = t < a.n;
    const T* from = gy + t * stride;
    Vec<T, V> g[C];
    const auto load_g = [&](int j0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (ok && j0 + c * L < a.vecs) g[c] = load_vec<T, V>(from + (int64_t)(j0 + c * L) * V);
    };
    load_g(sub);
    for (int k0 = 0; k0 < a.top_k; k0 += KB) {
      int32_t p[KB];
      float wk[KB], dot[KB];
      float2 part[KB];   // a dot product, even and odd columns
#pragma unroll
      for (int u = 0; u < KB; ++u) {
        p[u] = ok && k0 + u < a.top_k ? a.pos[t * a.top_k + k0 + u] : -1;
        if (!live_row(a, p[u])) p[u] = -1;
        wk[u] = w && p[u] >= 0 ? w[t * a.top_k + k0 + u] : 1.f;
        part[u] = make_float2(0.f, 0.f);
      }
      for (int j0 = sub; j0 < a.vecs; j0 += C * L) {
        if (C == 4 && a.vecs > C * L) load_g(j0);
        Vec<T, V> r[KB][C];
        if (gw) {
#pragma unroll
          for (int u = 0; u < KB; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (p[u] >= 0 && j0 + c * L < a.vecs)
                r[u][c] = load_vec<T, V>(ys + ((int64_t)p[u] * a.vecs + j0 + c * L) * V);
        }
#pragma unroll
        for (int u = 0; u < KB; ++u)
#pragma unroll
          for (int c = 0; c < C; ++c) {
            if (p[u] < 0 || j0 + c * L >= a.vecs) continue;
            const Pairs<V> x = pairs_of(g[c]), y = pairs_of(r[u][c]);
            Pairs<V> o;
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) {
              if (gw) part[u] = __ffma2_rn(x.p[i], y.p[i], part[u]);
              o.p[i] = __fmul2_rn(make_float2(wk[u], wk[u]), x.p[i]);
            }
            store_last(gys + ((int64_t)p[u] * a.vecs + j0 + c * L) * V, vec_of<T>(o));
          }
      }
      if (gw) {
#pragma unroll
        for (int u = 0; u < KB; ++u) dot[u] = part[u].x + part[u].y;
        for (int o = L >> 1; o; o >>= 1) {
#pragma unroll
          for (int u = 0; u < KB; ++u) dot[u] += __shfl_xor_sync(kFull, dot[u], o);
        }
#pragma unroll
        for (int u = 0; u < KB; ++u)
          if (sub == 0 && ok && k0 + u < a.top_k) gw[t * a.top_k + k0 + u] = dot[u];
      }
    }
  }
  zero_padding<T, V>(a, gys);
}

}  // namespace emb

using namespace emb;

namespace {

int64_t rows_of(const emb_moe_s* h, int64_t n) {
  const int64_t r = n * h->top_k + (int64_t)h->n_experts * (h->align - 1);
  return (r + h->align - 1) / h->align * h->align;
}

bool rows_ok(emb_moe h, int64_t n, int32_t dim, int32_t dtype) {
  return h && n >= 0 && n <= h->max_tokens && dim >= 1 && dim <= (1 << 20) && dtype_size(dtype) != 0 &&
         on_device(h->device);
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
  const int64_t need = ((groups << glog) + kRowThreads - 1) / kRowThreads, most = (int64_t)h->sm_count * 64;
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
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) e = dev_alloc((void**)&h->part, sizeof(uint32_t) * h->sm_count * n_experts);
  if (e == cudaSuccess) e = dev_alloc(&h->gate, gate_bytes(h->sm_count, n_experts));
  if (e == cudaSuccess) e = gate_clear(h->gate, h->sm_count, n_experts);
  for (auto k : {k_route_place<true>, k_route_place<false>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (kRouteWarps + 2) * kMaxExperts * (int)sizeof(uint32_t));
  if (e != cudaSuccess) {
    dev_free(h->part);
    dev_free(h->gate);
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
  dev_free(h->gate);
  delete h;
  return cuda_status(e);
}

extern "C" emb_status moe_route(emb_moe h, int64_t n, const int32_t* experts, int32_t* offsets, int32_t* counts,
                                int32_t* pos, int32_t* src, void* stream) {
  if (!h || n < 0 || n > h->max_tokens || !on_device(h->device) || !offsets || !counts || (n > 0 && (!experts || !pos)) ||
      (rows_of(h, n) > 0 && !src))
    return EMB_ERR_INVALID_ARG;
  for (const void* p : {(const void*)experts, (const void*)offsets, (const void*)counts, (const void*)pos, (const void*)src})
    if (!aligned_to(p, 4)) return EMB_ERR_INVALID_ARG;
  RouteArgs a{experts, n * h->top_k, h->n_experts, h->align, rows_of(h, n), 0, h->part, offsets, counts, pos, src};
  cudaStream_t s = (cudaStream_t)stream;
  const size_t smem = sizeof(uint32_t) * a.n_experts * (kRouteWarps + 2);
  const auto round = [](int64_t n) { return (n + kRouteThreads - 1) / kRouteThreads * kRouteThreads; };
  if (a.n <= kRouteOne) {
    a.span = round(a.n);
    k_route_place<true><<<1, kRouteThreads, smem, s>>>(a);
    return cuda_status(cudaGetLastError());
  }
  int64_t ctas = (a.n + kRouteMinSpan - 1) / kRouteMinSpan;
  if (ctas > h->sm_count) ctas = h->sm_count;
  a.span = round((a.n + ctas - 1) / ctas);
  k_route_count<<<(unsigned)ctas, kRouteThreads, sizeof(uint32_t) * a.n_experts, s>>>(a);
  EMB_CUDA_TRY(cudaGetLastError());
  return cuda_status(launch_dependent(k_route_place<false>, (unsigned)ctas, kRouteThreads, smem, s, a));
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
    constexpr int W = decltype(V)::value;
    auto k = h->top_k <= 2 ? k_dispatch<T, W, 2> : h->top_k <= 4 ? k_dispatch<T, W, 4> : k_dispatch<T, W, 8>;
    k<<<row_grid(h, n > R / 32 ? n : R / 32, glog), kRowThreads, 0, (cudaStream_t)stream>>>(a, (const T*)x, x_stride,
                                                                                          (T*)xs, glog);
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
    constexpr int W = decltype(V)::value;
    auto k = h->top_k <= 2 ? k_combine<T, W, 2> : h->top_k <= 4 ? k_combine<T, W, 4> : k_combine<T, W, 8>;
    k<<<row_grid(h, n, glog), kRowThreads, 0, (cudaStream_t)stream>>>(a, (const T*)ys, weights, (T*)y, y_stride, glog);
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
    constexpr int W = decltype(V)::value;
    auto k = a.vecs <= 32 ? k_combine_bwd<T, W, 1> : a.vecs <= 64 ? k_combine_bwd<T, W, 2> : k_combine_bwd<T, W, 4>;
    k<<<row_grid(h, n > R / 32 ? n : R / 32, glog), kRowThreads, 0, (cudaStream_t)stream>>>(
        a, (const T*)grad_y, grad_y_stride, (const T*)ys, weights, (T*)grad_ys, grad_weights, glog);
  });
  return cuda_status(cudaGetLastError());
}
