// rows.cuh -- element types and vector accesses the dense operators share
// (library-internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "plan.cuh"

namespace emb {

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Two neighbouring elements as fp32, and back, in one or two instructions.
__device__ __forceinline__ float2 widen2(const float* p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 widen2(const __half* p) {
  return __half22float2(__half2{p[0], p[1]});
}
__device__ __forceinline__ float2 widen2(const __nv_bfloat16* p) {
  const __nv_bfloat162 h{p[0], p[1]};
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void narrow2(float* p, float2 x) { p[0] = x.x, p[1] = x.y; }
__device__ __forceinline__ void narrow2(__half* p, float2 x) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  p[0] = h.x, p[1] = h.y;
}
__device__ __forceinline__ void narrow2(__nv_bfloat16* p, float2 x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  p[0] = h.x, p[1] = h.y;
}

// V consecutive elements, moved in one access (V * sizeof(T) = 2, 4, 8 or 16).
template <class T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& v) {
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// Stored once and not read again soon: leaves the caches first.
template <class T, int V>
__device__ __forceinline__ void store_last(T* p, const Vec<T, V>& v) {
  if constexpr (sizeof(v) == 16) __stcs(reinterpret_cast<float4*>(p), *reinterpret_cast<const float4*>(&v));
  else if constexpr (sizeof(v) == 8) __stcs(reinterpret_cast<float2*>(p), *reinterpret_cast<const float2*>(&v));
  else store_vec(p, v);
}

// V elements as fp32 pairs; V = 1 leaves the second of its pair 0.
template <int V>
struct Pairs {
  float2 p[(V + 1) / 2];
};
template <class T, int V>
__device__ __forceinline__ Pairs<V> pairs_of(const Vec<T, V>& x) {
  Pairs<V> o;
  if constexpr (V == 1) {
    o.p[0] = make_float2(to_f32(x.e[0]), 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) o.p[i / 2] = widen2(&x.e[i]);
  }
  return o;
}
template <class T, int V>
__device__ __forceinline__ Vec<T, V> vec_of(const Pairs<V>& x) {
  Vec<T, V> o;
  if constexpr (V == 1) {
    o.e[0] = from_f32<T>(x.p[0].x);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) narrow2(&o.e[i], x.p[i / 2]);
  }
  return o;
}

inline int dtype_size(int32_t dtype) {
  return dtype == EMB_DT_F32 ? 4 : dtype == EMB_DT_BF16 || dtype == EMB_DT_F16 ? 2 : 0;
}

// A handle's calls run on the device that it was created on.
inline bool on_device(int device) {
  int now = -1;
  return cudaGetDevice(&now) == cudaSuccess && now == device;
}

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Calls f with a null pointer of the element type `dtype` names.
template <class F>
inline auto with_element(int32_t dtype, F f) {
  switch (dtype) {
    case EMB_DT_BF16: return f((__nv_bfloat16*)nullptr);
    case EMB_DT_F16: return f((__half*)nullptr);
    default: return f((float*)nullptr);
  }
}

}  // namespace emb
