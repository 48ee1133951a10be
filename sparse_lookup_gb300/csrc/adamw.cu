// adamw.cu -- one AdamW step over many tensors (adamw_* in emb.h), states in
// 32 bits or in 8-bit block codes.
#include <cmath>
#include <new>
#include <vector>

#include "rows.cuh"

namespace emb {

constexpr int kBlock = 256;        // elements that share a top: one warp, eight elements per lane
constexpr int kAdamThreads = 256;
constexpr int kChunk = 2048;       // elements of a CTA's pass: one block per warp

struct AdamTensor {
  void* param;
  float* master;
  void* m;
  void* v;
  int16_t* m_top;
  int16_t* v_top;
  int64_t numel;
  int64_t start;         // first element in the padded order of all tensors (a multiple of kBlock)
  float decay;
  int32_t aligned;       // every pointer allows 16-byte accesses of eight elements
};

struct AdamChunk {
  int32_t tensor;
  int32_t chunk;         // first element / kChunk
};

// A step's scalars, each computed in 64 bits and rounded once.
struct AdamScalars {
  float lr, b1, nb1, b2, nb2, c1, c2, eps;
  uint64_t key;          // SplitMix64 output for seed and step
};

// The place of each magnitude on the 8-bit grid, and back (emb.h).
__device__ __forceinline__ uint32_t magnitude(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
template <int LEVELS>
__device__ __forceinline__ uint32_t encode(float x, uint32_t noise, int base) {
  const int c = (int)((magnitude(x) + (noise << 4)) >> 20) - base;
  const uint32_t code = (uint32_t)max(c, 0);
  return LEVELS == 127 ? code | ((__float_as_uint(x) >> 24) & 0x80u) : code;
}
template <int LEVELS>
__device__ __forceinline__ float decode(uint32_t code, int base) {
  const uint32_t c = code & LEVELS;
  const uint32_t mag = c ? (c + (uint32_t)base) << 20 : 0u;
  return __uint_as_float(LEVELS == 127 ? mag | ((code & 0x80u) << 24) : mag);
}

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&r)[8], int n, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      const auto a = load_vec<T, 4>(p), b = load_vec<T, 4>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = to_f32(a.e[i]), r[4 + i] = to_f32(b.e[i]);
    } else {
      const auto a = load_vec<T, 8>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = to_f32(a.e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&r)[8], int n, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      Vec<T, 4> a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) a.e[i] = from_f32<T>(r[i]), b.e[i] = from_f32<T>(r[4 + i]);
      store_vec(p, a);
      store_vec(p + 4, b);
    } else {
      Vec<T, 8> a;
#pragma unroll
      for (int i = 0; i < 8; ++i) a.e[i] = from_f32<T>(r[i]);
      store_vec(p, a);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(r[i]);
  }
}

__device__ __forceinline__ uint64_t load_codes(const uint8_t* p, int n, bool vec) {
  if (vec) return *reinterpret_cast<const uint64_t*>(p);
  uint64_t c = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) c |= (uint64_t)p[i] << (8 * i);
  return c;
}

__device__ __forceinline__ void store_codes(uint8_t* p, uint64_t c, int n, bool vec) {
  if (vec) {
    *reinterpret_cast<uint64_t*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)(c >> (8 * i));
  }
}

// Writes a block's eight elements per lane as codes and its top.
template <int LEVELS>
__device__ __forceinline__ void store_state(uint8_t* codes, int16_t* top_p, const float (&x)[8], uint64_t z0,
                                            uint64_t z1, int n, bool vec) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) big = max(big, i < n ? magnitude(x[i]) : 0u);
  big = __reduce_max_sync(kFull, big);
  const int top = (int)((big + 0xfffffu) >> 20), base = max(top - LEVELS, 0);
  uint64_t c = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t noise = (uint32_t)((i < 4 ? z0 : z1) >> (16 * (i & 3))) & 0xffffu;
    c |= (uint64_t)encode<LEVELS>(x[i], noise, base) << (8 * i);
  }
  if (n > 0) store_codes(codes, c, n, vec);
  if ((threadIdx.x & 31) == 0) *top_p = (int16_t)top;
}

template <class P, class G, bool MASTER, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads) k_adamw(const AdamTensor* __restrict__ tensors,
                                                        const void* const* __restrict__ grads,
                                                        const AdamChunk* __restrict__ chunks, AdamScalars s,
                                                        const float* __restrict__ grad_scale) {
  const AdamChunk ch = chunks[blockIdx.x];
  const AdamTensor t = tensors[ch.tensor];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t block0 = (int64_t)ch.chunk * kChunk + warp * kBlock;
  if (block0 >= t.numel) return;
  const int64_t i0 = block0 + lane * 8;
  const int64_t left = t.numel - i0;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  const bool vec = t.aligned && n == 8;
  const G* gp = (const G*)grads[ch.tensor];
  const bool gvec = vec && ((uintptr_t)gp & 15) == 0;
  float g[8], w[8], m[8], v[8];
  load8(gp + i0, g, n, gvec);
  if constexpr (MASTER) load8(t.master + i0, w, n, vec);
  else load8((const P*)t.param + i0, w, n, vec);
  if constexpr (EIGHT) {
    const uint64_t mc = n ? load_codes((const uint8_t*)t.m + i0, n, vec) : 0;
    const uint64_t vc = n ? load_codes((const uint8_t*)t.v + i0, n, vec) : 0;
    const int mb = max((int)t.m_top[block0 / kBlock] - 127, 0), vb = max((int)t.v_top[block0 / kBlock] - 255, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = decode<127>((uint32_t)(mc >> (8 * i)) & 255u, mb);
      v[i] = decode<255>((uint32_t)(vc >> (8 * i)) & 255u, vb);
    }
    __syncwarp();   // every lane has the old tops
  } else {
    load8((const float*)t.m + i0, m, n, vec);
    load8((const float*)t.v + i0, v, n, vec);
  }
  const float scale = grad_scale ? *grad_scale : 1.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = __fmul_rn(g[i], scale);
    // each operation rounded by itself: the codes are then a function of the
    // formulas alone, whatever the compiler would have contracted
    m[i] = __fadd_rn(__fmul_rn(m[i], s.b1), __fmul_rn(gi, s.nb1));
    v[i] = __fadd_rn(__fmul_rn(v[i], s.b2), __fmul_rn(__fmul_rn(gi, gi), s.nb2));
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v[i] * s.c2));
    const float u = __fdividef(m[i] * s.c1, r + s.eps);
    w[i] = w[i] - s.lr * t.decay * w[i] - s.lr * u;
  }
  if constexpr (MASTER) store8(t.master + i0, w, n, vec);
  store8((P*)t.param + i0, w, n, vec);
  if constexpr (EIGHT) {
    const uint64_t group = (uint64_t)(t.start + i0) / 4;
    const uint64_t z0 = splitmix64(s.key + group), z1 = splitmix64(s.key + group + 1);
    store_state<127>((uint8_t*)t.m + i0, t.m_top + block0 / kBlock, m, z0, z1, n, vec);
    store_state<255>((uint8_t*)t.v + i0, t.v_top + block0 / kBlock, v, z0, z1, n, vec);
  } else {
    store8((float*)t.m + i0, m, n, vec);
    store8((float*)t.v + i0, v, n, vec);
  }
}

__global__ void __launch_bounds__(kAdamThreads) k_adamw_export(const AdamTensor* __restrict__ tensors,
                                                               const AdamChunk* __restrict__ chunks,
                                                               __nv_bfloat16* __restrict__ m_out,
                                                               __nv_bfloat16* __restrict__ v_out) {
  const AdamChunk ch = chunks[blockIdx.x];
  const AdamTensor t = tensors[ch.tensor];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t block0 = (int64_t)ch.chunk * kChunk + warp * kBlock;
  if (block0 >= t.numel) return;
  const int64_t i0 = block0 + lane * 8, left = t.numel - i0;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  const bool vec = t.aligned && n == 8;
  const uint64_t mc = n ? load_codes((const uint8_t*)t.m + i0, n, vec) : 0;
  const uint64_t vc = n ? load_codes((const uint8_t*)t.v + i0, n, vec) : 0;
  const int mb = max((int)t.m_top[block0 / kBlock] - 127, 0), vb = max((int)t.v_top[block0 / kBlock] - 255, 0);
  float m[8], v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = decode<127>((uint32_t)(mc >> (8 * i)) & 255u, mb);
    v[i] = decode<255>((uint32_t)(vc >> (8 * i)) & 255u, vb);
  }
  store8(m_out + t.start + i0, m, 8, true);   // a tensor's room is whole blocks: the rest of the last one is zeros
  store8(v_out + t.start + i0, v, 8, true);
}

// A kind of tensors: element types and master decide the kernel.
using AdamKernel = void (*)(const AdamTensor*, const void* const*, const AdamChunk*, AdamScalars, const float*);

template <class P, class G, bool MASTER>
AdamKernel adam_states(bool eight) {
  return eight ? (AdamKernel)k_adamw<P, G, MASTER, true> : (AdamKernel)k_adamw<P, G, MASTER, false>;
}
template <class P>
AdamKernel adam_half(bool f32_grad, bool master, bool eight) {
  if (f32_grad) return master ? adam_states<P, float, true>(eight) : adam_states<P, float, false>(eight);
  return master ? adam_states<P, P, true>(eight) : adam_states<P, P, false>(eight);
}
AdamKernel adam_kernel(int32_t dtype, int32_t grad_dtype, bool master, bool eight) {
  if (dtype == EMB_DT_F32) return adam_states<float, float, false>(eight);
  if (dtype == EMB_DT_BF16) return adam_half<__nv_bfloat16>(grad_dtype == EMB_DT_F32, master, eight);
  return adam_half<__half>(grad_dtype == EMB_DT_F32, master, eight);
}

struct AdamKind {
  AdamKernel kernel;
  int64_t first, count;   // its chunks
};

}  // namespace emb

struct emb_adamw_s {
  int32_t n = 0;
  bool eight = false;
  int64_t elements = 0;                 // of the padded order
  int64_t n_chunks = 0;
  std::vector<emb::AdamKind> kinds;
  std::vector<int32_t> grad_size;       // alignment of each tensor's gradient
  std::vector<int64_t> numel;
  emb::AdamTensor* tensors_d = nullptr;
  const void** grads_d = nullptr;
  emb::AdamChunk* chunks_d = nullptr;
};

using namespace emb;

namespace {

void free_adamw(emb_adamw_s* h) {
  dev_free(h->tensors_d);
  dev_free((void*)h->grads_d);
  dev_free(h->chunks_d);
  delete h;
}

bool tensor_ok(const adamw_tensor& t, bool eight) {
  if (t.numel < 0 || t.reserved != 0 || !(t.weight_decay >= 0.f) || std::isinf(t.weight_decay)) return false;
  const int size = dtype_size(t.dtype);
  if (size == 0 || (t.grad_dtype != t.dtype && t.grad_dtype != EMB_DT_F32)) return false;
  if (t.master && size == 4) return false;
  if (t.numel == 0) return true;
  if (!t.param || !t.grad || !t.m || !t.v) return false;
  if (!aligned_to(t.param, size) || !aligned_to(t.grad, dtype_size(t.grad_dtype)) || !aligned_to(t.master, 4)) return false;
  if (!eight) return aligned_to(t.m, 4) && aligned_to(t.v, 4);
  return t.m_top && t.v_top && aligned_to(t.m_top, 2) && aligned_to(t.v_top, 2);
}

emb_status create_adamw(const adamw_tensor* tensors, int32_t n, bool eight, emb_adamw_s* h) {
  h->n = n;
  h->eight = eight;
  std::vector<AdamTensor> meta(n);
  std::vector<const void*> grads(n);
  std::vector<std::vector<int32_t>> of_kind;
  std::vector<uint32_t> kind_key;
  for (int32_t i = 0; i < n; ++i) {
    const adamw_tensor& t = tensors[i];
    const size_t state_align = eight ? 8 : 16;
    meta[i] = AdamTensor{t.param, t.master, t.m, t.v, t.m_top, t.v_top, t.numel, h->elements, t.weight_decay,
                         aligned_to(t.param, 16) && aligned_to(t.master, 16) && aligned_to(t.m, state_align) &&
                             aligned_to(t.v, state_align)};
    grads[i] = t.grad;
    h->grad_size.push_back(dtype_size(t.grad_dtype));
    h->numel.push_back(t.numel);
    if (t.numel >= (int64_t(1) << 40) - h->elements) return EMB_ERR_UNSUPPORTED;
    h->elements += (t.numel + kBlock - 1) / kBlock * kBlock;
    if (t.numel == 0) continue;
    const uint32_t key = (uint32_t)t.dtype * 16 + (t.grad_dtype == EMB_DT_F32 ? 2 : 0) + (t.master ? 1 : 0);
    size_t k = 0;
    while (k < kind_key.size() && kind_key[k] != key) ++k;
    if (k == kind_key.size()) {
      kind_key.push_back(key);
      of_kind.emplace_back();
      h->kinds.push_back(AdamKind{adam_kernel(t.dtype, t.grad_dtype, t.master != nullptr, eight), 0, 0});
    }
    of_kind[k].push_back(i);
  }
  std::vector<AdamChunk> chunks;
  for (size_t k = 0; k < of_kind.size(); ++k) {
    h->kinds[k].first = (int64_t)chunks.size();
    for (int32_t i : of_kind[k]) {
      const int64_t c = (meta[i].numel + kChunk - 1) / kChunk;
      if ((int64_t)chunks.size() + c >= (int64_t(1) << 31)) return EMB_ERR_UNSUPPORTED;
      for (int64_t j = 0; j < c; ++j) chunks.push_back(AdamChunk{i, (int32_t)j});
    }
    h->kinds[k].count = (int64_t)chunks.size() - h->kinds[k].first;
  }
  h->n_chunks = (int64_t)chunks.size();
  EMB_CUDA_TRY(dev_alloc((void**)&h->tensors_d, sizeof(AdamTensor) * n));
  EMB_CUDA_TRY(dev_alloc((void**)&h->grads_d, sizeof(void*) * n));
  EMB_CUDA_TRY(dev_alloc((void**)&h->chunks_d, sizeof(AdamChunk) * (chunks.empty() ? 1 : chunks.size())));
  EMB_CUDA_TRY(cudaMemcpy(h->tensors_d, meta.data(), sizeof(AdamTensor) * n, cudaMemcpyHostToDevice));
  EMB_CUDA_TRY(cudaMemcpy((void*)h->grads_d, grads.data(), sizeof(void*) * n, cudaMemcpyHostToDevice));
  if (!chunks.empty())
    EMB_CUDA_TRY(cudaMemcpy(h->chunks_d, chunks.data(), sizeof(AdamChunk) * chunks.size(), cudaMemcpyHostToDevice));
  return EMB_OK;
}

}  // namespace

extern "C" emb_status adamw_create(const adamw_tensor* tensors, int32_t n, uint32_t flags, emb_adamw* out) {
  if (!out) return EMB_ERR_INVALID_ARG;
  *out = nullptr;
  if (!tensors || n < 1 || (flags & ~ADAMW_STATES_8BIT)) return EMB_ERR_INVALID_ARG;
  if (n >= (1 << 24)) return EMB_ERR_UNSUPPORTED;
  const bool eight = flags & ADAMW_STATES_8BIT;
  for (int32_t i = 0; i < n; ++i)
    if (!tensor_ok(tensors[i], eight)) return EMB_ERR_INVALID_ARG;
  emb_adamw_s* h = nullptr;
  emb_status st = EMB_ERR_OOM;
  try {
    h = new emb_adamw_s();
    st = create_adamw(tensors, n, eight, h);
  } catch (const std::bad_alloc&) {
    st = EMB_ERR_OOM;
  }
  if (st != EMB_OK) {
    if (h) free_adamw(h);
    return st;
  }
  *out = h;
  return EMB_OK;
}

extern "C" emb_status adamw_destroy(emb_adamw h) {
  if (!h) return EMB_ERR_INVALID_ARG;
  const cudaError_t e = cudaDeviceSynchronize();
  free_adamw(h);
  return cuda_status(e);
}

extern "C" emb_status adamw_bind_grads(emb_adamw h, const void* const* grads, void* stream) {
  if (!h || !grads) return EMB_ERR_INVALID_ARG;
  for (int32_t i = 0; i < h->n; ++i)
    if (h->numel[i] > 0 && (!grads[i] || !aligned_to(grads[i], h->grad_size[i]))) return EMB_ERR_INVALID_ARG;
  // pageable host memory: the copy has left the array when the call returns
  return cuda_status(cudaMemcpyAsync((void*)h->grads_d, grads, sizeof(void*) * h->n, cudaMemcpyHostToDevice,
                                     (cudaStream_t)stream));
}

extern "C" emb_status adamw_step(emb_adamw h, int64_t step, double lr, double beta1, double beta2, double eps,
                                 const float* grad_scale, uint32_t seed, void* stream) {
  if (!h || step < 1 || !(lr >= 0) || !(eps >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
      std::isinf(lr) || std::isinf(eps) || !aligned_to(grad_scale, 4))
    return EMB_ERR_INVALID_ARG;
  AdamScalars s;
  s.lr = (float)lr;
  s.b1 = (float)beta1;
  s.nb1 = (float)(1.0 - beta1);
  s.b2 = (float)beta2;
  s.nb2 = (float)(1.0 - beta2);
  s.c1 = (float)(1.0 / (1.0 - std::pow(beta1, (double)step)));
  s.c2 = (float)(1.0 / (1.0 - std::pow(beta2, (double)step)));
  s.eps = (float)eps;
  s.key = splitmix64(((uint64_t)seed << 32) + (uint64_t)step);
  for (const AdamKind& k : h->kinds) {
    k.kernel<<<(unsigned)k.count, kAdamThreads, 0, (cudaStream_t)stream>>>(h->tensors_d, h->grads_d,
                                                                          h->chunks_d + k.first, s, grad_scale);
    EMB_CUDA_TRY(cudaGetLastError());
  }
  return EMB_OK;
}

extern "C" emb_status adamw_export_size(emb_adamw h, int64_t* elements) {
  if (!h || !elements) return EMB_ERR_INVALID_ARG;
  *elements = h->elements;
  return EMB_OK;
}

extern "C" emb_status adamw_export_states(emb_adamw h, void* m_out, void* v_out, void* stream) {
  if (!h) return EMB_ERR_INVALID_ARG;
  if (!h->eight) return EMB_ERR_UNSUPPORTED;
  if (h->n_chunks == 0) return EMB_OK;
  if (!m_out || !v_out || !aligned16(m_out) || !aligned16(v_out)) return EMB_ERR_INVALID_ARG;
  k_adamw_export<<<(unsigned)h->n_chunks, kAdamThreads, 0, (cudaStream_t)stream>>>(
      h->tensors_d, h->chunks_d, (__nv_bfloat16*)m_out, (__nv_bfloat16*)v_out);
  return cuda_status(cudaGetLastError());
}
