// adamw.cu -- one AdamW step over many tensors (adamw_* in emb.h), states in
// 32 bits or in 8-bit block codes.
#include <cmath>
#include <new>
#include <vector>

#include "rows.cuh"

namespace emb {

constexpr int kBlock = 256;        // elements that share a top: one warp, eight elements per lane
constexpr int kAdamThreads = 128;
constexpr int kExportUnits = 2;
// CTAs on an SM: as many as hold a block's values without spilling much.
// Measured with 8-bit states on 128 M weights: bf16 262 us with 10, 267 with 9;
// bf16 with fp32 masters 365 and 353; 100 M fp32 283 and 248.
template <class P, bool MASTER>
constexpr int adam_ctas() { return sizeof(P) == 4 || MASTER ? 9 : 10; }

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

// A warp's work: one block of one tensor.
struct AdamUnit {
  int32_t tensor;
  int32_t block;
};

// A step's scalars, each computed in 64 bits and rounded once: those of its
// number, and the others.
struct AdamNumber {
  float lr_c1, c2;
  float limit;           // of the quotient before its correction by beta1; 0: none
  uint64_t key;          // SplitMix64 output for seed and step
};
struct AdamScalars {
  float lr, b1, nb1, b2, nb2, eps, one;
  bool flush;            // eps is large enough to drop roots below fp32's normal range
  AdamNumber n;
  int64_t step;
};
struct AdamHyper {
  double lr, beta1, beta2, eps, limit;
  uint32_t seed;
};
// The handle's count of steps, on the device, and the scalars of the number of a
// step that is counted there.
struct AdamCount {
  int64_t step;
  AdamNumber n;
};

// b^n by squaring, n >= 0: products alone, the same bits on host and device.
__host__ __device__ __noinline__ inline double power(double b, int64_t n) {
  double r = 1.0;
  for (; n; n >>= 1, b *= b)
    if (n & 1) r *= b;
  return r;
}
EMB_HD AdamNumber adam_number(const AdamHyper& h, int64_t step) {
  const double c1 = 1.0 - power(h.beta1, step);
  return {(float)(h.lr / c1), (float)(1.0 / (1.0 - power(h.beta2, step))), (float)(h.limit * c1),
          splitmix64(((uint64_t)h.seed << 32) + (uint64_t)step)};
}
inline AdamScalars adam_scalars(const AdamHyper& h, int64_t step) {
  AdamScalars s;
  s.lr = (float)h.lr;
  s.b1 = (float)h.beta1;
  s.nb1 = (float)(1.0 - h.beta1);
  s.b2 = (float)h.beta2;
  s.nb2 = (float)(1.0 - h.beta2);
  s.eps = (float)h.eps;
  s.one = 1.f;
  s.flush = h.eps >= 1e-12;
  s.n = step > 0 ? adam_number(h, step) : AdamNumber{};
  s.step = step;
  return s;
}

// The next step's number and what follows from it, on the device: where a call is
// replayed, its host part does not run again.  step > 0 sets the count.
__global__ void k_adamw_count(AdamHyper h, int64_t step, AdamCount* count) {
  count->step = step > 0 ? step : count->step + 1;
  count->n = adam_number(h, count->step);
}

// Places on the 8-bit grid, and back (emb.h).  Codes of eight elements are
// handled as two words of four bytes.
__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return __byte_perm(w, 0, 0x4440 + i); }
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t top4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

template <int LEVELS>
__device__ __forceinline__ void decode8(uint2 codes, int base, float (&x)[8]) {
  const uint32_t base20 = (uint32_t)base << 20;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? codes.y : codes.x;
    const uint32_t mags = LEVELS == 127 ? w & 0x7f7f7f7fu : w, signs = w & 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = byte_of(mags, i);
      uint32_t u = c ? (c << 20) + base20 : 0u;
      if (LEVELS == 127) u |= __byte_perm(signs, 0, 0x0444 | (i << 12));
      x[4 * h + i] = __uint_as_float(u);
    }
  }
}

// Largest magnitude of three and of eight, NaN if there is one.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max8(const float (&x)[8]) {
  return max3(max3(max3(x[0], x[1], x[2]), x[3], x[4]), max3(x[5], x[6], x[7]), 0.f);
}
__device__ __forceinline__ uint32_t magnitude(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// Rounds a block's eight elements per lane to codes; noise: 16 bits for each,
// two to a word.  Returns the block's top.  All lanes call.
template <int LEVELS>
__device__ __forceinline__ int encode8(const float (&x)[8], const uint32_t (&noise)[4], uint2& codes) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(x[i]) & 0x7fffffffu;
  uint32_t big = __reduce_max_sync(kFull, __float_as_uint(max8(x)));
  if (big >= 0x7f800000u) {   // some are not finite: they count for nothing and become 0
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, u[i] = magnitude(x[i]));
    big = __reduce_max_sync(kFull, most);
  }
  const int top = (int)((big + 0xfffffu) >> 20), base = max(top - LEVELS, 0);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t n = __byte_perm(noise[i >> 1], 0, i & 1 ? 0x4432 : 0x4410);
    // the code ends up in the top byte: shifts as products, which are not bound by the integer pipe
    c[i] = (uint32_t)__viaddmax_s32((int)(u[i] + 16u * n), -(base << 20), 0) * 16u;
  }
  codes = make_uint2(top4(c[0], c[1], c[2], c[3]), top4(c[4], c[5], c[6], c[7]));
  if (LEVELS == 127) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* f = x + 4 * h;
      (h ? codes.y : codes.x) |= top4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                      __float_as_uint(f[3])) & 0x80808080u;
    }
  }
  return top;
}

// Eight consecutive elements, as they are stored.
template <class T>
struct Eight {
  T e[8];
};
template <class T>
__device__ __forceinline__ void load8(const T* p, Eight<T>& r, int n, bool vec) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; i += V) {
      const auto x = load_vec<T, V>(p + i);
#pragma unroll
      for (int k = 0; k < V; ++k) r.e[i + k] = x.e[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
}
template <class T>
__device__ __forceinline__ void widen8(const Eight<T>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 f = widen2(&r.e[i]);
    x[i] = f.x, x[i + 1] = f.y;
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
      for (int i = 0; i < 8; i += 2) narrow2(&a.e[i], make_float2(r[i], r[i + 1]));
      store_last(p, a);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(r[i]);
  }
}

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n, bool vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = i < n ? p[i] : 0u;
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

__device__ __forceinline__ void store_codes(uint8_t* p, uint2 c, int n, bool vec) {
  if (vec) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)byte_of(i < 4 ? c.x : c.y, i & 3);
  }
}

__device__ __forceinline__ int lane_elements(const AdamTensor& t, int64_t i0) {
  const int64_t left = t.numel - i0;
  return left >= 8 ? 8 : left > 0 ? (int)left : 0;
}

// One block of one tensor, eight consecutive elements per lane, n of them the
// tensor's.  VEC: all of the block's are, and every access is wide.
template <class P, class G, bool MASTER, bool EIGHT, bool VEC>
__device__ __forceinline__ void adam_block(const AdamTensor& t, const G* gp, int64_t block, const AdamScalars& s,
                                           const AdamNumber& step, const float* grad_scale) {
  const int64_t i0 = block * kBlock + (threadIdx.x & 31) * 8;
  const int n = VEC ? 8 : lane_elements(t, i0);
  Eight<G> gr;
  Eight<std::conditional_t<MASTER, float, P>> wr;
  Eight<float> mr, vr;
  uint2 mc = make_uint2(0, 0), vc = make_uint2(0, 0);
  int mt, vt;
  load8(gp + i0, gr, n, VEC);
  if constexpr (MASTER) load8(t.master + i0, wr, n, VEC);
  else load8((const P*)t.param + i0, wr, n, VEC);
  if constexpr (EIGHT) {
    if (n) mc = load_codes((const uint8_t*)t.m + i0, n, VEC), vc = load_codes((const uint8_t*)t.v + i0, n, VEC);
    mt = t.m_top[block], vt = t.v_top[block];
  } else {
    load8((const float*)t.m + i0, mr, n, VEC);
    load8((const float*)t.v + i0, vr, n, VEC);
  }
  // the decay is a share of w taken off with the update, where the sum alone is
  // rounded to w's place: 1 - lr decay would itself be rounded to a place of 1
  // (lr decay = 1e-7: 19 % too much for every weight; below 3e-8: none)
  const float scale = grad_scale ? *grad_scale : 1.f, off = -(s.lr * t.decay);
  float g[8], w[8], m[8], v[8];
  if constexpr (EIGHT) {
    decode8<127>(mc, max(mt - 127, 0), m);
    decode8<255>(vc, max(vt - 255, 0), v);
  } else {
    widen8(mr, m);
    widen8(vr, v);
  }
  widen8(gr, g);
  widen8(wr, w);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const auto both = [](float x) { return make_float2(x, x); };
    float2 gi = make_float2(g[i], g[i + 1]), mi = make_float2(m[i], m[i + 1]), vi = make_float2(v[i], v[i + 1]);
    gi = __fmul2_rn(gi, both(scale));
    // Each operation rounded by itself, so that the codes are a function of the
    // formulas alone.  A packed product and sum would be joined to one
    // multiply-add by the compiler; a sum as a multiply-add by a 1 that it does
    // not know stays a sum.
    mi = __ffma2_rn(__fmul2_rn(mi, both(s.b1)), both(s.one), __fmul2_rn(gi, both(s.nb1)));
    vi = __ffma2_rn(__fmul2_rn(vi, both(s.b2)), both(s.one), __fmul2_rn(__fmul2_rn(gi, gi), both(s.nb2)));
    m[i] = mi.x, m[i + 1] = mi.y, v[i] = vi.x, v[i + 1] = vi.y;
    float2 r = __fmul2_rn(vi, both(step.c2)), q;
    if (s.flush) {
      // the flushing forms are single instructions; what they drop (a root
      // below 1.1e-19) is under 2^-23 of eps
      asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(r.x));
      asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(r.y));
      r = __fadd2_rn(r, both(s.eps));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.x));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.y));
      q = __fmul2_rn(mi, r);
    } else {
      asm("sqrt.approx.f32 %0, %0;" : "+f"(r.x));
      asm("sqrt.approx.f32 %0, %0;" : "+f"(r.y));
      r = __fadd2_rn(r, both(s.eps));
      q = make_float2(__fdividef(mi.x, r.x), __fdividef(mi.y, r.y));
    }
    if (step.limit > 0.f) {
      asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(q.x) : "f"(step.limit));
      asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(q.y) : "f"(step.limit));
    }
    const float2 w0 = make_float2(w[i], w[i + 1]);
    const float2 wi = __fadd2_rn(w0, __ffma2_rn(q, both(-step.lr_c1), __fmul2_rn(w0, both(off))));
    w[i] = wi.x, w[i + 1] = wi.y;
  }
  if constexpr (MASTER) store8(t.master + i0, w, n, VEC);
  store8((P*)t.param + i0, w, n, VEC);
  if constexpr (EIGHT) {
    const uint64_t group = (uint64_t)(t.start + i0) / 4;
    const uint64_t z0 = splitmix64(step.key + group), z1 = splitmix64(step.key + group + 1);
    const uint32_t noise[4] = {(uint32_t)z0, (uint32_t)(z0 >> 32), (uint32_t)z1, (uint32_t)(z1 >> 32)};
    mt = encode8<127>(m, noise, mc);
    if (n) store_codes((uint8_t*)t.m + i0, mc, n, VEC);
    vt = encode8<255>(v, noise, vc);
    if (n) store_codes((uint8_t*)t.v + i0, vc, n, VEC);
    if ((threadIdx.x & 31) == 0) t.m_top[block] = (int16_t)mt, t.v_top[block] = (int16_t)vt;
  } else {
    store8((float*)t.m + i0, m, n, VEC);
    store8((float*)t.v + i0, v, n, VEC);
  }
}

// The blocks at tensors' ends and off the 16-byte boundaries, out of line: they
// would cost the others registers.
template <class P, class G, bool MASTER, bool EIGHT>
__device__ __noinline__ void adam_ragged(const AdamTensor* t, const G* gp, int64_t block, const AdamScalars* s,
                                         const AdamNumber* step, const float* grad_scale) {
  adam_block<P, G, MASTER, EIGHT, false>(*t, gp, block, *s, *step, grad_scale);
}

// All bytes are read once and written once; a warp takes one block, and the
// other warps of the SM hide its loads.  With 16-bit weights and 8-bit states
// (10 bytes an element) the kernel is bound by instruction issue and the
// latency in front of it: arithmetic goes in pairs, codes in words of four.
// Warps that walked several blocks with the next one's loads ahead held fewer
// blocks in flight for the registers that took, and were slower.  128 M
// weights: fp32 506 us (7.1 TB/s), bf16 401 us and with masters 512 (7.0), 8-bit
// states with bf16 264 us (4.85 TB/s), with bf16 and masters 351 us (5.8 TB/s).
// Tensors off 16-byte boundaries go element by element (fp32 979 us, 8-bit states
// with bf16 540).
// COUNTED: the step's number is k_adamw_count's; otherwise it comes as an argument,
// like the other scalars, which costs no registers, and the count follows it
// (128 M weights with 8-bit states, replayed: bf16 268 us, with masters 329).
template <class P, class G, bool MASTER, bool EIGHT, bool COUNTED>
__global__ void __launch_bounds__(kAdamThreads, (adam_ctas<P, MASTER>()))
    k_adamw(const AdamTensor* __restrict__ tensors, const void* const* __restrict__ grads,
            const AdamUnit* __restrict__ units, int64_t n_units, const __grid_constant__ AdamScalars s,
            AdamCount* __restrict__ count, const float* __restrict__ grad_scale) {
  const int64_t i = (blockIdx.x * (int64_t)kAdamThreads + threadIdx.x) >> 5;
  if (i >= n_units) return;
  const AdamNumber& step = COUNTED ? count->n : s.n;
  if (!COUNTED && i == 0 && threadIdx.x == 0) count->step = s.step;
  const AdamUnit u = units[i];
  const AdamTensor& t = tensors[u.tensor];
  const G* gp = (const G*)grads[u.tensor];
  if (t.aligned && ((uintptr_t)gp & 15) == 0 && ((int64_t)u.block + 1) * kBlock <= t.numel)
    adam_block<P, G, MASTER, EIGHT, true>(t, gp, u.block, s, step, grad_scale);
  else
    adam_ragged<P, G, MASTER, EIGHT>(&t, gp, u.block, &s, &step, grad_scale);
}

// What the codes stand for, in bf16 (exact: three bits of fraction).  Bound by
// memory: 128 M elements 125 us, 6.2 TB/s.
__global__ void __launch_bounds__(kAdamThreads) k_adamw_export(const AdamTensor* __restrict__ tensors,
                                                               const AdamUnit* __restrict__ units, int64_t n_units,
                                                               __nv_bfloat16* __restrict__ m_out,
                                                               __nv_bfloat16* __restrict__ v_out) {
  constexpr int K = kExportUnits;   // a warp's units, their loads in flight together
  const int64_t first = ((blockIdx.x * (int64_t)kAdamThreads + threadIdx.x) >> 5) * K;
  uint2 mc[K], vc[K];
  int mt[K], vt[K];
  int64_t at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    at[k] = -1;
    if (first + k >= n_units) continue;
    const AdamUnit u = units[first + k];
    const AdamTensor& t = tensors[u.tensor];
    const int64_t i0 = (int64_t)u.block * kBlock + (threadIdx.x & 31) * 8;
    const int n = lane_elements(t, i0);
    const bool vec = t.aligned && n == 8;
    mc[k] = vc[k] = make_uint2(0, 0);
    if (n) mc[k] = load_codes((const uint8_t*)t.m + i0, n, vec), vc[k] = load_codes((const uint8_t*)t.v + i0, n, vec);
    mt[k] = t.m_top[u.block], vt[k] = t.v_top[u.block];
    at[k] = t.start + i0;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k] < 0) continue;
    float m[8], v[8];
    decode8<127>(mc[k], max(mt[k] - 127, 0), m);
    decode8<255>(vc[k], max(vt[k] - 255, 0), v);
    store8(m_out + at[k], m, 8, true);   // a tensor's room is whole blocks: the rest of the last one is zeros
    store8(v_out + at[k], v, 8, true);
  }
}

// Gradient addresses, by value: a launch holds them itself, whenever it runs (a
// copy from the host's array would read it later, and again in every replay of
// a graph).  As many as the 4 KB of arguments that any launch takes.
constexpr int kBindAtOnce = 480;
struct AdamBind {
  const void* grad[kBindAtOnce];
};
__global__ void __launch_bounds__(kBindAtOnce) k_adamw_bind(const __grid_constant__ AdamBind a, int n,
                                                            const void** __restrict__ grads) {
  const int i = threadIdx.x;
  if (i < n) grads[i] = a.grad[i];
}

// A kind of tensors: element types and master decide the kernel.
using AdamKernel = void (*)(const AdamTensor*, const void* const*, const AdamUnit*, int64_t, AdamScalars, AdamCount*,
                            const float*);
struct AdamKernels {
  AdamKernel given, counted;
};

template <class P, class G, bool MASTER>
AdamKernels adam_states(bool eight) {
  if (eight) return {k_adamw<P, G, MASTER, true, false>, k_adamw<P, G, MASTER, true, true>};
  return {k_adamw<P, G, MASTER, false, false>, k_adamw<P, G, MASTER, false, true>};
}
template <class P>
AdamKernels adam_half(bool f32_grad, bool master, bool eight) {
  if (f32_grad) return master ? adam_states<P, float, true>(eight) : adam_states<P, float, false>(eight);
  return master ? adam_states<P, P, true>(eight) : adam_states<P, P, false>(eight);
}
AdamKernels adam_kernels(int32_t dtype, int32_t grad_dtype, bool master, bool eight) {
  if (dtype == EMB_DT_F32) return adam_states<float, float, false>(eight);
  if (dtype == EMB_DT_BF16) return adam_half<__nv_bfloat16>(grad_dtype == EMB_DT_F32, master, eight);
  return adam_half<__half>(grad_dtype == EMB_DT_F32, master, eight);
}

struct AdamKind {
  AdamKernels kernels;
  int64_t first, count;   // its units
};

}  // namespace emb

struct emb_adamw_s {
  int32_t n = 0;
  int device = 0;
  bool eight = false;
  double limit = 0.0;                   // adamw_set_max_update
  int64_t elements = 0;                 // of the padded order
  int64_t n_units = 0;
  std::vector<emb::AdamKind> kinds;
  std::vector<int32_t> grad_size;       // alignment of each tensor's gradient
  std::vector<int64_t> numel;
  emb::AdamTensor* tensors_d = nullptr;
  const void** grads_d = nullptr;
  emb::AdamUnit* units_d = nullptr;
  emb::AdamCount* count_d = nullptr;
};

using namespace emb;

namespace {

void free_adamw(emb_adamw_s* h) {
  dev_free(h->tensors_d);
  dev_free((void*)h->grads_d);
  dev_free(h->units_d);
  dev_free(h->count_d);
  delete h;
}

// One warp per unit.
unsigned unit_grid(int64_t units) { return (unsigned)((units + kAdamThreads / 32 - 1) / (kAdamThreads / 32)); }

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
      h->kinds.push_back(AdamKind{adam_kernels(t.dtype, t.grad_dtype, t.master != nullptr, eight), 0, 0});
    }
    of_kind[k].push_back(i);
  }
  std::vector<AdamUnit> units;
  for (size_t k = 0; k < of_kind.size(); ++k) {
    h->kinds[k].first = (int64_t)units.size();
    for (int32_t i : of_kind[k]) {
      const int64_t blocks = (meta[i].numel + kBlock - 1) / kBlock;
      if ((int64_t)units.size() + blocks >= (int64_t(1) << 31)) return EMB_ERR_UNSUPPORTED;
      for (int64_t j = 0; j < blocks; ++j) units.push_back(AdamUnit{i, (int32_t)j});
    }
    h->kinds[k].count = (int64_t)units.size() - h->kinds[k].first;
  }
  h->n_units = (int64_t)units.size();
  EMB_CUDA_TRY(cudaGetDevice(&h->device));
  EMB_CUDA_TRY(dev_alloc((void**)&h->tensors_d, sizeof(AdamTensor) * n));
  EMB_CUDA_TRY(dev_alloc((void**)&h->grads_d, sizeof(void*) * n));
  EMB_CUDA_TRY(dev_alloc((void**)&h->units_d, sizeof(AdamUnit) * (units.empty() ? 1 : units.size())));
  EMB_CUDA_TRY(dev_alloc((void**)&h->count_d, sizeof(AdamCount)));
  EMB_CUDA_TRY(cudaMemset(h->count_d, 0, sizeof(AdamCount)));
  EMB_CUDA_TRY(cudaMemcpy(h->tensors_d, meta.data(), sizeof(AdamTensor) * n, cudaMemcpyHostToDevice));
  EMB_CUDA_TRY(cudaMemcpy((void*)h->grads_d, grads.data(), sizeof(void*) * n, cudaMemcpyHostToDevice));
  if (!units.empty())
    EMB_CUDA_TRY(cudaMemcpy(h->units_d, units.data(), sizeof(AdamUnit) * units.size(), cudaMemcpyHostToDevice));
  // a copy from pageable memory may return before it has arrived, and a step on
  // a non-blocking stream does not wait for the stream that it runs on
  return cuda_status(cudaStreamSynchronize(nullptr));
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
  if (!h || !grads || !on_device(h->device)) return EMB_ERR_INVALID_ARG;
  for (int32_t i = 0; i < h->n; ++i)
    if (h->numel[i] > 0 && (!grads[i] || !aligned_to(grads[i], h->grad_size[i]))) return EMB_ERR_INVALID_ARG;
  for (int32_t first = 0; first < h->n; first += kBindAtOnce) {
    const int32_t left = h->n - first, k = left < kBindAtOnce ? left : kBindAtOnce;
    AdamBind a{};
    for (int32_t i = 0; i < k; ++i) a.grad[i] = grads[first + i];
    k_adamw_bind<<<1, kBindAtOnce, 0, (cudaStream_t)stream>>>(a, k, h->grads_d + first);
    EMB_CUDA_TRY(cudaGetLastError());
  }
  return EMB_OK;
}

extern "C" emb_status adamw_step(emb_adamw h, int64_t step, double lr, double beta1, double beta2, double eps,
                                 const float* grad_scale, uint32_t seed, void* stream) {
  if (!h || step < 0 || !(lr >= 0) || !(eps >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
      std::isinf(lr) || std::isinf(eps) || !aligned_to(grad_scale, 4) || !on_device(h->device))
    return EMB_ERR_INVALID_ARG;
  const cudaStream_t st = (cudaStream_t)stream;
  if (step > 0) {   // a replay would take the same step again
    cudaStreamCaptureStatus capture;
    EMB_CUDA_TRY(cudaStreamIsCapturing(st, &capture));
    if (capture != cudaStreamCaptureStatusNone) return EMB_ERR_UNSUPPORTED;
  }
  const AdamHyper hyper{lr, beta1, beta2, eps, h->limit, seed};
  const AdamScalars s = adam_scalars(hyper, step);
  if (step == 0 || h->kinds.empty()) {
    k_adamw_count<<<1, 1, 0, st>>>(hyper, step, h->count_d);
    EMB_CUDA_TRY(cudaGetLastError());
  }
  for (const AdamKind& k : h->kinds) {
    (step > 0 ? k.kernels.given : k.kernels.counted)<<<unit_grid(k.count), kAdamThreads, 0, st>>>(
        h->tensors_d, h->grads_d, h->units_d + k.first, k.count, s, h->count_d, grad_scale);
    EMB_CUDA_TRY(cudaGetLastError());
  }
  return EMB_OK;
}

extern "C" emb_status adamw_set_max_update(emb_adamw h, double limit) {
  if (!h || !(limit >= 0)) return EMB_ERR_INVALID_ARG;
  h->limit = std::isinf(limit) ? 0.0 : limit;
  return EMB_OK;
}

extern "C" emb_status adamw_get_step(emb_adamw h, int64_t* step, void* stream) {
  if (!h || !step) return EMB_ERR_INVALID_ARG;
  EMB_CUDA_TRY(cudaMemcpyAsync(step, &h->count_d->step, sizeof(int64_t), cudaMemcpyDeviceToHost, (cudaStream_t)stream));
  return cuda_status(cudaStreamSynchronize((cudaStream_t)stream));
}

extern "C" emb_status adamw_set_step(emb_adamw h, int64_t step, void* stream) {
  if (!h || step < 0) return EMB_ERR_INVALID_ARG;
  EMB_CUDA_TRY(cudaMemcpyAsync(&h->count_d->step, &step, sizeof(int64_t), cudaMemcpyHostToDevice, (cudaStream_t)stream));
  return cuda_status(cudaStreamSynchronize((cudaStream_t)stream));
}

extern "C" emb_status adamw_export_size(emb_adamw h, int64_t* elements) {
  if (!h || !elements) return EMB_ERR_INVALID_ARG;
  *elements = h->elements;
  return EMB_OK;
}

extern "C" emb_status adamw_export_states(emb_adamw h, void* m_out, void* v_out, void* stream) {
  if (!h || !on_device(h->device)) return EMB_ERR_INVALID_ARG;
  if (!h->eight) return EMB_ERR_UNSUPPORTED;
  if (h->n_units == 0) return EMB_OK;
  if (!m_out || !v_out || !aligned16(m_out) || !aligned16(v_out)) return EMB_ERR_INVALID_ARG;
  k_adamw_export<<<unit_grid((h->n_units + kExportUnits - 1) / kExportUnits), kAdamThreads, 0, (cudaStream_t)stream>>>(
      h->tensors_d, h->units_d, h->n_units, (__nv_bfloat16*)m_out, (__nv_bfloat16*)v_out);
  return cuda_status(cudaGetLastError());
}
