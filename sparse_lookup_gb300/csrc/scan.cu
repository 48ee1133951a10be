// scan.cu -- gated linear recurrence over padded sequences, forward, backward
// and one position at a time (scan_* in emb.h).
#include <new>

#include "rows.cuh"

struct emb_scan_s {
  int32_t dim = 0, max_batch = 0, max_len = 0;
  int sm_count = 0;
  uint32_t* status_d = nullptr;
};

namespace emb {

// sigmoid(g) and sigmoid(-g), each from its own quotient: 1 - a would lose
// every digit of the smaller one where the gate saturates.
__device__ __forceinline__ void gates(float g, float& a, float& na) {
  const float e = __expf(-fabsf(g));
  const float hi = __fdividef(1.f, 1.f + e), lo = e * hi;
  a = g >= 0.f ? hi : lo;
  na = g >= 0.f ? lo : hi;
  if (g != g) a = na = g;
}

template <class T>
struct View {
  T* p;
  int64_t bs, ts;
  __device__ T* at(int64_t b, int64_t t, int64_t d) const { return p + b * bs + t * ts + d; }
};

struct ScanArgs {
  int32_t batch, len, dim;
  const int32_t* offsets;
  uint32_t* status;
};

__device__ __forceinline__ int live_len(const ScanArgs& s, int b) {
  if (!s.offsets) return s.len;
  const int64_t n = (int64_t)__ldg(s.offsets + b + 1) - __ldg(s.offsets + b);
  if (n < 0) latch(s.status, EMB_ERR_BAD_INDEX);
  return n < 0 ? 0 : n > s.len ? s.len : (int)n;
}

template <class T>
__global__ void __launch_bounds__(128) k_scan_fwd(ScanArgs s, View<const T> x, View<const T> g, View<T> y,
                                                  const float* state_in, float* state_out) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i >= (int64_t)s.batch * s.dim) return;
  const int b = (int)(i / s.dim), d = (int)(i % s.dim);
  const int n = live_len(s, b);
  float h = state_in ? state_in[i] : 0.f;
  for (int t = 0; t < n; ++t) {
    float a, na;
    gates(to_f32(*g.at(b, t, d)), a, na);
    h = a * h + na * to_f32(*x.at(b, t, d));
    *y.at(b, t, d) = from_f32<T>(h);
  }
  for (int t = n; t < s.len; ++t) *y.at(b, t, d) = from_f32<T>(0.f);
  if (state_out) state_out[i] = h;
}

template <class T>
__global__ void __launch_bounds__(128) k_scan_bwd(ScanArgs s, View<const T> x, View<const T> g, View<const T> y,
                                                  View<const T> gy, const float* state_in, const float* grad_out,
                                                  View<T> gx, View<T> gg, float* grad_in) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i >= (int64_t)s.batch * s.dim) return;
  const int b = (int)(i / s.dim), d = (int)(i % s.dim);
  const int n = live_len(s, b);
  for (int t = n; t < s.len; ++t) *gx.at(b, t, d) = *gg.at(b, t, d) = from_f32<T>(0.f);
  float c = grad_out ? grad_out[i] : 0.f;   // what the next position passes back
  for (int t = n - 1; t >= 0; --t) {
    float a, na;
    gates(to_f32(*g.at(b, t, d)), a, na);
    const float xv = to_f32(*x.at(b, t, d));
    const float before = t ? to_f32(*y.at(b, t - 1, d)) : state_in ? state_in[i] : 0.f;
    const float G = to_f32(*gy.at(b, t, d)) + c;
    *gx.at(b, t, d) = from_f32<T>(na * G);
    *gg.at(b, t, d) = from_f32<T>(a * na * (before - xv) * G);
    c = a * G;
  }
  if (grad_in) grad_in[i] = c;
}

template <class T>
__global__ void __launch_bounds__(256) k_scan_step(int64_t n, int32_t dim, const T* __restrict__ x, int64_t xs,
                                                   const T* __restrict__ g, int64_t gs,
                                                   const int64_t* __restrict__ rows, float* __restrict__ states,
                                                   int64_t num_rows, T* __restrict__ y, int64_t ys) {
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t row = rows[i];
    const bool live = row >= 0 && row < num_rows;
    for (int d = threadIdx.x; d < dim; d += blockDim.x) {
      float h = 0.f;
      if (live) {
        float a, na;
        gates(to_f32(g[i * gs + d]), a, na);
        h = a * states[row * dim + d] + na * to_f32(x[i * xs + d]);
        states[row * dim + d] = h;
      }
      y[i * ys + d] = from_f32<T>(h);
    }
  }
}

// A view is usable: pointer aligned to its element, strides not negative,
// and (outputs) no two elements at one place.
bool view_ok(const scan_view* v, int32_t dtype, int64_t batch, int64_t len, int64_t dim, bool output) {
  if (!v || v->batch_stride < 0 || v->time_stride < 0) return false;
  if (batch == 0 || len == 0) return true;
  if (!v->data || !aligned_to(v->data, dtype_size(dtype))) return false;
  if (!output) return true;
  if (len > 1 && v->time_stride < dim) return false;
  if (batch > 1 && v->batch_stride < dim) return false;
  return batch == 1 || len == 1 || v->batch_stride >= (len - 1) * v->time_stride + dim ||
         v->time_stride >= (batch - 1) * v->batch_stride + dim;
}

template <class T>
View<T> as_view(const scan_view* v) {
  return View<T>{(T*)v->data, v->batch_stride, v->time_stride};
}

bool call_ok(emb_scan h, int32_t batch, int32_t len, int32_t dtype) {
  return h && batch >= 0 && batch <= h->max_batch && len >= 0 && len <= h->max_len && dtype_size(dtype) != 0;
}

}  // namespace emb

using namespace emb;

extern "C" emb_status scan_create(int32_t dim, int32_t max_batch, int32_t max_len, emb_scan* out) {
  if (!out) return EMB_ERR_INVALID_ARG;
  *out = nullptr;
  if (dim < 1 || max_batch < 1 || max_len < 1) return EMB_ERR_INVALID_ARG;
  if (dim > 65536) return EMB_ERR_UNSUPPORTED;
  emb_scan_s* h = new (std::nothrow) emb_scan_s();
  if (!h) return EMB_ERR_OOM;
  h->dim = dim;
  h->max_batch = max_batch;
  h->max_len = max_len;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = dev_alloc((void**)&h->status_d, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemset(h->status_d, 0, sizeof(uint32_t));
  if (e != cudaSuccess) {
    dev_free(h->status_d);
    delete h;
    return cuda_status(e);
  }
  *out = h;
  return EMB_OK;
}

extern "C" emb_status scan_destroy(emb_scan h) {
  if (!h) return EMB_ERR_INVALID_ARG;
  const cudaError_t e = cudaDeviceSynchronize();
  dev_free(h->status_d);
  delete h;
  return cuda_status(e);
}

extern "C" emb_status scan_get_device_status(emb_scan h, void* stream) {
  if (!h) return EMB_ERR_INVALID_ARG;
  uint32_t st = 0;
  EMB_CUDA_TRY(cudaStreamSynchronize((cudaStream_t)stream));
  EMB_CUDA_TRY(cudaMemcpy(&st, h->status_d, sizeof(uint32_t), cudaMemcpyDeviceToHost));
  EMB_CUDA_TRY(cudaMemset(h->status_d, 0, sizeof(uint32_t)));
  return (emb_status)st;
}

extern "C" emb_status scan_forward(emb_scan h, int32_t batch, int32_t len, int32_t dtype, const scan_view* x,
                                   const scan_view* gate, const int32_t* offsets, const float* state_in,
                                   const scan_view* y, float* state_out, void* stream) {
  if (!call_ok(h, batch, len, dtype) || !view_ok(x, dtype, batch, len, h->dim, false) ||
      !view_ok(gate, dtype, batch, len, h->dim, false) || !view_ok(y, dtype, batch, len, h->dim, true))
    return EMB_ERR_INVALID_ARG;
  if (batch == 0) return EMB_OK;
  const ScanArgs s{batch, len, h->dim, offsets, h->status_d};
  const int64_t n = (int64_t)batch * h->dim, grid = (n + 127) / 128;
  if (grid >= (int64_t(1) << 31)) return EMB_ERR_UNSUPPORTED;
  with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_scan_fwd<T><<<(unsigned)grid, 128, 0, (cudaStream_t)stream>>>(s, as_view<const T>(x), as_view<const T>(gate),
                                                                   as_view<T>(y), state_in, state_out);
  });
  return cuda_status(cudaGetLastError());
}

extern "C" emb_status scan_backward(emb_scan h, int32_t batch, int32_t len, int32_t dtype, const scan_view* x,
                                    const scan_view* gate, const int32_t* offsets, const float* state_in,
                                    const scan_view* y, const scan_view* grad_y, const float* grad_state_out,
                                    const scan_view* grad_x, const scan_view* grad_gate, float* grad_state_in,
                                    void* stream) {
  if (!call_ok(h, batch, len, dtype) || !view_ok(x, dtype, batch, len, h->dim, false) ||
      !view_ok(gate, dtype, batch, len, h->dim, false) || !view_ok(y, dtype, batch, len, h->dim, false) ||
      !view_ok(grad_y, dtype, batch, len, h->dim, false) || !view_ok(grad_x, dtype, batch, len, h->dim, true) ||
      !view_ok(grad_gate, dtype, batch, len, h->dim, true))
    return EMB_ERR_INVALID_ARG;
  if (batch == 0) return EMB_OK;
  const ScanArgs s{batch, len, h->dim, offsets, h->status_d};
  const int64_t n = (int64_t)batch * h->dim, grid = (n + 127) / 128;
  if (grid >= (int64_t(1) << 31)) return EMB_ERR_UNSUPPORTED;
  with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_scan_bwd<T><<<(unsigned)grid, 128, 0, (cudaStream_t)stream>>>(
        s, as_view<const T>(x), as_view<const T>(gate), as_view<const T>(y), as_view<const T>(grad_y), state_in,
        grad_state_out, as_view<T>(grad_x), as_view<T>(grad_gate), grad_state_in);
  });
  return cuda_status(cudaGetLastError());
}

extern "C" emb_status scan_step(int64_t n, int32_t dim, int32_t dtype, const void* x, int64_t x_stride,
                                const void* gate, int64_t gate_stride, const int64_t* rows, float* states,
                                int64_t num_rows, void* y, int64_t y_stride, void* stream) {
  if (n < 0 || dim < 1 || dtype_size(dtype) == 0 || num_rows < 0 || x_stride < 0 || gate_stride < 0)
    return EMB_ERR_INVALID_ARG;
  if (n == 0) return EMB_OK;
  const int size = dtype_size(dtype);
  if (!x || !gate || !rows || !y || (num_rows > 0 && !states) || !aligned_to(x, size) || !aligned_to(gate, size) ||
      !aligned_to(y, size) || !aligned_to(states, 4) || !aligned_to(rows, 8) || (n > 1 && y_stride < dim))
    return EMB_ERR_INVALID_ARG;
  if (dim > 65536) return EMB_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)(n < (1 << 20) ? n : (1 << 20));
  with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_scan_step<T><<<grid, 256, 0, (cudaStream_t)stream>>>(n, dim, (const T*)x, x_stride, (const T*)gate, gate_stride,
                                                         rows, states, num_rows, (T*)y, y_stride);
  });
  return cuda_status(cudaGetLastError());
}
