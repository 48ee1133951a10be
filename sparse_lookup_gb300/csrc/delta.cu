// delta.cu -- the gated delta rule: handle, checks of arguments, and one position at
// a time (delta_* in emb.h).
#include <new>

#include "delta.cuh"

namespace emb {

constexpr int kStepThreads = 256;

struct StepArgs {
  int32_t heads, share, key_dim, value_dim;
  float scale;
  const int64_t* rows;
  int64_t num_rows;
  float* states;
  DView<const float> decay, beta;
};

// CTAs of it on an SM, as many as the registers leave room for: 4096 sessions of 8 heads of
// 128 x 128 take 880 us with one and 733 with two, 4 heads of 64 x 64 145 with three, 102 with four.
constexpr int step_ctas(int v, int r) { return v * r <= 8 ? 6 : v * r <= 16 ? 4 : v * r <= 32 ? 3 : v > 1 ? 2 : 1; }

// One position of a session's head: with S' = exp(g) S,
//   y = scale (S'^T q + beta <k, q> e),  S = S' + beta k e^T,  e = v - S'^T k
// so both products with the state are ready after one pass over it, which stays in
// registers until it is written back.  A thread holds V neighbouring channels of R
// rows; the rows' partial sums meet in shared memory.  Bound by memory where there are
// many sessions (4096 of 8 heads of 128 x 128 bf16 5.9 TB/s, of 4 heads of 64 x 64 5.4), by a
// CTA's two barriers where heads are small (20000 of 2 heads of 32 x 32 2.1), by the launch
// where sessions are few (192 of 4 heads of 64 x 64: 6 us).
template <class T, int V, int R>
__global__ void __launch_bounds__(kStepThreads, step_ctas(V, R)) k_delta_step(StepArgs a, DView<const T> q, DView<const T> k,
                                                             DView<const T> v, DView<T> y, int log_cols) {
  __shared__ float ks[128], qs[128], kq[kStepThreads / 32];
  __shared__ alignas(16) float part[2][kStepThreads * V];
  const int i = blockIdx.x / a.heads, h = blockIdx.x % a.heads, hk = h / a.share;
  const int64_t row = a.rows[i];
  const bool on = row >= 0 && row < a.num_rows;
  T* out = y.data + i * y.batch + h * y.head;
  if (!on) {
    for (int e = threadIdx.x; e < a.value_dim; e += kStepThreads) out[e] = from_f32<T>(0.f);
    return;
  }
  const int cols = 1 << log_cols, group = threadIdx.x >> log_cols, groups = kStepThreads >> log_cols;
  const int c = (threadIdx.x & (cols - 1)) * V;
  float* S = a.states + (row * a.heads + h) * a.key_dim * a.value_dim + c;
  Vec<float, V> s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int d = group + r * groups;
    if (d < a.key_dim && c < a.value_dim) {
      s[r] = load_vec<float, V>(S + (int64_t)d * a.value_dim);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u) s[r].e[u] = 0.f;
    }
  }
  float both = 0.f;
  if (threadIdx.x < 128) {
    const bool in = (int)threadIdx.x < a.key_dim;
    const float kx = in ? to_f32(k.data[i * k.batch + hk * k.head + threadIdx.x]) : 0.f;
    const float qx = in ? to_f32(q.data[i * q.batch + hk * q.head + threadIdx.x]) : 0.f;
    ks[threadIdx.x] = kx, qs[threadIdx.x] = qx;
    both = kx * qx;
  }
  for (int o = 16; o > 0; o >>= 1) both += __shfl_xor_sync(kFull, both, o);
  if ((threadIdx.x & 31) == 0) kq[threadIdx.x >> 5] = both;
  const float decay = expf(a.decay.data[i * a.decay.batch + h * a.decay.head]);
  const float beta = a.beta.data[i * a.beta.batch + h * a.beta.head];
  float vs[V];
#pragma unroll
  for (int u = 0; u < V; ++u)
    vs[u] = c + u < a.value_dim ? to_f32(v.data[i * v.batch + h * v.head + c + u]) : 0.f;
  __syncthreads();
  float sk[V], sq[V];
#pragma unroll
  for (int u = 0; u < V; ++u) sk[u] = sq[u] = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int d = group + r * groups;
    const float kx = d < 128 ? ks[d] : 0.f, qx = d < 128 ? qs[d] : 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      s[r].e[u] = decay == 0.f ? 0.f : s[r].e[u] * decay;
      sk[u] += s[r].e[u] * kx, sq[u] += s[r].e[u] * qx;
    }
  }
  // a warp's rows first
  for (int o = cols; o < 32; o <<= 1)
#pragma unroll
    for (int u = 0; u < V; ++u)
      sk[u] += __shfl_xor_sync(kFull, sk[u], o), sq[u] += __shfl_xor_sync(kFull, sq[u], o);
  const int sums = cols < 32 ? kStepThreads / 32 : groups, mine = cols < 32 ? threadIdx.x >> 5 : group;
  if (cols >= 32 || (int)(threadIdx.x & 31) < cols)
#pragma unroll
    for (int u = 0; u < V; ++u) part[0][mine * cols * V + c + u] = sk[u], part[1][mine * cols * V + c + u] = sq[u];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < V; ++u) sk[u] = sq[u] = 0.f;
  for (int w = 0; w < sums; ++w)
#pragma unroll
    for (int u = 0; u < V; ++u) sk[u] += part[0][w * cols * V + c + u], sq[u] += part[1][w * cols * V + c + u];
  both = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) both += kq[w];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    vs[u] = beta * (vs[u] - sk[u]);
    sq[u] = a.scale * (sq[u] + vs[u] * both);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int d = group + r * groups;
    if (d >= a.key_dim || c >= a.value_dim) continue;
#pragma unroll
    for (int u = 0; u < V; ++u) s[r].e[u] += ks[d] * vs[u];
    store_vec(S + (int64_t)d * a.value_dim, s[r]);
  }
  if (group == 0)
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (c + u < a.value_dim) out[c + u] = from_f32<T>(sq[u]);
}

namespace {

int dk_of(int key_dim) { return key_dim <= 32 ? 32 : key_dim <= 64 ? 64 : 128; }

bool delta_view_ok(const delta_view* v, int size, int64_t batch, int64_t len, int64_t heads, int64_t dim, bool out) {
  if (!v || v->batch_stride < 0 || v->time_stride < 0 || v->head_stride < 0) return false;
  if (batch == 0 || len == 0) return true;
  if (!v->data || !aligned_to(v->data, size)) return false;
  if (!out) return true;
  // heads within positions within entries, each behind the one before
  const int64_t pos = (heads - 1) * v->head_stride + dim, entry = (len - 1) * v->time_stride + pos;
  return (heads == 1 || v->head_stride >= dim) && (len == 1 || v->time_stride >= pos) &&
         (batch == 1 || v->batch_stride >= entry);
}

// Whether rows of `dim` elements move in accesses of `n`.
bool whole_pieces(int size, int64_t dim, std::initializer_list<const delta_view*> views, int n, int of) {
  if (dim % of) return false;
  for (const delta_view* v : views)
    if (v->batch_stride % n || v->time_stride % n || v->head_stride % n || !aligned_to(v->data, n * size)) return false;
  return true;
}

bool delta_ok(emb_delta h, int32_t batch, int32_t len, int32_t dtype, const int32_t* offsets, double scale) {
  return h && batch >= 0 && batch <= h->max_batch && len >= 0 && len <= h->max_len && on_device(h->device) &&
         dtype_size(dtype) != 0 && aligned_to(offsets, 4) && scale - scale == 0.0;
}

DeltaArgs delta_args(emb_delta h, int32_t batch, int32_t len, const int32_t* offsets, double scale,
                     const float* state_in) {
  DeltaArgs a = {};
  a.batch = batch, a.len = len, a.heads = h->heads, a.share = h->heads / h->key_heads;
  a.key_dim = h->key_dim, a.value_dim = h->value_dim;
  a.chunks = (len + kChunk - 1) / kChunk;
  a.parts = 1;
  a.warps = (h->value_dim + 15) / 16;
  a.scale = (float)scale;
  a.offsets = offsets;
  a.state_in = state_in;
  a.work = {h->record, {h->s[0], h->s[1], h->s[2]}, {h->ds[0], h->ds[1], h->ds[2]}, h->e, h->dz, h->sums, h->along,
            h->totals, (int64_t)batch * h->heads * a.chunks, h->effect, h->between};
  return a;
}

cudaError_t run(emb_delta h, const DeltaArgs& a, const DeltaViews& w, int32_t dtype, bool backward, void* stream) {
  return with_element(dtype, [&](auto* t) {
    return run_delta<std::remove_pointer_t<decltype(t)>>(h, a, w, backward, (cudaStream_t)stream);
  });
}

void delta_free(emb_delta h) {
  dev_free(h->record);
  dev_free(h->order);
  for (uint4* p : h->s) dev_free(p);
  for (uint4* p : h->ds) dev_free(p);
  dev_free(h->e);
  dev_free(h->dz);
  dev_free(h->sums);
  dev_free(h->along);
  dev_free(h->totals);
  dev_free(h->effect);
  dev_free(h->between);
  delete h;
}

}  // namespace

}  // namespace emb

using namespace emb;

extern "C" emb_status delta_create(int32_t key_dim, int32_t value_dim, int32_t heads, int32_t key_heads,
                                   int32_t max_batch, int32_t max_len, int32_t training, emb_delta* out) {
  if (!out) return EMB_ERR_INVALID_ARG;
  *out = nullptr;
  if (key_dim < 1 || value_dim < 1 || heads < 1 || key_heads < 1 || heads % key_heads || max_batch < 1 || max_len < 1)
    return EMB_ERR_INVALID_ARG;
  if (key_dim > 128 || value_dim > 128 || heads > 65536 || max_len > (1 << 30) ||
      (int64_t)max_batch * heads >= (int64_t(1) << 27) ||
      (int64_t)max_batch * heads * (max_len / kChunk + 1) >= (int64_t(1) << 30))
    return EMB_ERR_UNSUPPORTED;
  emb_delta_s* h = new (std::nothrow) emb_delta_s();
  if (!h) return EMB_ERR_OOM;
  h->key_dim = key_dim, h->value_dim = value_dim, h->heads = heads, h->key_heads = key_heads;
  h->max_batch = max_batch, h->max_len = max_len, h->training = training != 0;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
  const int64_t all = (int64_t)max_batch * heads, chunks = ((int64_t)max_len + kChunk - 1) / kChunk;
  if (e == cudaSuccess) e = dev_alloc((void**)&h->record, all * chunks * Record::bytes);
  if (e == cudaSuccess) e = dev_alloc((void**)&h->order, sizeof(int32_t) * kMostOrdered);
  const int64_t W = (value_dim + 15) / 16, dk = dk_of(key_dim);
  if (chunks >= kLeastChunks && e == cudaSuccess) {
    // calls of a few heads are cut into segments, one an SM: an effect forward and one backward
    h->max_pairs = h->sm_count;
    e = dev_alloc((void**)&h->effect, h->max_pairs * (2 * W * 16 + dk) * dk * sizeof(float));
    if (e == cudaSuccess) e = dev_alloc((void**)&h->between, h->max_pairs * W * 16 * dk * sizeof(float));
  }
  if (training) {
    const int64_t state = W * (dk / 16) * 32 * sizeof(uint4), each = W * 4 * 32 * sizeof(float4);
    for (uint4*& p : h->s)
      if (e == cudaSuccess) e = dev_alloc((void**)&p, all * (chunks + 1) * state);
    for (uint4*& p : h->ds)
      if (e == cudaSuccess) e = dev_alloc((void**)&p, all * chunks * state);
    if (e == cudaSuccess) e = dev_alloc((void**)&h->e, all * chunks * each);
    if (e == cudaSuccess) e = dev_alloc((void**)&h->dz, all * chunks * each);
    if (e == cudaSuccess) e = dev_alloc((void**)&h->sums, 3 * W * all * chunks * kChunk * sizeof(float));
    if (e == cudaSuccess) e = dev_alloc((void**)&h->along, W * all * (chunks + 1) * sizeof(float));
    if (e == cudaSuccess) e = dev_alloc((void**)&h->totals, W * all * chunks * sizeof(float));
  }
  if (e != cudaSuccess) {
    delta_free(h);
    return cuda_status(e);
  }
  *out = h;
  return EMB_OK;
}

extern "C" emb_status delta_destroy(emb_delta h) {
  if (!h) return EMB_ERR_INVALID_ARG;
  const cudaError_t e = cudaDeviceSynchronize();
  delta_free(h);
  return cuda_status(e);
}

extern "C" emb_status delta_forward(emb_delta h, int32_t batch, int32_t len, int32_t dtype, const delta_view* q,
                                    const delta_view* k, const delta_view* v, const delta_view* decay,
                                    const delta_view* beta, const int32_t* offsets, double scale,
                                    const float* state_in, const delta_view* y, float* state_out, void* stream) {
  if (!delta_ok(h, batch, len, dtype, offsets, scale)) return EMB_ERR_INVALID_ARG;
  const int size = dtype_size(dtype), H = h->heads, J = h->key_heads, N = h->key_dim, D = h->value_dim;
  if (!delta_view_ok(q, size, batch, len, J, N, false) || !delta_view_ok(k, size, batch, len, J, N, false) ||
      !delta_view_ok(v, size, batch, len, H, D, false) || !delta_view_ok(y, size, batch, len, H, D, true) ||
      !delta_view_ok(decay, 4, batch, len, H, 1, false) || !delta_view_ok(beta, 4, batch, len, H, 1, false) ||
      !aligned_to(state_in, 4) || !aligned_to(state_out, 4))
    return EMB_ERR_INVALID_ARG;
  if (batch == 0) return EMB_OK;
  DeltaArgs a = delta_args(h, batch, len, offsets, scale, state_in);
  a.state_out = state_out;
  a.decay = dview<const float>(decay), a.beta = dview<const float>(beta);
  a.wide_qk = whole_pieces(size, N, {q, k}, 16 / size, 8);
  a.wide_v = whole_pieces(size, D, {v}, 16 / size, 8);
  a.wide_y = whole_pieces(size, D, {y}, 16 / size, 8);
  DeltaViews w = {};
  w.q = q, w.k = k, w.v = v, w.y = y;
  return cuda_status(run(h, a, w, dtype, false, stream));
}

extern "C" emb_status delta_backward(emb_delta h, int32_t batch, int32_t len, int32_t dtype, const delta_view* q,
                                     const delta_view* k, const delta_view* v, const delta_view* decay,
                                     const delta_view* beta, const int32_t* offsets, double scale,
                                     const float* state_in, const delta_view* grad_y, const float* grad_state_out,
                                     const delta_view* grad_q, const delta_view* grad_k, const delta_view* grad_v,
                                     const delta_view* grad_decay, const delta_view* grad_beta,
                                     float* grad_state_in, void* stream) {
  if (!delta_ok(h, batch, len, dtype, offsets, scale)) return EMB_ERR_INVALID_ARG;
  const int size = dtype_size(dtype), H = h->heads, J = h->key_heads, N = h->key_dim, D = h->value_dim;
  if (!delta_view_ok(q, size, batch, len, J, N, false) || !delta_view_ok(k, size, batch, len, J, N, false) ||
      !delta_view_ok(v, size, batch, len, H, D, false) || !delta_view_ok(grad_y, size, batch, len, H, D, false) ||
      !delta_view_ok(decay, 4, batch, len, H, 1, false) || !delta_view_ok(beta, 4, batch, len, H, 1, false) ||
      !delta_view_ok(grad_q, size, batch, len, J, N, true) || !delta_view_ok(grad_k, size, batch, len, J, N, true) ||
      !delta_view_ok(grad_v, size, batch, len, H, D, true) ||
      !delta_view_ok(grad_decay, 4, batch, len, H, 1, true) || !delta_view_ok(grad_beta, 4, batch, len, H, 1, true) ||
      !aligned_to(state_in, 4) || !aligned_to(grad_state_out, 4) || !aligned_to(grad_state_in, 4))
    return EMB_ERR_INVALID_ARG;
  if (!h->training) return EMB_ERR_UNSUPPORTED;
  if (batch == 0) return EMB_OK;
  DeltaArgs a = delta_args(h, batch, len, offsets, scale, state_in);
  a.grad_last = grad_state_out, a.grad_state = grad_state_in;
  a.decay = dview<const float>(decay), a.beta = dview<const float>(beta);
  a.grad_decay = dview<float>(grad_decay), a.grad_beta = dview<float>(grad_beta);
  a.wide_qk = whole_pieces(size, N, {q, k}, 16 / size, 8);
  a.wide_v = whole_pieces(size, D, {v, grad_y}, 16 / size, 8);
  a.wide_y = whole_pieces(size, D, {grad_v}, 16 / size, 8);
  a.wide_gy = whole_pieces(size, N, {grad_q, grad_k}, 16 / size, 8);
  DeltaViews w = {};
  w.q = q, w.k = k, w.v = v, w.gy = grad_y, w.gq = grad_q, w.gk = grad_k, w.gv = grad_v;
  return cuda_status(run(h, a, w, dtype, true, stream));
}

extern "C" emb_status delta_step(int64_t n, int32_t key_dim, int32_t value_dim, int32_t heads, int32_t key_heads,
                                 int32_t dtype, const delta_view* q, const delta_view* k, const delta_view* v,
                                 const delta_view* decay, const delta_view* beta, double scale, const int64_t* rows,
                                 float* states, int64_t num_rows, const delta_view* y, void* stream) {
  if (n < 0 || num_rows < 0 || key_dim < 1 || value_dim < 1 || heads < 1 || key_heads < 1 || heads % key_heads ||
      dtype_size(dtype) == 0 || !(scale - scale == 0.0))
    return EMB_ERR_INVALID_ARG;
  const int size = dtype_size(dtype);
  if (!delta_view_ok(q, size, n, 1, key_heads, key_dim, false) ||
      !delta_view_ok(k, size, n, 1, key_heads, key_dim, false) ||
      !delta_view_ok(v, size, n, 1, heads, value_dim, false) || !delta_view_ok(y, size, n, 1, heads, value_dim, true) ||
      !delta_view_ok(decay, 4, n, 1, heads, 1, false) || !delta_view_ok(beta, 4, n, 1, heads, 1, false) ||
      (n > 0 && (!rows || (num_rows > 0 && !states))) || !aligned_to(rows, 8) || !aligned_to(states, 4))
    return EMB_ERR_INVALID_ARG;
  if (key_dim > 128 || value_dim > 128 || heads > 65536 || n >= (int64_t(1) << 31) || n * heads >= (int64_t(1) << 31))
    return EMB_ERR_UNSUPPORTED;
  if (n == 0) return EMB_OK;
  const StepArgs a{heads, heads / key_heads, key_dim, value_dim, (float)scale, rows, num_rows, states,
                   dview<const float>(decay), dview<const float>(beta)};
  const int width = value_dim % 4 == 0 && aligned16(states) ? 4 : value_dim % 2 == 0 && aligned_to(states, 8) ? 2 : 1;
  int log_cols = 0;
  while ((width << log_cols) < value_dim) ++log_cols;
  const int groups = kStepThreads >> log_cols, need = (key_dim + groups - 1) / groups;
  return cuda_status(with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const auto kernel = width == 4   ? (need <= 2    ? k_delta_step<T, 4, 2>
                                        : need <= 4  ? k_delta_step<T, 4, 4>
                                        : need <= 8  ? k_delta_step<T, 4, 8>
                                                     : k_delta_step<T, 4, 16>)
                        : width == 2 ? (need <= 8    ? k_delta_step<T, 2, 8>
                                        : need <= 16 ? k_delta_step<T, 2, 16>
                                                     : k_delta_step<T, 2, 32>)
                                     : (need <= 8    ? k_delta_step<T, 1, 8>
                                        : need <= 16 ? k_delta_step<T, 1, 16>
                                        : need <= 32 ? k_delta_step<T, 1, 32>
                                                     : k_delta_step<T, 1, 64>);
    kernel<<<(unsigned)(n * heads), kStepThreads, 0, (cudaStream_t)stream>>>(
        a, dview<const T>(q), dview<const T>(k), dview<const T>(v), dview<T>(y), log_cols);
    return cudaGetLastError();
  }));
}
