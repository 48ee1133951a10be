// norm.cu -- layer norm over rows, forward and backward with the gradients of
// weight and bias (norm_* in emb.h).
#include <new>

#include "rows.cuh"

struct emb_norm_s {
  int32_t dim = 0;
  int sm_count = 0, device = 0;
  float* part_d = nullptr;   // [CTAs][2][dim] sums of dy xh and of dy over a CTA's rows
};

namespace emb {

constexpr int kNormThreads = 128;      // of a CTA whose groups are within a warp
constexpr int kNormWide = 512;         // threads of a row at most
constexpr int kNormCtas = 4;           // CTAs of kNormThreads on an SM at most
constexpr int kNormMaxDim = 16384;
constexpr int kSumCols = 16, kSumRows = 32;   // columns of the last reduction's CTA, and partial rows side by side

// Rows are (b, t) of a [batch, len] array; a plain matrix is one batch entry.
struct NormRows {
  int64_t n;                // batch * len
  int64_t len;
  DivMagic by_len;
  const int32_t* offsets;   // NULL: every position is live
  int32_t dim, vecs;
  float eps;
};
template <class T>
struct NormView {
  T* data;
  int64_t batch, time;
};

struct Place {
  int64_t b, t;
  bool live;
};
__device__ __forceinline__ Place place_of(const NormRows& a, int64_t r) {
  Place p{0, r, true};
  if (a.len != a.n) {
    p.b = (int64_t)div_magic((uint64_t)r, a.by_len);
    p.t = r - p.b * a.len;
  }
  if (a.offsets) {
    const int64_t n = (int64_t)a.offsets[p.b + 1] - a.offsets[p.b];
    p.live = p.t < n;
  }
  return p;
}
template <class T>
__device__ __forceinline__ T* row_of(const NormView<T>& v, const Place& p) {
  return v.data + p.b * v.batch + p.t * v.time;
}

// The sum over a row's group of lanes: within a warp, or over the CTA.
template <bool WIDE>
struct RowSum {
  float2* buf;   // [2][warps], used in turn so that one barrier a sum is enough
  int lanes, turn;
  __device__ __forceinline__ float2 operator()(float2 x) {
    const int most = WIDE ? 32 : lanes;
    for (int o = 1; o < most; o <<= 1) {
      x.x += __shfl_xor_sync(kFull, x.x, o);
      x.y += __shfl_xor_sync(kFull, x.y, o);
    }
    if constexpr (WIDE) {
      const int warps = blockDim.x >> 5;
      float2* at = buf + turn * (kNormWide / 32);
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = x;
      __syncthreads();
      x = at[0];
      for (int w = 1; w < warps; ++w) x.x += at[w].x, x.y += at[w].y;
    }
    return x;
  }
};

// Whether a row's accesses are started a round early: not where a thread of a wide
// CTA, or of the backward, holds 32 elements: the registers are worth more warps
// (131072 x 1024 bf16 backward 200 us without, 290 with).
template <int V, int N, bool WIDE>
constexpr bool kAhead = !(WIDE && V * N >= 32);
template <int V, int N>
constexpr bool kBwdAhead = V * N < 32;

// CTAs of a backward on an SM, as many as its registers allow: a fourth would run after
// them, alone (1024 x 1000 x 64 fp32 141 us with four, 101 with three).
constexpr int kBwdCtas = 3;

// One row in a lane: N accesses of V elements, `lanes` accesses apart.  Arithmetic is in
// pairs: neighbours of an access, or of single elements two accesses.
template <class T, int V, int N>
struct RowPart {
  static constexpr int per = V == 1 && N > 1 ? 2 : 1, groups = N / per, pairs = V > 1 ? V / 2 : 1;
  Vec<T, V> v[N];
  __device__ __forceinline__ void load(const T* row, int sub, int lanes, int vecs, bool live) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = sub + i * lanes;
      if (live && j < vecs) {
        v[i] = load_vec<T, V>(row + (int64_t)j * V);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[i].e[e] = from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ Pairs<V> at(int i) const {
    Pairs<V> f = pairs_of(v[i * per]);
    if constexpr (per == 2) f.p[0].y = to_f32(v[i * per + 1].e[0]);
    return f;
  }
};
// Such a group's results to its places, the first of which is access j.
template <class T, int V, int N>
__device__ __forceinline__ void store_group(T* row, const Pairs<V>& f, int j, int lanes, int vecs) {
  store_vec(row + (int64_t)j * V, vec_of<T, V>(f));
  if constexpr (RowPart<T, V, N>::per == 2)
    if (j + lanes < vecs) row[j + lanes] = from_f32<T>(f.p[0].y);
}
// Columns of pair e of such a group; the second is there where it is below `dim`.
template <int V>
__device__ __forceinline__ int2 columns_of(int j, int e, int lanes) {
  return V == 1 ? make_int2(j, j + lanes) : make_int2(j * V + 2 * e, j * V + 2 * e + 1);
}

template <class W>
__device__ __forceinline__ float weight_at(const W* w, int32_t c, float none) {
  return w ? to_f32(w[c]) : none;
}

// A weight in shared memory: of accesses of four and more in groups of four, the groups
// of neighbouring accesses side by side, so that lanes read 16 bytes each without
// conflicts (read one by one, 131072 x 1024 bf16 took 240 us where it takes 104).
template <int V>
__device__ __forceinline__ int place_in(int c, int vecs) {
  if constexpr (V < 4) return c;
  const int j = c / V, e = c % V;
  return ((e >> 2) * vecs + j) * 4 + (e & 3);
}
template <int V>
__device__ __forceinline__ Pairs<V> weights_of(const float* w, int j, int lanes, int vecs) {
  Pairs<V> o;
  if constexpr (V >= 4) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 x = *reinterpret_cast<const float4*>(w + ((e >> 2) * vecs + j) * 4);
      o.p[e / 2] = make_float2(x.x, x.y), o.p[e / 2 + 1] = make_float2(x.z, x.w);
    }
  } else {
    const int second = V > 1 ? j * V + 1 : j + lanes;
    o.p[0] = make_float2(w[j * V], V > 1 || second < vecs ? w[second] : 0.f);
  }
  return o;
}

// Registers are kept to two CTAs of 512 threads an SM where a thread has 16 elements in
// pairs or more (19550 x 2046 bf16 114 us without that, 68 with; single elements 72 and 98).
// y = (x - mean) rstd w + b.  A row stays in its lanes' registers, so x is
// read once although mean and deviations need a pass each; the next row's
// accesses are in flight meanwhile.  131072 x 1024 bf16 104 us (5.2 TB/s), 1024 x
// 1000 x 64 fp32 with lengths 200 .. 1000 70 us (6.0 TB/s).
template <class T, class W, int V, int N, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kNormWide : kNormThreads, !WIDE ? kNormCtas : V > 1 && V * N < 32 ? 2 : 1)
    k_norm_fwd(NormRows a, NormView<const T> x, const W* __restrict__ w, const W* __restrict__ b, NormView<T> y,
               float2* __restrict__ stats, int glog) {
  extern __shared__ float held[];   // [2][dim] weight, bias
  __shared__ float2 sums[2 * (kNormWide / 32)];
  float *ws = held, *bs = held + a.dim;
  for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
    ws[place_in<V>(c, a.vecs)] = weight_at(w, c, 1.f);
    bs[place_in<V>(c, a.vecs)] = weight_at(b, c, 0.f);
  }
  __syncthreads();
  using Part = RowPart<T, V, N>;
  constexpr int P = Part::pairs;
  const int L = WIDE ? blockDim.x : 1 << glog, sub = WIDE ? threadIdx.x : threadIdx.x & (L - 1);
  const int per = WIDE ? 1 : kNormThreads >> glog, mine = WIDE ? 0 : threadIdx.x >> glog;
  RowSum<WIDE> sum{sums, L, 0};
  const float inv = 1.f / (float)a.dim;
  const int64_t step = (int64_t)gridDim.x * per;
  // every lane of a warp makes the same number of rounds: the sums are joint
  int64_t r = (int64_t)blockIdx.x * per + mine;
  const int64_t rounds = (a.n - (int64_t)blockIdx.x * per + step - 1) / step;
  Part next;
  Place p = r < a.n ? place_of(a, r) : Place{0, 0, false};
  if constexpr (kAhead<V, N, WIDE>) next.load(row_of(x, p), sub, L, a.vecs, p.live);
  for (int64_t k = 0; k < rounds; ++k, r += step) {
    if constexpr (!kAhead<V, N, WIDE>) next.load(row_of(x, p), sub, L, a.vecs, p.live);
    const Part now = next;
    const Place q = p;
    const int64_t s = r + step;
    p = s < a.n ? place_of(a, s) : Place{0, 0, false};
    if constexpr (kAhead<V, N, WIDE>) next.load(row_of(x, p), sub, L, a.vecs, p.live);
    float2 m = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < Part::groups; ++i) {
      const Pairs<V> f = now.at(i);
#pragma unroll
      for (int e = 0; e < P; ++e) m = __fadd2_rn(m, f.p[e]);
    }
    m = sum(m);
    const float mean = (m.x + m.y) * inv;
    float2 d = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < Part::groups; ++i) {
      const int j = sub + i * Part::per * L;
      if (j >= a.vecs) continue;
      const Pairs<V> f = now.at(i);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 u = __fadd2_rn(f.p[e], make_float2(-mean, V > 1 || j + L < a.vecs ? -mean : 0.f));
        d = __ffma2_rn(u, u, d);
      }
    }
    d = sum(d);
    const float rstd = rsqrtf((d.x + d.y) * inv + a.eps);
    if (r >= a.n) continue;
    if (stats && sub == 0) stats[r] = q.live ? make_float2(mean, rstd) : make_float2(0.f, 0.f);
    T* to = row_of(y, q);
#pragma unroll
    for (int i = 0; i < Part::groups; ++i) {
      const int j = sub + i * Part::per * L;
      if (j >= a.vecs) continue;
      Pairs<V> f = now.at(i);
      const Pairs<V> wj = weights_of<V>(ws, j, L, a.vecs), bj = weights_of<V>(bs, j, L, a.vecs);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 h = __fmul2_rn(__fadd2_rn(f.p[e], make_float2(-mean, -mean)), make_float2(rstd, rstd));
        const float2 o = __ffma2_rn(h, wj.p[e], bj.p[e]);
        f.p[e] = q.live ? o : make_float2(0.f, 0.f);
      }
      store_group<T, V, N>(to, f, j, L, a.vecs);
    }
  }
}

// dx = rstd (g - mean(g) - xh mean(g xh)), g = dy w; the sums of dy xh and dy
// over a CTA's rows in registers, lane by lane, joined at the end in a fixed
// order.  131072 x 1024 bf16 190 us (4.2 TB/s): 900 instructions a row on half of the
// issue slots, with the 12 warps an SM that 32 channels' sums in a lane leave room for.
// 1024 x 1000 x 64 fp32 98 us.
template <class T, class W, int V, int N, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kNormWide : kNormThreads, WIDE ? 1 : kBwdCtas)
    k_norm_bwd(NormRows a, NormView<const T> x, NormView<const T> dy, const float2* __restrict__ stats,
               const W* __restrict__ w, NormView<T> dx, float* __restrict__ part, int glog) {
  extern __shared__ float held[];   // [dim] weight; at the end [2][dim] sums
  __shared__ float2 sums[2 * (kNormWide / 32)];
  for (int c = threadIdx.x; c < a.dim; c += blockDim.x) held[place_in<V>(c, a.vecs)] = weight_at(w, c, 1.f);
  __syncthreads();
  using Part = RowPart<T, V, N>;
  constexpr int P = Part::pairs;
  const int L = WIDE ? blockDim.x : 1 << glog, sub = WIDE ? threadIdx.x : threadIdx.x & (L - 1);
  const int per = WIDE ? 1 : kNormThreads >> glog, mine = WIDE ? 0 : threadIdx.x >> glog;
  RowSum<WIDE> sum{sums, L, 0};
  const float inv = 1.f / (float)a.dim;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t r = (int64_t)blockIdx.x * per + mine;
  const int64_t rounds = (a.n - (int64_t)blockIdx.x * per + step - 1) / step;
  float2 gw[Part::groups][P], gb[Part::groups][P];
#pragma unroll
  for (int i = 0; i < Part::groups; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) gw[i][e] = gb[i][e] = make_float2(0.f, 0.f);
  Part nx, ng;
  Place p = r < a.n ? place_of(a, r) : Place{0, 0, false};
  float2 ns = p.live ? stats[r] : make_float2(0.f, 0.f);
  const auto load = [&] {
    nx.load(row_of(x, p), sub, L, a.vecs, p.live);
    ng.load(row_of(dy, p), sub, L, a.vecs, p.live);
  };
  if constexpr (kBwdAhead<V, N>) load();
  for (int64_t k = 0; k < rounds; ++k, r += step) {
    if constexpr (!kBwdAhead<V, N>) load();
    const Part xv = nx, gv = ng;
    const Place q = p;
    const float2 st = ns;
    const int64_t s = r + step;
    p = s < a.n ? place_of(a, s) : Place{0, 0, false};
    ns = p.live ? stats[s] : make_float2(0.f, 0.f);
    if constexpr (kBwdAhead<V, N>) load();
    // sums of g and of g xh, in pairs: the row is bound by the instructions it takes
    float2 m1 = make_float2(0.f, 0.f), m2 = m1;
    const float2 minus_mean = make_float2(-st.x, -st.x), rstd = make_float2(st.y, st.y);
#pragma unroll
    for (int i = 0; i < Part::groups; ++i) {
      const int j = sub + i * Part::per * L;
      if (j >= a.vecs) continue;
      const Pairs<V> f = xv.at(i), g = gv.at(i), wj = weights_of<V>(held, j, L, a.vecs);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 h = __fmul2_rn(__fadd2_rn(f.p[e], minus_mean), rstd), o = __fmul2_rn(g.p[e], wj.p[e]);
        m1 = __fadd2_rn(m1, o), m2 = __ffma2_rn(o, h, m2);
        gw[i][e] = __ffma2_rn(g.p[e], h, gw[i][e]), gb[i][e] = __fadd2_rn(gb[i][e], g.p[e]);
      }
    }
    float2 m = make_float2(m1.x + m1.y, m2.x + m2.y);
    m = sum(m);
    m.x *= inv, m.y *= inv;
    if (r >= a.n) continue;
    T* to = row_of(dx, q);
    const float2 scale1 = make_float2(-m.x * st.y, -m.x * st.y), scale2 = make_float2(-m.y * st.y, -m.y * st.y);
#pragma unroll
    for (int i = 0; i < Part::groups; ++i) {
      const int j = sub + i * Part::per * L;
      if (j >= a.vecs) continue;
      Pairs<V> f = xv.at(i), g = gv.at(i), wj = weights_of<V>(held, j, L, a.vecs);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 h = __fmul2_rn(__fadd2_rn(f.p[e], minus_mean), rstd), o = __fmul2_rn(g.p[e], wj.p[e]);
        const float2 x = __ffma2_rn(h, scale2, __ffma2_rn(o, rstd, scale1));
        f.p[e] = q.live ? x : make_float2(0.f, 0.f);
      }
      store_group<T, V, N>(to, f, j, L, a.vecs);
    }
  }
  pdl_trigger();
  if (!part) return;
  // a warp's groups first, then warp after warp in shared memory
  part += (int64_t)blockIdx.x * 2 * a.dim;
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < Part::groups; ++i)
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const int j = sub + i * Part::per * L;
        if (j >= a.vecs) continue;
        const int2 c = columns_of<V>(j, e, L);
        part[c.x] = gw[i][e].x, part[a.dim + c.x] = gb[i][e].x;
        if (c.y < a.dim) part[c.y] = gw[i][e].y, part[a.dim + c.y] = gb[i][e].y;
      }
  } else {
    for (int o = L; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < Part::groups; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          gw[i][e].x += __shfl_xor_sync(kFull, gw[i][e].x, o);
          gb[i][e].x += __shfl_xor_sync(kFull, gb[i][e].x, o);
          if (V * N > 1) gw[i][e].y += __shfl_xor_sync(kFull, gw[i][e].y, o);
          if (V * N > 1) gb[i][e].y += __shfl_xor_sync(kFull, gb[i][e].y, o);
        }
    for (int u = 0; u < kNormThreads / 32; ++u) {
      __syncthreads();
      if ((int)(threadIdx.x >> 5) != u || (int)(threadIdx.x & 31) >= L) continue;
#pragma unroll
      for (int i = 0; i < Part::groups; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const int j = sub + i * Part::per * L;
          if (j >= a.vecs) continue;
          const int2 c = columns_of<V>(j, e, L);
          held[c.x] = gw[i][e].x + (u ? held[c.x] : 0.f);
          held[a.dim + c.x] = gb[i][e].x + (u ? held[a.dim + c.x] : 0.f);
          if (c.y >= a.dim) continue;
          held[c.y] = gw[i][e].y + (u ? held[c.y] : 0.f);
          held[a.dim + c.y] = gb[i][e].y + (u ? held[a.dim + c.y] : 0.f);
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.dim; c += kNormThreads) part[c] = held[c];
  }
}

// The CTAs' sums, column by column, in a fixed order.
__global__ void __launch_bounds__(kSumCols* kSumRows) k_norm_sum(const float* __restrict__ part, int ctas, int dim,
                                                                float* __restrict__ gw, float* __restrict__ gb) {
  __shared__ float s[kSumRows][kSumCols + 1];
  pdl_wait();
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + col;
  float x = 0.f;
  if (c < 2 * dim)
#pragma unroll 8
    for (int i = row; i < ctas; i += kSumRows) x += part[(int64_t)i * 2 * dim + c];
  s[row][col] = x;
  __syncthreads();
  if (row || c >= 2 * dim) return;
#pragma unroll
  for (int i = 1; i < kSumRows; ++i) x += s[i][col];
  if (c < dim && gw) gw[c] = x;
  if (c >= dim && gb) gb[c - dim] = x;
}

namespace {

// CTAs on an SM at most (a thread of one that has a row to itself has 32 channels or
// fewer, and 1024 threads run).
int most_ctas(int dim) {
  if (dim <= 512) return kNormCtas;
  const int n = 1024 * 32 / dim;
  return n < 8 ? n : 8;
}

bool norm_view_ok(const scan_view* v, int32_t dtype, int64_t batch, int64_t len, int32_t dim, bool out) {
  if (!v || v->batch_stride < 0 || v->time_stride < 0) return false;
  if (batch == 0 || len == 0) return true;
  if (!v->data || !aligned_to(v->data, dtype_size(dtype))) return false;
  if (!out) return true;
  if (len > 1 && v->time_stride < dim) return false;
  return batch <= 1 || v->batch_stride >= (len - 1) * v->time_stride + dim;
}

template <class T>
NormView<T> norm_view(const scan_view* v) {
  return {(T*)v->data, v->batch_stride, v->time_stride};
}

// Elements of an access: whole rows move in accesses of one width.
int norm_width(int size, int32_t dim, std::initializer_list<const scan_view*> views) {
  const auto fits = [&](int v) {
    if (dim % v) return false;
    for (const scan_view* w : views)
      if (w->batch_stride % v || w->time_stride % v || !aligned_to(w->data, v * size)) return false;
    return true;
  };
  if (size == 4) return fits(4) ? 4 : 1;
  return fits(8) ? 8 : fits(2) ? 2 : 1;
}

// Calls f with (T*, W*, V, N, WIDE) and the log of the lanes (or the threads)
// of a row.  Rows of fewer than `least` accesses take one a lane.  Others take
// several, so that the sums' shuffles and the row's place are paid by fewer
// lanes; up to 1024 channels a warp holds a row (32 in a lane, where half as many do
// not do; single elements up to 512, their addresses take registers too), so that no barrier
// stands between its sums (52083 x 768 fp32 forward + backward 233 us in CTAs, 147 in
// warps).  Longer ones take a CTA of up to 512 threads, and only those beyond 16 elements a thread the most that registers hold (32).
template <class F>
cudaError_t with_norm(int32_t dtype, bool wide_weight, int v, int vecs, F f) {
  return with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const auto weights = [&](auto g) { return wide_weight ? g((float*)nullptr) : g((T*)nullptr); };
    return weights([&](auto* w) {
      using W = std::remove_pointer_t<decltype(w)>;
      using std::integral_constant;
      const auto of = [&](auto width, auto lean) {
        constexpr int V = decltype(width)::value, R = decltype(lean)::value;
        using One = integral_constant<int, 1>;
        using Half = integral_constant<int, 16 / V>;
        using Most = integral_constant<int, 32 / V>;
        const auto log2_of = [](int n) {
          int g = 0;
          while ((1 << g) < n) ++g;
          return g;
        };
        const auto warps = [&](int n) { return ((vecs + n - 1) / n + 31) / 32 * 32; };
        if (vecs < (V == 8 ? 8 : 16)) return f((T*)nullptr, (W*)nullptr, width, One(), std::false_type(), log2_of(vecs));
        if (vecs <= 32 * R) return f((T*)nullptr, (W*)nullptr, width, lean, std::false_type(), log2_of((vecs + R - 1) / R));
        using InWarp = std::conditional_t<V == 1, Half, Most>;
        if constexpr (R < InWarp::value)
          if (vecs <= 32 * InWarp::value) return f((T*)nullptr, (W*)nullptr, width, InWarp(), std::false_type(), 5);
        if (vecs <= kNormWide * Half::value) return f((T*)nullptr, (W*)nullptr, width, Half(), std::true_type(), warps(Half::value));
        return f((T*)nullptr, (W*)nullptr, width, Most(), std::true_type(), warps(Most::value));
      };
      if constexpr (sizeof(T) == 4) {
        if (v == 4) return of(integral_constant<int, 4>(), integral_constant<int, 4>());
      } else {
        if (v == 8) return of(integral_constant<int, 8>(), integral_constant<int, 4>());
        if (v == 2) return of(integral_constant<int, 2>(), integral_constant<int, 8>());
      }
      return of(integral_constant<int, 1>(), integral_constant<int, 8>());
    });
  });
}

// CTAs on an SM: where a CTA has a row, as many as its registers allow, up to 1024 threads
// (26041 x 1536 bf16 forward + backward 176 us with 512 threads, 140).
template <class K>
cudaError_t norm_grid(const emb_norm_s* h, int64_t rows, bool wide, int lanes, int ctas, K kernel, size_t smem, unsigned* grid) {
  const int per = wide ? 1 : kNormThreads >> lanes;
  const int64_t need = (rows + per - 1) / per;
  if (wide) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, lanes, smem);
    if (e != cudaSuccess) return e;
    ctas = ctas < 1024 / lanes ? ctas : 1024 / lanes;
    ctas = ctas < most_ctas(h->dim) ? ctas : most_ctas(h->dim);
    if (ctas < 1) ctas = 1;
  }
  const int64_t most = (int64_t)h->sm_count * ctas;
  *grid = (unsigned)(need < most ? need : most);
  return cudaSuccess;
}

bool norm_ok(emb_norm h, int32_t batch, int64_t len, int32_t dtype, const int32_t* offsets, int32_t weight_dtype) {
  return h && batch >= 0 && len >= 0 && on_device(h->device) && dtype_size(dtype) != 0 && aligned_to(offsets, 4) &&
         (weight_dtype == dtype || weight_dtype == EMB_DT_F32);
}

NormRows norm_rows(emb_norm h, int32_t batch, int64_t len, const int32_t* offsets, int v, float eps) {
  return {batch * len, len, make_div_magic((uint64_t)len), offsets, h->dim, h->dim / v, eps};
}

}  // namespace

}  // namespace emb

using namespace emb;

extern "C" emb_status norm_create(int32_t dim, emb_norm* out) {
  if (!out) return EMB_ERR_INVALID_ARG;
  *out = nullptr;
  if (dim < 1) return EMB_ERR_INVALID_ARG;
  if (dim > kNormMaxDim) return EMB_ERR_UNSUPPORTED;
  emb_norm_s* h = new (std::nothrow) emb_norm_s();
  if (!h) return EMB_ERR_OOM;
  h->dim = dim;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) e = dev_alloc((void**)&h->part_d, sizeof(float) * 2 * dim * h->sm_count * most_ctas(dim));
  if (e != cudaSuccess) {
    delete h;
    return cuda_status(e);
  }
  *out = h;
  return EMB_OK;
}

extern "C" emb_status norm_destroy(emb_norm h) {
  if (!h) return EMB_ERR_INVALID_ARG;
  const cudaError_t e = cudaDeviceSynchronize();
  dev_free(h->part_d);
  delete h;
  return cuda_status(e);
}

extern "C" emb_status norm_forward(emb_norm h, int32_t batch, int64_t len, int32_t dtype, const scan_view* x,
                                   const int32_t* offsets, int32_t weight_dtype, const void* weight, const void* bias,
                                   double eps, const scan_view* y, float* stats, void* stream) {
  if (!norm_ok(h, batch, len, dtype, offsets, weight_dtype) || !(eps >= 0) ||
      !norm_view_ok(x, dtype, batch, len, h->dim, false) || !norm_view_ok(y, dtype, batch, len, h->dim, true) ||
      !aligned_to(weight, dtype_size(weight_dtype)) || !aligned_to(bias, dtype_size(weight_dtype)) ||
      !aligned_to(stats, 8))
    return EMB_ERR_INVALID_ARG;
  if (batch == 0 || len == 0) return EMB_OK;
  const int v = norm_width(dtype_size(dtype), h->dim, {x, y});
  const NormRows a = norm_rows(h, batch, len, offsets, v, (float)eps);
  return cuda_status(with_norm(dtype, weight_dtype == EMB_DT_F32, v, a.vecs,
                               [&](auto* t, auto* w, auto width, auto count, auto wide, int lanes) {
    using T = std::remove_pointer_t<decltype(t)>;
    using W = std::remove_pointer_t<decltype(w)>;
    constexpr bool WIDE = decltype(wide)::value;
    const auto kernel = k_norm_fwd<T, W, decltype(width)::value, decltype(count)::value, WIDE>;
    const size_t smem = sizeof(float) * 2 * h->dim;
    if (smem > 48 << 10) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    unsigned ctas;
    const cudaError_t e = norm_grid(h, a.n, WIDE, lanes, kNormCtas, kernel, smem, &ctas);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, WIDE ? lanes : kNormThreads, smem, (cudaStream_t)stream>>>(
        a, norm_view<const T>(x), (const W*)weight, (const W*)bias, norm_view<T>(y), (float2*)stats, lanes);
    return cudaGetLastError();
  }));
}

extern "C" emb_status norm_backward(emb_norm h, int32_t batch, int64_t len, int32_t dtype, const scan_view* x,
                                    const int32_t* offsets, int32_t weight_dtype, const void* weight,
                                    const scan_view* grad_y, const float* stats, const scan_view* grad_x,
                                    float* grad_weight, float* grad_bias, void* stream) {
  if (!norm_ok(h, batch, len, dtype, offsets, weight_dtype) || !norm_view_ok(x, dtype, batch, len, h->dim, false) ||
      !norm_view_ok(grad_y, dtype, batch, len, h->dim, false) ||
      !norm_view_ok(grad_x, dtype, batch, len, h->dim, true) || !aligned_to(weight, dtype_size(weight_dtype)) ||
      !aligned_to(stats, 8) || !aligned_to(grad_weight, 4) || !aligned_to(grad_bias, 4))
    return EMB_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (batch == 0 || len == 0) {   // sums of nothing
    if (grad_weight) EMB_CUDA_TRY(cudaMemsetAsync(grad_weight, 0, sizeof(float) * h->dim, s));
    if (grad_bias) EMB_CUDA_TRY(cudaMemsetAsync(grad_bias, 0, sizeof(float) * h->dim, s));
    return EMB_OK;
  }
  if (!stats) return EMB_ERR_INVALID_ARG;
  const int v = norm_width(dtype_size(dtype), h->dim, {x, grad_y, grad_x});
  const NormRows a = norm_rows(h, batch, len, offsets, v, 0.f);
  float* part = grad_weight || grad_bias ? h->part_d : nullptr;
  unsigned ctas = 0;
  EMB_CUDA_TRY(with_norm(dtype, weight_dtype == EMB_DT_F32, v, a.vecs,
                         [&](auto* t, auto* w, auto width, auto count, auto wide, int lanes) {
    using T = std::remove_pointer_t<decltype(t)>;
    using W = std::remove_pointer_t<decltype(w)>;
    constexpr bool WIDE = decltype(wide)::value;
    const auto kernel = k_norm_bwd<T, W, decltype(width)::value, decltype(count)::value, WIDE>;
    const size_t smem = sizeof(float) * (WIDE ? 1 : 2) * h->dim;
    if (smem > 48 << 10) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    const cudaError_t e = norm_grid(h, a.n, WIDE, lanes, kBwdCtas, kernel, smem, &ctas);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, WIDE ? lanes : kNormThreads, smem, s>>>(a, norm_view<const T>(x), norm_view<const T>(grad_y),
                                                          (const float2*)stats, (const W*)weight,
                                                          norm_view<T>(grad_x), part, lanes);
    return cudaGetLastError();
  }));
  if (!part) return EMB_OK;
  return cuda_status(launch_dependent(k_norm_sum, (unsigned)((2 * h->dim + kSumCols - 1) / kSumCols), kSumCols * kSumRows, 0, s,
                                      (const float*)part, (int)ctas, (int)h->dim, grad_weight, grad_bias));
}
