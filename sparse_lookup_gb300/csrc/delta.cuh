// delta.cuh -- the gated delta rule's chunked kernels (library-internal); each
// element type's are compiled by a source of its own.
//
// Per sequence and head, S [key_dim][value_dim]:
//   S' = exp(g_t) S_{t-1};  e_t = v_t - S'^T k_t;  S_t = S' + beta_t k_t e_t^T;  y_t = scale S_t^T q_t
// Over a chunk of 32 positions, with G the running sum of g in it, S0 the state
// before it, D_ij = exp(G_i - G_j), M = strictly lower part of D o (K K^T) and
// A = scale times the lower part of D o (Q K^T):
//   E = (I + M diag(beta))^-1 (V - diag(exp G) K S0),  U = diag(beta) E
//   Y = scale diag(exp G) Q S0 + A U
//   S1 = exp(G_31) S0 + K^T diag(exp(G_31 - G)) U
// so a sequence is a chain of small matrix products whose length is time / 32.
//
// Columns of S (value channels) do not meet in this chain.  A consumer warp keeps 16
// of them, transposed, as the fp32 accumulators of its matrix instructions:
// S^T (16 x key_dim) and every intermediate (16 x 32) then pass from one product's
// result to the next one's left operand in registers, without shared memory or a
// barrier.  That, and operands that have to be split after each product, is why
// these are warp-wide products (m16n8k16) and not tcgen05 ones: a tensor-memory
// accumulator would have to come back through registers and shared memory after each
// of the chain's five products, and 16 x 32 results fill an eighth of its smallest
// tile.  Producer warps, each with a stage of shared memory, load a chunk and find
// its inverse and A, one chunk each, ahead of the consumers.
//
// Precision: sums are fp32.  An fp32 operand is split into bf16 terms (x = x0 + x1 +
// x2, each the rounded rest of those before); the products of terms i and j with i +
// j < the number of terms are summed.  Three terms carry 24 bits, two carry 16 (a
// value is off by 2^-17 at most).  Inputs of 16 bits are exact in one (bf16) or two
// (fp16) terms.
#pragma once

#include "rows.cuh"

struct emb_delta_s {
  int32_t key_dim = 0, value_dim = 0, heads = 0, key_heads = 0, max_batch = 0, max_len = 0, training = 0;
  int sm_count = 0, device = 0;
  // for the backward (see DeltaWork)
  uint4* s[3] = {nullptr, nullptr, nullptr};
  float4* e = nullptr;
  float* dots = nullptr;
  float* shared = nullptr;
};

namespace emb {

constexpr int kChunk = 32;

// A [batch, time, heads, dim] array (or [batch, time, heads]).
template <class T>
struct DView {
  T* data;
  int64_t batch, time, head;
};

// What the states' pass leaves for the reverse pass, chunk after chunk of each
// (entry, head), in the order of the lanes' registers.
struct DeltaWork {
  uint4* s[3];     // [chunks + 1][warps][DK / 16][32]: the state before a chunk in bf16 terms (fp32: three, else two)
  float4* e;       // [chunks][warps][4][32]: E
  float* dots;     // [warps][chunks][32]: <grad_y, y> over a warp's channels
  float* shared;   // [2][positions][heads][DK]: gradients of q and k before value heads are joined
  int64_t chunks;  // batch * heads * chunks of an entry
};

struct DeltaArgs {
  int32_t batch, len, heads, share;   // share: value heads of a key head
  int32_t key_dim, value_dim;
  int32_t chunks;                     // of an entry: (len + 31) / 32
  int32_t parts;                      // CTAs that share an (entry, head)'s value channels
  float scale;
  const int32_t* offsets;
  const float *state_in, *grad_last;
  float *state_out, *grad_state;
  DView<const float> decay, beta;
  DView<float> grad_decay, grad_beta;
  bool wide_qk, wide_v, wide_y, wide_gy;   // accesses of 16 bytes (of grad_q and grad_k: of two elements)
  DeltaWork work;
};

// ---------------------------------------------------------------------------
// matrix instructions
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two neighbours as N bf16 terms, from the largest.
template <int N>
__device__ __forceinline__ void split(float x, float y, uint32_t (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = pack(x, y);
    if (i + 1 < N) {
      const float2 h = unpack(t[i]);
      x -= h.x, y -= h.y;
    }
  }
}

// Rows of 2^n 16-byte pieces, 2 at least, whose places are exchanged so that eight
// rows of a matrix load lie in different banks.
__device__ __forceinline__ uint32_t piece(int row, int p, int log_pieces) {
  const int shift = log_pieces < 3 ? 3 - log_pieces : 0;
  return (uint32_t)(((row << log_pieces) + (p ^ ((row >> shift) & ((1 << (log_pieces < 3 ? log_pieces : 3)) - 1)))) << 4);
}
// Byte offset of a 16-bit element of such a tile.
__device__ __forceinline__ uint32_t element_at(int row, int col, int log_pieces) {
  return piece(row, col >> 3, log_pieces) + ((col & 7) << 1);
}

// A lower triangular 32 x 32 matrix: blocks (0,0), (1,0), (1,1) of 16 x 16.
constexpr int kLower = 1536;
__device__ __forceinline__ uint32_t lower_at(int row, int col) {
  return (uint32_t)(((row >> 4) + (col >> 4)) * 512) + element_at(row & 15, col & 15, 1);
}

// Addresses of the matrix loads for a lane.  X [n][k] as right operand: rows n0..+15,
// columns k0..+15 (not transposed); X [k][n]: rows k0, columns n0 (transposed).  As left
// operand: X [m][k] (not transposed), X [k][m] (transposed).
__device__ __forceinline__ uint32_t right_rows(int lane, int n0, int k0, int lp) {
  return piece(n0 + (lane & 7) + ((lane >> 4) << 3), (k0 >> 3) + ((lane >> 3) & 1), lp);
}
__device__ __forceinline__ uint32_t right_cols(int lane, int n0, int k0, int lp) {
  return piece(k0 + (lane & 15), (n0 >> 3) + (lane >> 4), lp);
}
__device__ __forceinline__ uint32_t left_rows(int lane, int m0, int k0, int lp) {
  return piece(m0 + (lane & 15), (k0 >> 3) + (lane >> 4), lp);
}
__device__ __forceinline__ uint32_t left_cols(int lane, int m0, int k0, int lp) {
  return piece(k0 + (lane & 7) + ((lane >> 4) << 3), (m0 >> 3) + ((lane >> 3) & 1), lp);
}

// acc += X Y over KS steps of 16.  left(s, a): the step's TA terms of X;
// right(p, s, j): address of term j of Y for the p-th 16 columns.  Products of
// terms i + j < N.  TRI 1: Y's steps s > p are zero, 2: s < p are.
template <int KS, int NP, int TA, int TB, int N, bool TRANS, int TRI, class L, class R>
__device__ __forceinline__ void product(float (&acc)[2 * NP][4], L left, R right) {
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint32_t a[TA][4];
    left(s, a);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      if ((TRI == 1 && s > p) || (TRI == 2 && s < p)) continue;
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        uint32_t b[4];
        load_matrices<TRANS>(b, right(p, s, j));
#pragma unroll
        for (int i = 0; i < TA; ++i)
          if (i + j < N) {
            multiply(acc[2 * p], a[i], b[0], b[1]);
            multiply(acc[2 * p + 1], a[i], b[2], b[3]);
          }
      }
    }
  }
}

// The left operand of a step from an earlier product's accumulators.
template <int N, int W>
__device__ __forceinline__ void left_of(const float (&x)[W][4], int s, uint32_t (&a)[N][4]) {
  uint32_t t[N];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      split<N>(x[2 * s + h][2 * r], x[2 * s + h][2 * r + 1], t);
#pragma unroll
      for (int i = 0; i < N; ++i) a[i][2 * h + r] = t[i];
    }
}

template <int W>
__device__ __forceinline__ void zero(float (&x)[W][4]) {
#pragma unroll
  for (int i = 0; i < W; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
}

// Barrier `id` between `n` threads: waiting, or only arriving.
__device__ __forceinline__ void meet(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// ---------------------------------------------------------------------------
// a stage: one chunk's inputs and what follows from them alone
// ---------------------------------------------------------------------------

// Numbers of a position in its chunk.
struct Spot {
  float since, until;   // exp(G_i), exp(G_31 - G_i)
  float beta;
  float g_hi, g_lo;     // G_i, as a multiple of 1/64 and the rest: differences keep their digits beside a large G
};

template <class T>
struct Terms;   // bf16 terms of an input, of which n are asked for
template <>
struct Terms<__nv_bfloat16> { static constexpr int of(int) { return 1; } };
template <>
struct Terms<__half> { static constexpr int of(int) { return 2; } };
template <>
struct Terms<float> { static constexpr int of(int n) { return n; } };

// Eight neighbouring elements.
template <class T>
struct Eight {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void gather(const T* p, int n) {   // n of them, zeros behind
    T* e = reinterpret_cast<T*>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int i) const { return to_f32(reinterpret_cast<const T*>(u)[i]); }
};

// Rows 0 .. 31 (`live` of them) of `cols` columns, by one warp: as bf16 terms in tiles
// `plane` bytes apart of 2^lp pieces a row, or as fp32 rows of `width` (a multiple of
// 16) and four floats.  Columns and rows beyond the array's are 0.
template <class T, int IT>
__device__ __forceinline__ void load_terms(unsigned char* tile, int plane, int lp, const T* rows, int64_t stride, int live,
                                           int cols, bool wide, int lane) {
  constexpr int U = sizeof(T) == 2 ? 8 : 4;
  const int pieces = 1 << lp, units = kChunk << lp;
  for (int u0 = lane; u0 < units; u0 += 32 * U) {
    Eight<T> x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + 32 * k, r = u >> lp, c = (u & (pieces - 1)) << 3;
      if (u >= units || r >= live || c >= cols) x[k].clear();
      else if (wide) x[k].load(rows + r * stride + c);
      else x[k].gather(rows + r * stride + c, cols - c);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + 32 * k;
      if (u >= units) continue;
      const uint32_t at = piece(u >> lp, u & (pieces - 1), lp);
      if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        *reinterpret_cast<uint4*>(tile + at) = x[k].u[0];
      } else {
        uint32_t w[4][IT];
#pragma unroll
        for (int i = 0; i < 4; ++i) split<IT>(x[k].at(2 * i), x[k].at(2 * i + 1), w[i]);
#pragma unroll
        for (int i = 0; i < IT; ++i)
          *reinterpret_cast<uint4*>(tile + i * plane + at) = make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
      }
    }
  }
}
template <class T>
__device__ __forceinline__ void load_floats(float* tile, int width, const T* rows, int64_t stride, int live, int cols,
                                            bool wide, int lane) {
  constexpr int U = sizeof(T) == 2 ? 8 : 4;
  const int lp = 32 - __clz((width >> 3) - 1), pieces = 1 << lp, units = kChunk << lp;
  for (int u0 = lane; u0 < units; u0 += 32 * U) {
    Eight<T> x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + 32 * k, r = u >> lp, c = (u & (pieces - 1)) << 3;
      if (u >= units || r >= live || c >= cols) x[k].clear();
      else if (wide) x[k].load(rows + r * stride + c);
      else x[k].gather(rows + r * stride + c, cols - c);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + 32 * k, c = (u & (pieces - 1)) << 3;
      if (u >= units || c >= width) continue;
      float* to = tile + (u >> lp) * (width + 4) + c;
      *reinterpret_cast<float4*>(to) = make_float4(x[k].at(0), x[k].at(1), x[k].at(2), x[k].at(3));
      *reinterpret_cast<float4*>(to + 4) = make_float4(x[k].at(4), x[k].at(5), x[k].at(6), x[k].at(7));
    }
  }
}

// The chunk's positions, by one warp: position i is lane i.  A decay below -512 counts
// as -512 (exp is 0 long before), so that -infinity forgets and sums stay exact.
__device__ __forceinline__ void find_spots(Spot* spots, float g, float beta, int lane) {
  g = g < -512.f ? -512.f : g;
  float hi = rintf(g * 64.f) * 0.015625f, lo = g - hi;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float a = __shfl_up_sync(kFull, hi, o), b = __shfl_up_sync(kFull, lo, o);
    if (lane >= o) hi += a, lo += b;
  }
  const float end_hi = __shfl_sync(kFull, hi, 31), end_lo = __shfl_sync(kFull, lo, 31);
  Spot s;
  s.since = expf(hi) * expf(lo);
  s.until = expf((end_hi - hi) + (end_lo - lo));
  s.beta = beta;
  s.g_hi = hi, s.g_lo = lo;
  spots[lane] = s;
}

// exp(G_i - G_j)
__device__ __forceinline__ float between(const Spot& i, const Spot& j) {
  return expf((i.g_hi - j.g_hi) + (i.g_lo - j.g_lo));
}

// Lower blocks of D o (X K^T) by one warp, X and K in tiles of IT terms; put(i, j, value)
// gets every element of the three blocks.
template <int DK, int IT, class F>
__device__ __forceinline__ void find_lower(uint32_t x, uint32_t k, int plane, const Spot* spots, int lane, F put) {
  constexpr int lp = DK == 128 ? 4 : DK == 64 ? 3 : 2;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float acc[4][4];
    zero(acc);
    const auto left = [&](int s, uint32_t (&a)[IT][4]) {
#pragma unroll
      for (int i = 0; i < IT; ++i) load_matrices<false>(a[i], x + i * plane + left_rows(lane, 16 * m, 16 * s, lp));
    };
    const auto right = [&](int p, int s, int j) { return k + j * plane + right_rows(lane, 16 * p, 16 * s, lp); };
    if (m == 0) {
      float one[2][4];
      zero(one);
      product<DK / 16, 1, IT, IT, 3, false, 0>(one, left, right);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = one[i][r];
    } else {
      product<DK / 16, 2, IT, IT, 3, false, 0>(acc, left, right);
    }
#pragma unroll
    for (int n = 0; n < 2 * (m + 1); ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * m + g + (r >> 1) * 8, j = 8 * n + 2 * t + (r & 1);
        put(i, j, i >= j ? acc[n][r] * between(spots[i], spots[j]) : 0.f);
      }
  }
}

template <int N>
__device__ __forceinline__ void put_lower(unsigned char* tile, int i, int j, float x) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    *reinterpret_cast<__nv_bfloat16*>(tile + k * kLower + lower_at(i, j)) = h;
    x -= __bfloat162float(h);
  }
}

// (I + M diag(beta))^-1 by forward substitution, column j in lane j; row i of `m`
// (32 x 36 floats) holds M_ij beta_j.  By substitution, not by powers of M, which
// cancel where keys repeat.
template <int N>
__device__ __forceinline__ void invert(const float* m, unsigned char* tile, int lane) {
  float x[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    float a = i == lane ? 1.f : 0.f, b = 0.f, c = 0.f, d = 0.f;
#pragma unroll
    for (int l = 0; l < i; l += 4) {
      const float4 w = *reinterpret_cast<const float4*>(m + i * 36 + l);
      a -= w.x * x[l];
      if (l + 1 < i) b -= w.y * x[l + 1];
      if (l + 2 < i) c -= w.z * x[l + 2];
      if (l + 3 < i) d -= w.w * x[l + 3];
    }
    x[i] = (a + b) + (c + d);
    if (i >= 16 || lane < 16) put_lower<N>(tile, i, lane, x[i]);
  }
}

__device__ __forceinline__ int length_of(const DeltaArgs& a, int b) {
  if (!a.offsets) return a.len;
  const int64_t n = (int64_t)a.offsets[b + 1] - a.offsets[b];
  return n < 0 ? 0 : n < a.len ? (int)n : a.len;
}

constexpr int log_of(int n) { return n <= 1 ? 0 : 1 + log_of(n / 2); }

// ---------------------------------------------------------------------------
// forward, and the states' pass before a backward
// ---------------------------------------------------------------------------

constexpr int kForwardTerms = 3;
template <class T>
constexpr int kKept = sizeof(T) == 2 ? 2 : 3;   // terms of the states that are kept for a backward

// Bytes of a stage.  STATES: the states' pass, which has grad_y in it.
template <class T, int DK, bool STATES>
struct ForwardStage {
  static constexpr int NT = kForwardTerms, IT = Terms<T>::of(NT), lp = log_of(DK / 8), plane = kChunk * DK * 2;
  static constexpr int k = 0, q = k + IT * plane, inverse = q + IT * plane, a = inverse + NT * kLower,
                       spots = a + NT * kLower, scratch = spots + kChunk * (int)sizeof(Spot),
                       v = scratch + kChunk * 36 * 4;
  // V and grad_y are fp32 rows of `dv` columns and four more, which keep the banks of a read apart
  static constexpr int bytes(int dv) { return v + (STATES ? 2 : 1) * kChunk * (dv + 4) * 4; }
};

// Consumer warps first (one for 16 value channels), then the producers.
template <class T, int DK, bool STATES>
__global__ void __launch_bounds__(384)
    k_delta_fwd(DeltaArgs a, DView<const T> q, DView<const T> k, DView<const T> v, DView<const T> gy, DView<T> y,
                int producers) {
  using Stage = ForwardStage<T, DK, STATES>;
  constexpr int NT = Stage::NT, IT = Stage::IT, lp = Stage::lp, plane = Stage::plane;
  // terms of what goes into y alone: 16 bits are stored of it, so two carry enough.  The
  // decays' gradients are sums of <grad_y, y> over many positions: all terms
  constexpr int NO = !STATES && sizeof(T) == 2 ? 2 : NT;
  extern __shared__ __align__(128) unsigned char held[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int consumers = (blockDim.x >> 5) - producers, meeting = 32 * (consumers + 1);
  const int dv = 16 * consumers, size = Stage::bytes(dv);
  const int part = blockIdx.x % a.parts, bh = blockIdx.x / a.parts, b = bh / a.heads, h = bh % a.heads;
  const int hk = h / a.share, first_v = part * dv;
  const int len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk;
  if (warp >= consumers) {
    const int p = warp - consumers;
    unsigned char* st = held + p * size;
    Spot* spots = reinterpret_cast<Spot*>(st + Stage::spots);
    float* scratch = reinterpret_cast<float*>(st + Stage::scratch);
    const int cols_v = min(dv, a.value_dim - first_v);
    for (int c = p; c < chunks; c += producers) {
      if (c >= producers) meet(1 + producers + p, meeting);
      const int t0 = c * kChunk, live = min(kChunk, len - t0), t = t0 + lane;
      const float g = lane < live ? a.decay.data[b * a.decay.batch + t * a.decay.time + h * a.decay.head] : 0.f;
      const float beta = lane < live ? a.beta.data[b * a.beta.batch + t * a.beta.time + h * a.beta.head] : 0.f;
      load_terms<T, IT>(st + Stage::k, plane, lp, k.data + b * k.batch + t0 * k.time + hk * k.head, k.time, live,
                        a.key_dim, a.wide_qk, lane);
      load_terms<T, IT>(st + Stage::q, plane, lp, q.data + b * q.batch + t0 * q.time + hk * q.head, q.time, live,
                        a.key_dim, a.wide_qk, lane);
      float* tile = reinterpret_cast<float*>(st + Stage::v);
      for (int w = 0; w < (STATES ? 2 : 1); ++w) {
        const DView<const T>& x = w ? gy : v;
        load_floats<T>(tile + w * kChunk * (dv + 4), dv, x.data + b * x.batch + t0 * x.time + h * x.head + first_v,
                       x.time, live, cols_v, a.wide_v, lane);
      }
      find_spots(spots, g, beta, lane);
      __syncwarp();
      find_lower<DK, IT>(smem_of(st + Stage::k), smem_of(st + Stage::k), plane, spots, lane,
                         [&](int i, int j, float x) { scratch[i * 36 + j] = i > j ? x * spots[j].beta : 0.f; });
      find_lower<DK, IT>(smem_of(st + Stage::q), smem_of(st + Stage::k), plane, spots, lane,
                         [&](int i, int j, float x) { put_lower<NO>(st + Stage::a, i, j, x * a.scale); });
      __syncwarp();
      invert<NT>(scratch, st + Stage::inverse, lane);
      arrive(1 + p, meeting);
    }
    return;
  }
  const int g = lane >> 2, t = lane & 3, e0 = first_v + 16 * warp;
  const int64_t head = (int64_t)b * a.heads + h;
  float S[DK / 8][4];   // S^T: channel e0 + g (+ 8), key columns 8 n + 2 t (+ 1)
#pragma unroll
  for (int n = 0; n < DK / 8; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
      S[n][r] = a.state_in && d < a.key_dim && e < a.value_dim
                    ? a.state_in[(head * a.key_dim + d) * a.value_dim + e] : 0.f;
    }
  const int64_t warps = (int64_t)consumers * a.parts;
  const auto keep = [&](int c) {   // the state before chunk c, for the reverse pass
    const int64_t at = ((head * (a.chunks + 1) + c) * warps + part * consumers + warp) * (DK / 16) * 32 + lane;
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t x[kKept<T>][4];
      left_of<kKept<T>>(S, s, x);
#pragma unroll
      for (int j = 0; j < kKept<T>; ++j) a.work.s[j][at + s * 32] = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
    }
  };
  float* own = reinterpret_cast<float*>(held + producers * size) + warp * kChunk * 17;   // a warp's results, turned
  int stage = 0;
  for (int c = 0; c < chunks; ++c) {
    unsigned char* st = held + stage * size;
    const uint32_t base = smem_of(st);
    const Spot* spots = reinterpret_cast<const Spot*>(st + Stage::spots);
    const float* vt = reinterpret_cast<const float*>(st + Stage::v) + 16 * warp;
    if constexpr (STATES) keep(c);
    meet(1 + stage, meeting);
    const int t0 = c * kChunk, live = min(kChunk, len - t0);
    // Z = V - exp(G) K S0
    float Z[4][4], E[4][4];
    zero(Z);
    product<DK / 16, 2, NT, IT, NT, false, 0>(
        Z, [&](int s, uint32_t (&x)[NT][4]) { left_of<NT>(S, s, x); },
        [&](int p, int s, int j) { return base + Stage::k + j * plane + right_rows(lane, 16 * p, 16 * s, lp); });
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 8 * n + 2 * t + (r & 1);
        Z[n][r] = vt[i * (dv + 4) + g + (r >> 1) * 8] - spots[i].since * Z[n][r];
      }
    zero(E);
    product<2, 2, NT, NT, NT, false, 1>(
        E, [&](int s, uint32_t (&x)[NT][4]) { left_of<NT>(Z, s, x); },
        [&](int p, int s, int j) {
          return base + Stage::inverse + j * kLower + (p + s) * 512 + right_rows(lane, 0, 0, 1);
        });
    {
      float Y[4][4], U[4][4];
      zero(Y);
      product<DK / 16, 2, NO, IT, NO, false, 0>(
          Y, [&](int s, uint32_t (&x)[NO][4]) { left_of<NO>(S, s, x); },
          [&](int p, int s, int j) { return base + Stage::q + j * plane + right_rows(lane, 16 * p, 16 * s, lp); });
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const Spot& s = spots[8 * n + 2 * t + (r & 1)];
          Y[n][r] *= a.scale * s.since;
          U[n][r] = s.beta * E[n][r];
        }
      product<2, 2, NO, NO, NO, false, 1>(
          Y, [&](int s, uint32_t (&x)[NO][4]) { left_of<NO>(U, s, x); },
          [&](int p, int s, int j) { return base + Stage::a + j * kLower + (p + s) * 512 + right_rows(lane, 0, 0, 1); });
      if constexpr (STATES) {
        // <grad_y, y> over the warp's channels; E for the reverse pass
        const float* gt = vt + kChunk * (dv + 4);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int i = 8 * n + 2 * t + r;
            float x = Y[n][r] * gt[i * (dv + 4) + g] + Y[n][2 + r] * gt[i * (dv + 4) + g + 8];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
            if (g == 0) own[i] = x;
          }
          a.work.e[(((head * a.chunks + c) * warps + part * consumers + warp) * 4 + n) * 32 + lane] =
              make_float4(E[n][0], E[n][1], E[n][2], E[n][3]);
        }
        __syncwarp();
        a.work.dots[((part * consumers + warp) * a.work.chunks + head * a.chunks + c) * kChunk + lane] = own[lane];
        __syncwarp();
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) own[(8 * n + 2 * t + (r & 1)) * 17 + g + (r >> 1) * 8] = Y[n][r];
        __syncwarp();
        if (t0 + lane < a.len) {   // dead positions of the chunk too: 0
          T* to = y.data + b * y.batch + (int64_t)(t0 + lane) * y.time + h * y.head + e0;
          const float* from = own + lane * 17;
          const bool on = lane < live;
          if (a.wide_y && e0 + 16 <= a.value_dim) {
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int i = 0; i < 16; i += V) {
              Vec<T, V> o;
#pragma unroll
              for (int u = 0; u < V; ++u) o.e[u] = from_f32<T>(on ? from[i + u] : 0.f);
              store_vec(to + i, o);
            }
          } else {
            for (int i = 0; i < 16 && e0 + i < a.value_dim; ++i) to[i] = from_f32<T>(on ? from[i] : 0.f);
          }
        }
        __syncwarp();
      }
    }
    // S1 = exp(G_31) S0 + K^T (exp(G_31 - G) beta E)
    const float whole = spots[kChunk - 1].since;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const Spot& s = spots[8 * n + 2 * t + (r & 1)];
        E[n][r] *= s.until * s.beta;
      }
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[n][r] *= whole;
    product<2, DK / 16, NT, IT, NT, true, 0>(
        S, [&](int s, uint32_t (&x)[NT][4]) { left_of<NT>(E, s, x); },
        [&](int p, int s, int j) { return base + Stage::k + j * plane + right_cols(lane, 16 * p, 16 * s, lp); });
    if (c + producers < chunks) arrive(1 + producers + stage, meeting);
    stage = stage + 1 == producers ? 0 : stage + 1;
  }
  if constexpr (STATES) keep(chunks);
  if constexpr (!STATES) {
    if (a.state_out)
#pragma unroll
      for (int n = 0; n < DK / 8; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
          if (d < a.key_dim && e < a.value_dim) a.state_out[(head * a.key_dim + d) * a.value_dim + e] = S[n][r];
        }
    // positions past the last chunk
    for (int64_t i = (int64_t)chunks * kChunk + (lane >> 4); i < a.len; i += 2)
      if (e0 + (lane & 15) < a.value_dim)
        y.data[b * y.batch + i * y.time + h * y.head + e0 + (lane & 15)] = from_f32<T>(0.f);
  }
}

// ---------------------------------------------------------------------------
// reverse
// ---------------------------------------------------------------------------

// Terms of the reverse pass' operands: of the recursion (R), of the states (S) and of
// U, dZ, dA and X (U) in the products that give the gradients of q and k.  Those alone
// are of 16 bits where q is: the states are rounded once for a bf16 result, as its own
// store rounds it.  128 key channels of fp16 or fp32 leave shared memory for two terms
// (2^-17 of an operand at most, 5e-6 of an fp32 gradient); <dS, S> is then taken anew
// in every chunk.
template <class T, int DK>
struct ReverseTerms {
  static constexpr bool tight = DK == 128 && !std::is_same_v<T, __nv_bfloat16>;
  static constexpr int R = tight ? 2 : 3;
  static constexpr int S = std::is_same_v<T, __nv_bfloat16> ? 1 : std::is_same_v<T, float> && !tight ? 3 : 2;
  static constexpr int U = std::is_same_v<T, float> && !tight ? 3 : 2;
  static constexpr int again = tight ? 1 : 4;   // chunks between the exact values of <dS, S>
};

template <class T, int DK>
struct ReverseStage {
  static constexpr int NR = ReverseTerms<T, DK>::R;
  static constexpr int IT = Terms<T>::of(NR), lp = log_of(DK / 8), plane = kChunk * DK * 2;
  static constexpr int k = 0, q = k + IT * plane, inverse = q + IT * plane, a = inverse + NR * kLower,
                       m = a + NR * kLower, spots = m + NR * kLower, gy = spots + kChunk * (int)sizeof(Spot);
  // before grad_y is there, its place holds the matrix that is inverted
  static constexpr int bytes(int dvp) {
    return gy + (IT * kChunk * dvp * 2 > kChunk * 36 * 4 ? IT * kChunk * dvp * 2 : kChunk * 36 * 4);
  }
};
// What the consumers share: dS and S [channels][DK], U and dZ [32][channels], dA and X +
// X^T [32][32], sums.
template <class T, int DK>
struct ReverseShared {
  static constexpr int NS = ReverseTerms<T, DK>::S, NU = ReverseTerms<T, DK>::U;
  int ds, s, u, dz, da, xs, red, bytes;
  __host__ __device__ ReverseShared(int warps, int dvp) {
    ds = 0;
    s = ds + NS * warps * 16 * DK * 2;
    u = s + NS * warps * 16 * DK * 2;
    dz = u + NU * kChunk * dvp * 2;
    da = dz + NU * kChunk * dvp * 2;
    xs = da + NU * kLower;
    red = xs + NU * 2048;
    bytes = red + (warps * 66 + 3) / 4 * 16;
  }
};

// From the last chunk to the first, with dS (the gradient of the state after the
// chunk) in the accumulators as S was:
//   dU = A^T dY + diag(exp(G_31 - G)) K dS;  dE = diag(beta) dU;  dZ = (..)^-T dE = dV
//   dbeta = E . (dU - M^T dZ)                        (sums over the channels)
//   dS0 = exp(G_31) dS + Q^T (scale exp(G) dY) - K^T (exp(G) dZ)
// and, with the channels of all warps in shared memory, dA = scale D o (dY U^T) and X =
// -D o (dZ U^T) below the diagonal,
//   dQ = scale exp(G) dY S0^T + dA K
//   dK = exp(G_31 - G) U dS^T - exp(G) dZ S0^T + dA^T Q + (X + X^T) K
// Decays: y and S1 are homogeneous in (S0, V), so dG_i = dY_i . Y_i - dV_i . V_i, and
// the gradient of g_t is their sum from t to the chunk's end and <dS, S1> there.  That
// number is carried from chunk to chunk by the same sums, and taken anew from the
// states every few chunks, before roundings add up.
template <class T, int DK>
__global__ void __launch_bounds__(320)
    k_delta_bwd(DeltaArgs a, DView<const T> q, DView<const T> k, DView<const T> v, DView<const T> gy, DView<T> gq,
                DView<T> gk, DView<T> gv, int producers) {
  using Stage = ReverseStage<T, DK>;
  using Shared = ReverseShared<T, DK>;
  constexpr int IT = Stage::IT, lp = Stage::lp, plane = Stage::plane, NR = Stage::NR, NS = Shared::NS, NU = Shared::NU,
                kAgain = ReverseTerms<T, DK>::again;
  extern __shared__ __align__(128) unsigned char held[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = (blockDim.x >> 5) - producers, meeting = 32 * (W + 1);
  const int lv = W == 1 ? 1 : 32 - __clz(2 * W - 1), dvp = 8 << lv, plane_v = kChunk * dvp * 2;
  const int size = Stage::bytes(dvp);
  const int bh = blockIdx.x, b = bh / a.heads, h = bh % a.heads, hk = h / a.share;
  const int len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk;
  const Shared at(W, dvp);
  unsigned char* shared = held + producers * size;
  if (warp >= W) {
    const int p = warp - W;
    unsigned char* st = held + p * size;
    Spot* spots = reinterpret_cast<Spot*>(st + Stage::spots);
    float* scratch = reinterpret_cast<float*>(st + Stage::gy);
    for (int n = p; n < chunks; n += producers) {
      if (n >= producers) meet(1 + producers + p, meeting);
      const int t0 = (chunks - 1 - n) * kChunk, live = min(kChunk, len - t0), t = t0 + lane;
      const float g = lane < live ? a.decay.data[b * a.decay.batch + t * a.decay.time + h * a.decay.head] : 0.f;
      const float beta = lane < live ? a.beta.data[b * a.beta.batch + t * a.beta.time + h * a.beta.head] : 0.f;
      load_terms<T, IT>(st + Stage::k, plane, lp, k.data + b * k.batch + t0 * k.time + hk * k.head, k.time, live,
                        a.key_dim, a.wide_qk, lane);
      load_terms<T, IT>(st + Stage::q, plane, lp, q.data + b * q.batch + t0 * q.time + hk * q.head, q.time, live,
                        a.key_dim, a.wide_qk, lane);
      find_spots(spots, g, beta, lane);
      __syncwarp();
      find_lower<DK, IT>(smem_of(st + Stage::k), smem_of(st + Stage::k), plane, spots, lane,
                         [&](int i, int j, float x) {
                           x = i > j ? x : 0.f;
                           scratch[i * 36 + j] = x * spots[j].beta;
                           put_lower<NR>(st + Stage::m, i, j, x);
                         });
      find_lower<DK, IT>(smem_of(st + Stage::q), smem_of(st + Stage::k), plane, spots, lane,
                         [&](int i, int j, float x) { put_lower<NR>(st + Stage::a, i, j, x * a.scale); });
      __syncwarp();
      invert<NR>(scratch, st + Stage::inverse, lane);
      __syncwarp();
      load_terms<T, IT>(st + Stage::gy, plane_v, lv, gy.data + b * gy.batch + t0 * gy.time + h * gy.head, gy.time, live,
                        a.value_dim, a.wide_v, lane);
      arrive(1 + p, meeting);
    }
    return;
  }
  const int g = lane >> 2, t = lane & 3, e0 = 16 * warp;
  const int64_t head = (int64_t)b * a.heads + h;
  float dS[DK / 8][4];
#pragma unroll
  for (int n = 0; n < DK / 8; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
      dS[n][r] = a.grad_last && d < a.key_dim && e < a.value_dim
                     ? a.grad_last[(head * a.key_dim + d) * a.value_dim + e] : 0.f;
    }
  float* red = reinterpret_cast<float*>(shared + at.red);   // [warps][2][32]: dbeta, <dV, V>
  float* along = red + W * 64;                              // [2][warps]: <dS, S>, of chunks in turn
  const uint32_t sh = smem_of(shared);
  const auto state_at = [&](int c) { return ((head * (a.chunks + 1) + c) * W + warp) * (DK / 16) * 32 + lane; };
  const auto word = [](const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; };
  // <dS, S> over the warp's channels
  const auto find_along = [&](int c) {
    const int64_t from = state_at(c);
    float x = 0.f;
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint4 u[kKept<T>];
#pragma unroll
      for (int j = 0; j < kKept<T>; ++j) u[j] = a.work.s[j][from + s * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f = unpack(word(u[kKept<T> - 1], i));
#pragma unroll
        for (int j = kKept<T> - 2; j >= 0; --j) {
          const float2 w = unpack(word(u[j], i));
          f.x += w.x, f.y += w.y;
        }
        x += dS[2 * s + (i >> 1)][2 * (i & 1)] * f.x + dS[2 * s + (i >> 1)][2 * (i & 1) + 1] * f.y;
      }
    }
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    if (lane == 0) along[(c & 1) * W + warp] = x;
  };
  find_along(chunks);
  float carry = 0.f;
  int stage = 0;
  for (int n0 = 0; n0 < chunks; ++n0) {
    const int c = chunks - 1 - n0, t0 = c * kChunk, live = min(kChunk, len - t0);
    unsigned char* st = held + stage * size;
    const uint32_t base = smem_of(st);
    const Spot* spots = reinterpret_cast<const Spot*>(st + Stage::spots);
    // what the states' pass left, and V where this lane's dV will be
    uint4 s0[DK / 16];
    const int64_t from = state_at(c);
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) s0[s] = a.work.s[0][from + s * 32];
    float E[4][4], V[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float4 x = a.work.e[(((head * a.chunks + c) * W + warp) * 4 + n) * 32 + lane];
      E[n][0] = x.x, E[n][1] = x.y, E[n][2] = x.z, E[n][3] = x.w;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
        V[n][r] = i < live && e < a.value_dim
                      ? to_f32(v.data[b * v.batch + (int64_t)(t0 + i) * v.time + h * v.head + e]) : 0.f;
      }
    }
    float dots = 0.f;
    if (warp == 0)
      for (int w = 0; w < W; ++w) dots += a.work.dots[(w * a.work.chunks + head * a.chunks + c) * kChunk + lane];
    meet(1 + stage, meeting);   // the stage is there, and every warp is through with the chunk before
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t x[NS][4];
      left_of<NS>(dS, s, x);
      uint4 u[NS];
      u[0] = s0[s];
#pragma unroll
      for (int j = 1; j < NS; ++j) u[j] = a.work.s[j][from + s * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t to = element_at(e0 + g + 8 * (i & 1), 16 * s + 8 * (i >> 1) + 2 * t, lp);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int tile = j * W * 16 * DK * 2;
          *reinterpret_cast<uint32_t*>(shared + at.ds + tile + to) = x[j][i];
          *reinterpret_cast<uint32_t*>(shared + at.s + tile + to) = word(u[j], i);
        }
      }
    }
    float dU[4][4], dZ[4][4];
    zero(dU);
    product<DK / 16, 2, NR, IT, NR, false, 0>(
        dU, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(dS, s, x); },
        [&](int p, int s, int j) { return base + Stage::k + j * plane + right_rows(lane, 16 * p, 16 * s, lp); });
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) dU[n][r] *= spots[8 * n + 2 * t + (r & 1)].until;
    const auto lower = [&](int tile, int p, int s, int j) {
      return base + tile + j * kLower + (p + s) * 512 + right_cols(lane, 0, 0, 1);
    };
    product<2, 2, IT, NR, NR, true, 2>(
        dU,
        [&](int s, uint32_t (&x)[IT][4]) {
#pragma unroll
          for (int i = 0; i < IT; ++i)
            load_matrices<true>(x[i], base + Stage::gy + i * plane_v + left_cols(lane, e0, 16 * s, lv));
        },
        [&](int p, int s, int j) { return lower(Stage::a, p, s, j); });
    zero(dZ);
    {
      float dE[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) dE[n][r] = spots[8 * n + 2 * t + (r & 1)].beta * dU[n][r];
      product<2, 2, NR, NR, NR, true, 2>(
          dZ, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(dE, s, x); },
          [&](int p, int s, int j) { return lower(Stage::inverse, p, s, j); });
    }
    {
      float R[4][4];
      zero(R);
      product<2, 2, NR, NR, NR, true, 2>(
          R, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(dZ, s, x); },
          [&](int p, int s, int j) { return lower(Stage::m, p, s, j); });
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = E[n][r] * (dU[n][r] - R[n][r]) + E[n][2 + r] * (dU[n][2 + r] - R[n][2 + r]);
          float y = dZ[n][r] * V[n][r] + dZ[n][2 + r] * V[n][2 + r];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            x += __shfl_xor_sync(kFull, x, o);
            y += __shfl_xor_sync(kFull, y, o);
          }
          if (g == 0) {
            red[warp * 64 + 8 * n + 2 * t + r] = x;
            red[warp * 64 + 32 + 8 * n + 2 * t + r] = y;
          }
        }
    }
    // U and dZ for the other warps; dV
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
        const uint32_t to = element_at(i, e, lv);
        float u = spots[i].beta * E[n][r], z = dZ[n][r];
        if (t0 + i < a.len && e < a.value_dim)
          gv.data[b * gv.batch + (int64_t)(t0 + i) * gv.time + h * gv.head + e] = from_f32<T>(i < live ? z : 0.f);
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          const __nv_bfloat16 uh = __float2bfloat16_rn(u), zh = __float2bfloat16_rn(z);
          *reinterpret_cast<__nv_bfloat16*>(shared + at.u + j * plane_v + to) = uh;
          *reinterpret_cast<__nv_bfloat16*>(shared + at.dz + j * plane_v + to) = zh;
          u -= __bfloat162float(uh), z -= __bfloat162float(zh);
        }
      }
    // the gradient of the state before the chunk
    const float whole = spots[kChunk - 1].since;
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) dS[n][r] *= whole;
    product<2, DK / 16, NR, IT, NR, true, 0>(
        dS,
        [&](int s, uint32_t (&x)[NR][4]) {
          uint32_t y[IT][4];
#pragma unroll
          for (int i = 0; i < IT; ++i)
            load_matrices<true>(y[i], base + Stage::gy + i * plane_v + left_cols(lane, e0, 16 * s, lv));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at_i = 16 * s + 8 * (i >> 1) + 2 * t;
            float2 f = unpack(y[IT - 1][i]);
#pragma unroll
            for (int j = IT - 2; j >= 0; --j) {
              const float2 l = unpack(y[j][i]);
              f.x += l.x, f.y += l.y;
            }
            uint32_t w[NR];
            split<NR>(f.x * (a.scale * spots[at_i].since), f.y * (a.scale * spots[at_i + 1].since), w);
#pragma unroll
            for (int j = 0; j < NR; ++j) x[j][i] = w[j];
          }
        },
        [&](int p, int s, int j) { return base + Stage::q + j * plane + right_cols(lane, 16 * p, 16 * s, lp); });
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) dZ[n][r] *= -spots[8 * n + 2 * t + (r & 1)].since;
    product<2, DK / 16, NR, IT, NR, true, 0>(
        dS, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(dZ, s, x); },
        [&](int p, int s, int j) { return base + Stage::k + j * plane + right_cols(lane, 16 * p, 16 * s, lp); });
    meet(1 + 2 * producers, 32 * W);
    if (warp == 0) {
      float gb = 0.f, dv = 0.f;
      for (int w = 0; w < W; ++w) gb += red[w * 64 + lane], dv += red[w * 64 + 32 + lane];
      if (n0 == 0 || (c + 1) % kAgain == 0) {
        carry = 0.f;
        for (int w = 0; w < W; ++w) carry += along[((c + 1) & 1) * W + w];
      }
      float x = dots - dv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(kFull, x, o);
        if (lane + o < 32) x += y;
      }
      const int i = t0 + lane;
      if (i < a.len) {
        const bool on = lane < live;
        // where exp(g) is 0 so is its gradient, which the sums give to their rounding
        const float g_i = on ? a.decay.data[b * a.decay.batch + i * a.decay.time + h * a.decay.head] : 0.f;
        a.grad_decay.data[b * a.grad_decay.batch + i * a.grad_decay.time + h * a.grad_decay.head] =
            on && expf(g_i) != 0.f ? x + carry : 0.f;
        a.grad_beta.data[b * a.grad_beta.batch + i * a.grad_beta.time + h * a.grad_beta.head] = on ? gb : 0.f;
      }
      carry += __shfl_sync(kFull, x, 0);
    }
    // dA and X, a 16 x 16 block at a time
    for (int u = warp; u < 6; u += W) {
      const bool is_x = u >= 3;
      const int blk = is_x ? u - 3 : u, mi = (blk + 1) >> 1, pj = blk >> 1;
      float acc[2][4];
      zero(acc);
      for (int s = 0; s < W; ++s) {
        uint32_t x[NU][4], y[NU][4];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          load_matrices<false>(y[i], sh + at.u + i * plane_v + right_rows(lane, 16 * pj, 16 * s, lv));
          if (is_x) load_matrices<false>(x[i], sh + at.dz + i * plane_v + left_rows(lane, 16 * mi, 16 * s, lv));
          else if (i < IT) load_matrices<false>(x[i], base + Stage::gy + i * plane_v + left_rows(lane, 16 * mi, 16 * s, lv));
          else x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0u;
        }
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int j = 0; j + i < NU; ++j) {
            multiply(acc[0], x[i], y[j][0], y[j][1]);
            multiply(acc[1], x[i], y[j][2], y[j][3]);
          }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * mi + g + (r >> 1) * 8, j = 16 * pj + 8 * n + 2 * t + (r & 1);
          float x = i >= j ? acc[n][r] * between(spots[i], spots[j]) : 0.f;
          x = is_x ? (i > j ? -x : 0.f) : a.scale * x;
          unsigned char* tile = shared + (is_x ? at.xs : at.da);
#pragma unroll
          for (int w = 0; w < NU; ++w) {
            const __nv_bfloat16 y = __float2bfloat16_rn(x);
            if (!is_x) *reinterpret_cast<__nv_bfloat16*>(tile + w * kLower + lower_at(i, j)) = y;
            if (is_x && i >= j) *reinterpret_cast<__nv_bfloat16*>(tile + w * 2048 + element_at(i, j, 2)) = y;
            if (is_x && i > j) *reinterpret_cast<__nv_bfloat16*>(tile + w * 2048 + element_at(j, i, 2)) = y;
            x -= __bfloat162float(y);
          }
        }
    }
    meet(1 + 2 * producers, 32 * W);
    // dQ and dK, 16 of their columns at a time
    for (int p = warp; p < DK / 16; p += W) {
      float aq[2][2][4], ak[2][2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) zero(aq[m]), zero(ak[m]);
      {
        float az[2][2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) zero(az[m]);
        for (int s = 0; s < W; ++s) {
          uint32_t bs[NS][4], bd[NS][4];
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const uint32_t to = j * W * 16 * DK * 2 + right_cols(lane, 16 * p, 16 * s, lp);
            load_matrices<true>(bs[j], sh + at.s + to);
            load_matrices<true>(bd[j], sh + at.ds + to);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t to = left_rows(lane, 16 * m, 16 * s, lv);
#pragma unroll
            for (int i = 0; i < NU; ++i) {
              uint32_t x[4];
              if (i < IT) {
                load_matrices<false>(x, base + Stage::gy + i * plane_v + to);
#pragma unroll
                for (int j = 0; j < NS && i + j < NU; ++j)
                  multiply(aq[m][0], x, bs[j][0], bs[j][1]), multiply(aq[m][1], x, bs[j][2], bs[j][3]);
              }
              load_matrices<false>(x, sh + at.dz + i * plane_v + to);
#pragma unroll
              for (int j = 0; j < NS && i + j < NU; ++j)
                multiply(az[m][0], x, bs[j][0], bs[j][1]), multiply(az[m][1], x, bs[j][2], bs[j][3]);
              load_matrices<false>(x, sh + at.u + i * plane_v + to);
#pragma unroll
              for (int j = 0; j < NS && i + j < NU; ++j)
                multiply(ak[m][0], x, bd[j][0], bd[j][1]), multiply(ak[m][1], x, bd[j][2], bd[j][3]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const Spot& s = spots[16 * m + g + (r >> 1) * 8];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              aq[m][n][r] *= a.scale * s.since;
              ak[m][n][r] = s.until * ak[m][n][r] - s.since * az[m][n][r];
            }
          }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t bk[IT][4], bq[IT][4];
#pragma unroll
        for (int j = 0; j < IT; ++j) {
          const uint32_t to = j * plane + right_cols(lane, 16 * p, 16 * s, lp);
          load_matrices<true>(bk[j], base + Stage::k + to);
          load_matrices<true>(bq[j], base + Stage::q + to);
        }
        const auto add = [&](float (&acc)[2][4], const uint32_t (&x)[4], const uint32_t (&y)[IT][4], int i) {
#pragma unroll
          for (int j = 0; j < IT; ++j)
            if (i + j < NU) multiply(acc[0], x, y[j][0], y[j][1]), multiply(acc[1], x, y[j][2], y[j][3]);
        };
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            uint32_t x[4];
            if (s <= m) {
              load_matrices<false>(x, sh + at.da + i * kLower + (m + s) * 512 + left_rows(lane, 0, 0, 1));
              add(aq[m], x, bk, i);
            }
            if (s >= m) {
              load_matrices<true>(x, sh + at.da + i * kLower + (m + s) * 512 + left_cols(lane, 0, 0, 1));
              add(ak[m], x, bq, i);
            }
            load_matrices<false>(x, sh + at.xs + i * 2048 + left_rows(lane, 16 * m, 16 * s, 2));
            add(ak[m], x, bk, i);
          }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * m + g + 8 * r;
          if (t0 + i >= a.len) continue;
          const bool on = i < live;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int d = 16 * p + 8 * n + 2 * t;
            const float2 x = on ? make_float2(aq[m][n][2 * r], aq[m][n][2 * r + 1]) : make_float2(0.f, 0.f);
            const float2 y = on ? make_float2(ak[m][n][2 * r], ak[m][n][2 * r + 1]) : make_float2(0.f, 0.f);
            if (a.share > 1) {
              const int64_t pos = ((int64_t)b * a.len + t0 + i) * a.heads + h;
              const int64_t all = (int64_t)a.batch * a.len * a.heads;
              *reinterpret_cast<float2*>(a.work.shared + pos * DK + d) = x;
              *reinterpret_cast<float2*>(a.work.shared + (all + pos) * DK + d) = y;
              continue;
            }
            T* tq = gq.data + b * gq.batch + (int64_t)(t0 + i) * gq.time + h * gq.head + d;
            T* tk = gk.data + b * gk.batch + (int64_t)(t0 + i) * gk.time + h * gk.head + d;
            if (a.wide_gy && d < a.key_dim) {
              Vec<T, 2> o;
              narrow2(o.e, x);
              store_vec(tq, o);
              narrow2(o.e, y);
              store_vec(tk, o);
            } else {
              if (d < a.key_dim) tq[0] = from_f32<T>(x.x), tk[0] = from_f32<T>(y.x);
              if (d + 1 < a.key_dim) tq[1] = from_f32<T>(x.y), tk[1] = from_f32<T>(y.y);
            }
          }
        }
    }
    if (c % kAgain == 0 && c > 0) find_along(c);
    if (n0 + producers < chunks) arrive(1 + producers + stage, meeting);
    stage = stage + 1 == producers ? 0 : stage + 1;
  }
  if (a.grad_state)
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
        if (d < a.key_dim && e < a.value_dim) a.grad_state[(head * a.key_dim + d) * a.value_dim + e] = dS[n][r];
      }
  // positions past the last chunk
  for (int64_t i = (int64_t)chunks * kChunk + warp; i < a.len; i += W) {
    T* to = gv.data + b * gv.batch + i * gv.time + h * gv.head;
    for (int e = lane; e < a.value_dim; e += 32) to[e] = from_f32<T>(0.f);
    if (a.share == 1) {
      T* tq = gq.data + b * gq.batch + i * gq.time + h * gq.head;
      T* tk = gk.data + b * gk.batch + i * gk.time + h * gk.head;
      for (int d = lane; d < a.key_dim; d += 32) tq[d] = tk[d] = from_f32<T>(0.f);
    }
    if (lane == 0) {
      a.grad_decay.data[b * a.grad_decay.batch + i * a.grad_decay.time + h * a.grad_decay.head] = 0.f;
      a.grad_beta.data[b * a.grad_beta.batch + i * a.grad_beta.time + h * a.grad_beta.head] = 0.f;
    }
  }
}

// A key head's gradients of q and k: the sum over its value heads, in their order.
template <class T>
__global__ void __launch_bounds__(256) k_delta_join(DeltaArgs a, int dk, DView<T> gq, DView<T> gk) {
  const int64_t rows = (int64_t)a.batch * a.len * a.heads, n = rows / a.share * a.key_dim;
  const int kh = a.heads / a.share;
  for (int64_t u = blockIdx.x * 256ll + threadIdx.x; u < n; u += gridDim.x * 256ll) {
    const int64_t r = u / a.key_dim, pos = r / kh, b = pos / a.len, i = pos - b * a.len;
    const int d = (int)(u - r * a.key_dim), j = (int)(r - pos * kh);
    float x = 0.f, y = 0.f;
    if (i < length_of(a, (int)b))
      for (int s = 0; s < a.share; ++s) {
        const int64_t from = (pos * a.heads + j * a.share + s) * dk + d;
        x += a.work.shared[from];
        y += a.work.shared[rows * dk + from];
      }
    gq.data[b * gq.batch + i * gq.time + j * gq.head + d] = from_f32<T>(x);
    gk.data[b * gk.batch + i * gk.time + j * gk.head + d] = from_f32<T>(y);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// The views of a call; grad_* of a backward only.
struct DeltaViews {
  const delta_view *q, *k, *v, *y, *gy, *gq, *gk, *gv;
};

template <class T>
DView<T> dview(const delta_view* v) {
  return v ? DView<T>{(T*)v->data, v->batch_stride, v->time_stride, v->head_stride} : DView<T>{nullptr, 0, 0, 0};
}

constexpr int kMostShared = 227 << 10;

template <class T, bool STATES, int DK>
cudaError_t launch_delta_fwd(const emb_delta_s* h, DeltaArgs a, const DeltaViews& w, cudaStream_t stream) {
  using Stage = ForwardStage<T, DK, STATES>;
  const int W = (a.value_dim + 15) / 16;
  const int64_t heads = (int64_t)a.batch * a.heads;
  // value channels over several CTAs where there are too few sequences for the SMs: each
  // finds the chunks' inverses for itself
  a.parts = 1;
  for (int d = 2; d <= W && heads * a.parts < h->sm_count; ++d)
    if (W % d == 0) a.parts = d;
  const int consumers = W / a.parts, own = consumers * kChunk * 17 * 4;
  const int64_t ctas = heads * a.parts;
  int producers = ctas > h->sm_count ? 2 : 4;
  while (producers > 1 && producers * Stage::bytes(16 * consumers) + own > kMostShared) --producers;
  const int smem = producers * Stage::bytes(16 * consumers) + own;
  const auto kernel = k_delta_fwd<T, DK, STATES>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)ctas, 32 * (consumers + producers), smem, stream>>>(
      a, dview<const T>(w.q), dview<const T>(w.k), dview<const T>(w.v), dview<const T>(w.gy), dview<T>(w.y), producers);
  return cudaGetLastError();
}

template <class T, int DK>
cudaError_t launch_delta_bwd(const emb_delta_s* h, const DeltaArgs& a, const DeltaViews& w, cudaStream_t stream) {
  cudaError_t e = launch_delta_fwd<T, true, DK>(h, a, w, stream);
  if (e != cudaSuccess) return e;
  const int W = (a.value_dim + 15) / 16;
  int dvp = 16;
  while (dvp < 16 * W) dvp *= 2;
  const ReverseShared<T, DK> at(W, dvp);
  int producers = 2;
  while (producers > 1 && producers * ReverseStage<T, DK>::bytes(dvp) + at.bytes > kMostShared) --producers;
  const int smem = producers * ReverseStage<T, DK>::bytes(dvp) + at.bytes;
  const auto kernel = k_delta_bwd<T, DK>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(a.batch * a.heads), 32 * (W + producers), smem, stream>>>(
      a, dview<const T>(w.q), dview<const T>(w.k), dview<const T>(w.v), dview<const T>(w.gy), dview<T>(w.gq),
      dview<T>(w.gk), dview<T>(w.gv), producers);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.share == 1 || a.len == 0) return e;
  const int64_t n = (int64_t)a.batch * a.len * (a.heads / a.share) * a.key_dim, need = (n + 255) / 256;
  const int64_t most = (int64_t)h->sm_count * 32;
  k_delta_join<T><<<(unsigned)(need < most ? need : most), 256, 0, stream>>>(a, DK, dview<T>(w.gq), dview<T>(w.gk));
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_delta(const emb_delta_s* h, const DeltaArgs& a, const DeltaViews& w, bool backward, cudaStream_t s) {
  const auto of = [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    return backward ? launch_delta_bwd<T, DK>(h, a, w, s) : launch_delta_fwd<T, false, DK>(h, a, w, s);
  };
  if (a.key_dim <= 32) return of(std::integral_constant<int, 32>());
  if (a.key_dim <= 64) return of(std::integral_constant<int, 64>());
  return of(std::integral_constant<int, 128>());
}

// One for each element type (delta_*.cu).
template <class T>
cudaError_t run_delta(const emb_delta_s* h, const DeltaArgs& a, const DeltaViews& w, bool backward, cudaStream_t s);
template <>
cudaError_t run_delta<__nv_bfloat16>(const emb_delta_s*, const DeltaArgs&, const DeltaViews&, bool, cudaStream_t);
template <>
cudaError_t run_delta<__half>(const emb_delta_s*, const DeltaArgs&, const DeltaViews&, bool, cudaStream_t);
template <>
cudaError_t run_delta<float>(const emb_delta_s*, const DeltaArgs&, const DeltaViews&, bool, cudaStream_t);

}  // namespace emb
