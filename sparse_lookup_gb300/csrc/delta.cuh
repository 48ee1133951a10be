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
// tile.  What follows from a chunk's keys, queries and decays alone (the inverse, A, M)
// is found before, all chunks at once, a warp each (k_delta_prepare): a warp needs some
// microseconds for it, and one that ran ahead of the consumers would hold them up.
// Producer warps, each with a stage of shared memory, copy a chunk's inputs and that
// record ahead of the consumers.
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
  unsigned char* record = nullptr;   // see DeltaWork
  int32_t* order = nullptr;          // [kMostOrdered]
  // for the backward
  uint4 *s[3] = {nullptr, nullptr, nullptr}, *ds[3] = {nullptr, nullptr, nullptr};
  float4 *e = nullptr, *dz = nullptr;
  float *sums = nullptr, *along = nullptr, *totals = nullptr;
  // for sequences in segments
  float *effect = nullptr, *between = nullptr;
  int64_t max_pairs = 0;
};

namespace emb {

constexpr int kChunk = 32;
constexpr int kMostOrdered = 4096;   // entries that are ordered by their length
constexpr int kLeastChunks = 64;   // of a sequence that is cut into segments

// A [batch, time, heads, dim] array (or [batch, time, heads]).
template <class T>
struct DView {
  T* data;
  int64_t batch, time, head;
};

// What the passes leave for each other, chunk after chunk of each (entry, head): a
// chunk's record, and for the backward states and intermediates in the order of the
// lanes' registers.
struct DeltaWork {
  unsigned char* record;   // [chunks][Record::bytes]
  uint4* s[3];             // [chunks + 1][warps][DK / 16][32]: the state before a chunk in bf16 terms
  uint4* ds[3];            // [chunks][warps][DK / 16][32]: the gradient of the state after it
  float4 *e, *dz;          // [chunks][warps][4][32]: E and dZ
  float* sums;             // [3][warps][chunks][32]: <grad_y, y>, <grad_v, v> and grad_beta over a warp's channels
  float* along;            // [chunks + 1][warps]: <dS, S> before a chunk, of every kAgain-th and the last
  float* totals;           // [chunks][warps]: the sum of <grad_y, y> - <grad_v, v> over a chunk
  int64_t chunks;          // batch * heads * chunks of an entry
  // [batch * heads * segments][channels][DK] floats: what a segment makes of a zero state and of
  // the identity; the state before a segment (its gradient after it)
  float *effect, *between;
};
constexpr int kAgain = 16;   // chunks between the states whose <dS, S> is taken

struct DeltaArgs {
  int32_t batch, len, heads, share;   // share: value heads of a key head
  int32_t key_dim, value_dim;
  int32_t chunks;                     // of an entry: (len + 31) / 32
  int32_t parts;                      // CTAs that share an (entry, head)'s value channels
  int32_t warps;                      // of 16 value channels, of all parts
  int32_t segments, span;             // of a sequence, and chunks of one
  float scale;
  const int32_t* offsets;
  const int32_t* order;               // NULL, or entries from the longest
  const float *state_in, *grad_last;
  float *state_out, *grad_state;
  DView<const float> decay, beta;
  DView<float> grad_decay, grad_beta;
  bool wide_qk, wide_v, wide_y, wide_gy;   // accesses of 16 bytes
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

// The way back, transposed: a lane's pairs to columns of rows of 8 elements; and as they are.
__device__ __forceinline__ void store_rows(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
               "r"(d) : "memory");
}
__device__ __forceinline__ void store_matrices(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
               "r"(d) : "memory");
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
      const float2 r = __ffma2_rn(unpack(t[i]), make_float2(-1.f, -1.f), make_float2(x, y));
      x = r.x, y = r.y;
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

// Addresses of the matrix loads of a lane in a tile that starts at a multiple of 256
// bytes: the first 16 x 16 elements' here, the others' by next().  X [n][k] as right
// operand (not transposed), X [k][n] (transposed); as left operand X [m][k] (not
// transposed), X [k][m] (transposed).
__device__ __forceinline__ uint32_t right_rows(int lane, int lp) {
  return piece((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1, lp);
}
__device__ __forceinline__ uint32_t right_cols(int lane, int lp) { return piece(lane & 15, lane >> 4, lp); }
__device__ __forceinline__ uint32_t left_rows(int lane, int lp) { return piece(lane & 15, lane >> 4, lp); }
__device__ __forceinline__ uint32_t left_cols(int lane, int lp) {
  return piece((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1, lp);
}
// 16 `rows` rows and 16 `cols` columns on: pieces are exchanged by their bits, so theirs are too.
__device__ __forceinline__ uint32_t next(uint32_t at, int rows, int cols, int lp) {
  return (at ^ (cols << 5)) + (rows << (lp + 8));
}

// acc += X Y over KS steps of 16.  left(s, a): the step's TA terms of X;
// right(p, s, j): address of term j of Y for the p-th 16 columns.  Products of
// terms i + j < N.  TRI 1: Y's steps s > p are zero, 2: s < p are.  Four accumulators
// in turn, as a matrix instruction's result takes that long.
template <int KS, int NP, int TA, int TB, int N, bool TRANS, int TRI, class L, class R>
__device__ __forceinline__ void product(float (&acc)[2 * NP][4], L left, R right) {
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint32_t a[TA][4];
    left(s, a);
#pragma unroll
    for (int p0 = 0; p0 < NP; p0 += 2) {
      const auto there = [&](int p) { return p < NP && !(TRI == 1 && s > p) && !(TRI == 2 && s < p); };
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        uint32_t b[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if (there(p0 + p)) load_matrices<TRANS>(b[p], right(p0 + p, s, j));
#pragma unroll
        for (int i = 0; i < TA; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if (i + j < N && there(p0 + p)) {
              multiply(acc[(2 * (p0 + p)) % (2 * NP)], a[i], b[p][0], b[p][1]);
              multiply(acc[(2 * (p0 + p) + 1) % (2 * NP)], a[i], b[p][2], b[p][3]);
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

// x = y times a pair of numbers a row pair (accumulators' columns).
__device__ __forceinline__ void times(float (&x)[4], const float (&y)[4], float2 f) {
  const float2 a = __fmul2_rn(make_float2(y[0], y[1]), f), b = __fmul2_rn(make_float2(y[2], y[3]), f);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// Sums over the eight lanes of equal lane % 4 of N values; lane keeps N / 8 of them: of
// N = 8 value 4 [lane & 16] + 2 [lane & 8] + [lane & 4], of N = 16 twice that and the next.
template <int N>
__device__ __forceinline__ void fold(float (&x)[N], int lane) {
#pragma unroll
  for (int o = 16, h = N / 2; o >= 4; o >>= 1, h >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = up ? x[i + h] : x[i], give = up ? x[i] : x[i + h];
      x[i] = keep + __shfl_xor_sync(kFull, give, o);
    }
  }
}
// The column of accumulators whose sums are value 2 n + r of 8 in that: 8 n + 2 t + r.
__device__ __forceinline__ int folded_column(int lane) {
  return ((lane & 16) ? 16 : 0) + ((lane & 8) ? 8 : 0) + 2 * (lane & 3) + ((lane & 4) ? 1 : 0);
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

// What follows from a chunk's keys, queries, decays and betas.
struct Record {
  // [32] floats each: exp(G_i), exp(G_31 - G_i), beta, and G_i as a multiple of 1/64 and the
  // rest (differences keep their digits beside a large G)
  static constexpr int since = 0, until = 128, beta = 256, g_hi = 384, g_lo = 512;
  // [3 terms] of lower triangular matrices
  static constexpr int inverse = 640, a = inverse + 3 * kLower, m = a + 3 * kLower, bytes = m + 3 * kLower;
  static constexpr int forward_bytes = m;   // M is the backward's
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

// A piece's terms to tiles `plane` bytes apart.
template <class T, int IT>
__device__ __forceinline__ void put_terms(unsigned char* to, int plane, const Eight<T>& x) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    *reinterpret_cast<uint4*>(to) = x.u[0];
  } else {
    uint32_t w[4][IT];
#pragma unroll
    for (int i = 0; i < 4; ++i) split<IT>(x.at(2 * i), x.at(2 * i + 1), w[i]);
#pragma unroll
    for (int i = 0; i < IT; ++i) *reinterpret_cast<uint4*>(to + i * plane) = make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
  }
}

__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Rows 0 .. 31 (`live` of them) of `cols` columns as bf16 terms in tiles `plane` bytes
// apart of 2^lp pieces a row.  Columns and rows beyond the array's are 0.
template <class T>
struct TileSource {
  unsigned char* tile;
  int plane, lp;
  const T* rows;
  int64_t stride;
  int cols;
  bool wide;
};

// N such tiles by one warp, all tiles' loads in flight together.  Aligned bf16 is only
// copied; copies_done() has to follow.
template <int IT, int N, class T>
__device__ __forceinline__ void load_tiles(const TileSource<T> (&x)[N], int live, int lane) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    bool wide = true;
#pragma unroll
    for (int w = 0; w < N; ++w) wide = wide && x[w].wide;
    if (wide) {
#pragma unroll
      for (int w = 0; w < N; ++w) {
        const uint32_t to = smem_of(x[w].tile);
        const int lp = x[w].lp;
#pragma unroll 4
        for (int u = lane; u < kChunk << lp; u += 32) {
          const int r = u >> lp, p = u & ((1 << lp) - 1);
          const bool on = r < live && p * 8 < x[w].cols;
          copy_async(to + piece(r, p, lp), on ? x[w].rows + r * x[w].stride + p * 8 : x[w].rows, on);
        }
      }
      return;
    }
  }
  constexpr int U = sizeof(T) == 2 || N <= 3 ? 4 : 2;
  int most = 0;
#pragma unroll
  for (int w = 0; w < N; ++w) most = max(most, kChunk << x[w].lp);
  for (int u0 = lane; u0 < most; u0 += 32 * U) {
    Eight<T> e[N][U];
#pragma unroll
    for (int w = 0; w < N; ++w)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = u0 + 32 * k, r = u >> x[w].lp, c = (u & ((1 << x[w].lp) - 1)) << 3;
        const T* from = x[w].rows + r * x[w].stride + c;
        if (r >= live || c >= x[w].cols) e[w][k].clear();
        else if (x[w].wide) e[w][k].load(from);
        else e[w][k].gather(from, x[w].cols - c);
      }
#pragma unroll
    for (int w = 0; w < N; ++w)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = u0 + 32 * k, lp = x[w].lp;
        if (u >= kChunk << lp) continue;
        put_terms<T, IT>(x[w].tile + piece(u >> lp, u & ((1 << lp) - 1), lp), x[w].plane, e[w][k]);
      }
  }
}

// One piece of such a tile: eight elements, `n` of them there.
template <class T, int IT>
__device__ __forceinline__ void put_eight(unsigned char* to, int plane, const T* from, int n, bool wide) {
  Eight<T> x;
  if (n <= 0) x.clear();
  else if (wide) x.load(from);
  else x.gather(from, n);
  put_terms<T, IT>(to, plane, x);
}

// X^T of such a tile in the layout of accumulators: rows are 16 of the tile's columns
// (`at` is left_cols' address of the first), columns its 32 rows.
template <int IT>
__device__ __forceinline__ void load_turned(float (&x)[4][4], uint32_t at, int plane, int lp) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t y[IT][4];
#pragma unroll
    for (int i = 0; i < IT; ++i) load_matrices<true>(y[i], next(at, s, 0, lp) + i * plane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = unpack(y[IT - 1][i]);
#pragma unroll
      for (int j = IT - 2; j >= 0; --j) {
        const float2 l = unpack(y[j][i]);
        f.x += l.x, f.y += l.y;
      }
      x[2 * s + (i >> 1)][2 * (i & 1)] = f.x, x[2 * s + (i >> 1)][2 * (i & 1) + 1] = f.y;
    }
  }
}

// 16 channels, e0 on, of 32 rows (`there` of them in the array, the live ones not 0) from a
// swizzled tile of 16-bit elements: two lanes a row, so that its 32 bytes leave together.
template <class T>
__device__ __forceinline__ void store_turned(const unsigned char* tile, T* rows, int64_t stride, int e0, int dim,
                                             int there, int live, bool wide, int lane) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = 16 * u + (lane >> 1), e = e0 + 8 * (lane & 1);
    if (r >= there) continue;
    Vec<T, 8> o = load_vec<T, 8>(reinterpret_cast<const T*>(tile + piece(r, lane & 1, 1)));
    if (r >= live)
#pragma unroll
      for (int i = 0; i < 8; ++i) o.e[i] = from_f32<T>(0.f);
    T* to = rows + r * stride + e;
    if (wide && e + 8 <= dim) {
      store_vec(to, o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < dim) to[i] = o.e[i];
    }
  }
}

__device__ __forceinline__ void copy_record(unsigned char* to, const unsigned char* from, int bytes, int lane) {
  const uint32_t at = smem_of(to);
#pragma unroll 4
  for (int u = lane * 16; u < bytes; u += 512) copy_async(at + u, from + u, true);
}

// A record's floats of a lane's columns 8 n + 2 t and the next.
__device__ __forceinline__ float2 pair_at(const unsigned char* record, int array, int n, int t) {
  return *reinterpret_cast<const float2*>(record + array + (8 * n + 2 * t) * 4);
}
__device__ __forceinline__ float float_at(const unsigned char* record, int array, int i) {
  return *reinterpret_cast<const float*>(record + array + i * 4);
}
// exp(G_i - G_j)
__device__ __forceinline__ float between(const unsigned char* record, int i, int j) {
  return expf((float_at(record, Record::g_hi, i) - float_at(record, Record::g_hi, j)) +
              (float_at(record, Record::g_lo, i) - float_at(record, Record::g_lo, j)));
}

// Neighbours of a row of a tile, as N terms `plane` bytes apart.
template <int N>
__device__ __forceinline__ void put_pair(unsigned char* at, int plane, float x, float y) {
  uint32_t t[N];
  split<N>(x, y, t);
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<uint32_t*>(at + i * plane) = t[i];
}

__device__ __forceinline__ int length_of(const DeltaArgs& a, int b) {
  if (!a.offsets) return a.len;
  const int64_t n = (int64_t)a.offsets[b + 1] - a.offsets[b];
  return n < 0 ? 0 : n < a.len ? (int)n : a.len;
}

// Entries from the longest, equal ones in their order: with more sequences than run at
// once, the last to start are then the short ones.
static __global__ void __launch_bounds__(256) k_delta_order(DeltaArgs a, int32_t* order) {
  __shared__ int32_t lens[256];
  const int b = blockIdx.x * 256 + threadIdx.x, mine = b < a.batch ? length_of(a, b) : 0;
  int rank = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 256) {
    __syncthreads();
    lens[threadIdx.x] = b0 + threadIdx.x < a.batch ? length_of(a, b0 + threadIdx.x) : -1;
    __syncthreads();
#pragma unroll 8
    for (int i = 0; i < 256; ++i) rank += lens[i] > mine || (lens[i] == mine && b0 + i < b);
  }
  if (b < a.batch) order[rank] = b;
}

constexpr int log_of(int n) { return n <= 1 ? 0 : 1 + log_of(n / 2); }
constexpr int kMostShared = 227 << 10;

// ---------------------------------------------------------------------------
// records
// ---------------------------------------------------------------------------

// A warp's shared memory: K and Q, then in their place the record's numbers and inverse,
// M diag(beta) of the two diagonal blocks in floats, and a block in terms.
template <class T, int DK>
struct PrepareShared {
  static constexpr int IT = Terms<T>::of(3), lp = log_of(DK / 8), plane = kChunk * DK * 2;
  static constexpr int tiles = 2 * IT * plane, m = Record::a, block = m + 2 * 16 * 20 * 4, rest = block + 3 * 512,
                       bytes = ((tiles > rest ? tiles : rest) + 255) / 256 * 256;
};

// A warp a chunk.  The inverse of I + N, N = M diag(beta) = [N11 0; N21 N22]: both
// diagonal blocks by forward substitution (column j of them in lane j and 16 + j; not by
// powers of N, which cancel where keys repeat), the block below them as -X22 N21 X11 on
// the matrix units.  32 sequences of 1024 .. 2048 positions, 8 heads of 128, bf16 (12.3
// thousand chunks, the workload of the figures below): 62 us, 2000 instructions a chunk.
template <class T, int DK>
__global__ void __launch_bounds__(384) k_delta_prepare(DeltaArgs a, DView<const T> q, DView<const T> k, int backward) {
  using Shared = PrepareShared<T, DK>;
  constexpr int IT = Shared::IT, lp = Shared::lp, plane = Shared::plane;
  extern __shared__ __align__(128) unsigned char held[];
  const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
  const uint32_t job = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (job >= a.work.chunks) return;
  const uint32_t bh = job / (uint32_t)a.chunks;
  const int c = (int)(job - bh * a.chunks), b = (int)(bh / (uint32_t)a.heads), h = (int)(bh - b * (uint32_t)a.heads);
  const int hk = h / a.share;
  const int len = length_of(a, b), t0 = c * kChunk, live = min(kChunk, len - t0), t = t0 + lane;
  if (live <= 0) return;
  unsigned char* mine = held + (threadIdx.x >> 5) * Shared::bytes;
  float g = lane < live ? a.decay.data[b * a.decay.batch + t * a.decay.time + h * a.decay.head] : 0.f;
  const float beta = lane < live ? a.beta.data[b * a.beta.batch + t * a.beta.time + h * a.beta.head] : 0.f;
  const TileSource<T> tiles[2] = {
      {mine, plane, lp, k.data + b * k.batch + t0 * k.time + hk * k.head, k.time, a.key_dim, a.wide_qk},
      {mine + IT * plane, plane, lp, q.data + b * q.batch + t0 * q.time + hk * q.head, q.time, a.key_dim, a.wide_qk}};
  load_tiles<IT>(tiles, live, lane);
  copies_done();
  __syncwarp();
  // lower blocks of K K^T and Q K^T: rows 0 .. 15 by columns 0 .. 15 (two accumulators),
  // rows 16 .. 31 by all (four)
  float kk[6][4], qk[6][4];
  zero(kk), zero(qk);
  const uint32_t kr = smem_of(mine) + right_rows(lane, lp), kl = smem_of(mine) + left_rows(lane, lp);
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    uint32_t bk[2][IT][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < IT; ++j) load_matrices<false>(bk[p][j], next(kr, p, s, lp) + j * plane);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        uint32_t x[4], y[4];
        load_matrices<false>(x, next(kl, m, s, lp) + i * plane);
        load_matrices<false>(y, next(kl, m, s, lp) + (IT + i) * plane);
#pragma unroll
        for (int p = 0; p <= m; ++p)
#pragma unroll
          for (int j = 0; j < IT && i + j < 3; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              multiply(kk[2 * (m + p) + n], x, bk[p][j][2 * n], bk[p][j][2 * n + 1]);
              multiply(qk[2 * (m + p) + n], y, bk[p][j][2 * n], bk[p][j][2 * n + 1]);
            }
      }
  }
  __syncwarp();
  // the positions: a decay below -512 counts as -512 (exp is 0 long before), so that
  // -infinity forgets and sums stay exact
  g = g < -512.f ? -512.f : g;
  float hi = rintf(g * 64.f) * 0.015625f, lo = g - hi;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(kFull, hi, o), y = __shfl_up_sync(kFull, lo, o);
    if (lane >= o) hi += x, lo += y;
  }
  const float end_hi = __shfl_sync(kFull, hi, 31), end_lo = __shfl_sync(kFull, lo, 31);
  float* numbers = reinterpret_cast<float*>(mine);
  numbers[Record::since / 4 + lane] = expf(hi) * expf(lo);
  numbers[Record::until / 4 + lane] = expf((end_hi - hi) + (end_lo - lo));
  numbers[Record::beta / 4 + lane] = beta;
  numbers[Record::g_hi / 4 + lane] = hi;
  numbers[Record::g_lo / 4 + lane] = lo;
  __syncwarp();
  float below[2][4];   // N21
  uint4* out = reinterpret_cast<uint4*>(a.work.record + (int64_t)job * Record::bytes);
  // a block that lies in terms at Shared::block to its place in the record
  const auto put_block = [&](int matrix, int blk) {
    __syncwarp();
    const uint4* in = reinterpret_cast<const uint4*>(mine + Shared::block);
#pragma unroll
    for (int j = 0; j < 3; ++j) out[(matrix + j * kLower + blk * 512) / 16 + lane] = in[j * 32 + lane];
    __syncwarp();
  };
#pragma unroll
  for (int blk = 0; blk < 3; ++blk) {
    float keys[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int u = 2 * blk + n, col = 16 * (blk >> 1) + 8 * n + 2 * t4, i = 16 * ((blk + 1) >> 1) + g4 + 8 * r;
        const float2 bj = *reinterpret_cast<const float2*>(mine + Record::beta + col * 4);
        const float d0 = i >= col ? between(mine, i, col) : 0.f, d1 = i > col ? between(mine, i, col + 1) : 0.f;
        put_pair<3>(mine + Shared::block + element_at(i & 15, col & 15, 1), 512, qk[u][2 * r] * d0 * a.scale,
                    qk[u][2 * r + 1] * d1 * a.scale);
        const float m0 = i > col ? kk[u][2 * r] * d0 : 0.f, m1 = i > col + 1 ? kk[u][2 * r + 1] * d1 : 0.f;
        keys[n][2 * r] = m0, keys[n][2 * r + 1] = m1;
        if (blk == 1) {
          below[n][2 * r] = m0 * bj.x, below[n][2 * r + 1] = m1 * bj.y;
        } else {
          float* at = reinterpret_cast<float*>(mine + Shared::m) + ((blk >> 1) * 16 + (i & 15)) * 20 + (col & 15);
          at[0] = m0 * bj.x, at[1] = m1 * bj.y;
        }
      }
    put_block(Record::a, blk);
    if (backward) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          put_pair<3>(mine + Shared::block + element_at(g4 + 8 * r, 8 * n + 2 * t4, 1), 512, keys[n][2 * r],
                      keys[n][2 * r + 1]);
      put_block(Record::m, blk);
    }
  }
  __syncwarp();
  {
    const float* n = reinterpret_cast<const float*>(mine + Shared::m) + (lane >> 4) * 320;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[4] = {i == (lane & 15) ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 w = *reinterpret_cast<const float4*>(n + i * 20 + l);
        s[0] -= w.x * x[l];
        if (l + 1 < i) s[1] -= w.y * x[l + 1];
        if (l + 2 < i) s[2] -= w.z * x[l + 2];
        if (l + 3 < i) s[3] -= w.w * x[l + 3];
      }
      x[i] = (s[0] + s[1]) + (s[2] + s[3]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      unsigned char* to = mine + Record::inverse + (lane >> 4) * 1024 + element_at(i, lane & 15, 1);
      float y = x[i];
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const __nv_bfloat16 e = __float2bfloat16_rn(y);
        *reinterpret_cast<__nv_bfloat16*>(to + j * kLower) = e;
        y -= __bfloat162float(e);
      }
    }
  }
  __syncwarp();
  const uint32_t inverse = smem_of(mine + Record::inverse), block = smem_of(mine + Shared::block);
  float x[2][4];
  zero(x);
  product<1, 1, 3, 3, 3, true, 0>(
      x, [&](int s, uint32_t (&y)[3][4]) { left_of<3>(below, s, y); },
      [&](int, int, int j) { return inverse + j * kLower + right_cols(lane, 1); });
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      put_pair<3>(mine + Shared::block + element_at(g4 + 8 * r, 8 * n + 2 * t4, 1), 512, x[n][2 * r], x[n][2 * r + 1]);
  __syncwarp();
  zero(x);
  product<1, 1, 3, 3, 3, true, 0>(
      x,
      [&](int, uint32_t (&y)[3][4]) {
#pragma unroll
        for (int i = 0; i < 3; ++i) load_matrices<false>(y[i], inverse + i * kLower + 1024 + left_rows(lane, 1));
      },
      [&](int, int, int j) { return block + j * 512 + right_cols(lane, 1); });
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      put_pair<3>(mine + Record::inverse + 512 + element_at(g4 + 8 * r, 8 * n + 2 * t4, 1), kLower, -x[n][2 * r],
                  -x[n][2 * r + 1]);
  __syncwarp();
  const uint4* in = reinterpret_cast<const uint4*>(mine);
  for (int u = lane; u < Record::a / 16; u += 32) out[u] = in[u];
}

// ---------------------------------------------------------------------------
// forward, and the states' pass before a backward
// ---------------------------------------------------------------------------

constexpr int kForwardTerms = 3;
// Terms of the states (and of their gradients) in the products that give the gradients
// of q and k: as many bits as those have.  A bf16 one rounds the states once, as its own
// store rounds it.  Where <dS, S> is taken the states are kept in three.
template <class T>
constexpr int kStateTerms = std::is_same_v<T, __nv_bfloat16> ? 1 : std::is_same_v<T, __half> ? 2 : 3;

enum DeltaMode {
  kForward,   // y and the last state
  kStates,    // what the reverse pass needs (DeltaWork)
  kEffect,    // what a segment makes of a zero state (value channels) and of the identity (key_dim channels more)
};

template <class T, int DK, DeltaMode MODE>
struct ForwardStage {
  static constexpr int NT = kForwardTerms, IT = Terms<T>::of(NT), lp = log_of(DK / 8), plane = kChunk * DK * 2;
  static constexpr int record = 0, k = (Record::forward_bytes + 255) / 256 * 256, q = k + IT * plane, v = q + IT * plane;
  // V (and grad_y) in terms, rows of dvp channels
  static constexpr int bytes(int dvp) { return v + (MODE == kStates ? 2 : 1) * IT * kChunk * dvp * 2; }
  // a warp's results on their way to rows: 16 bits swizzled, fp32 rows of 17
  static constexpr int own = MODE != kForward ? 0 : sizeof(T) == 2 ? 1024 : kChunk * 17 * 4;
};

// Consumer warps first (one for 16 value channels), then the producers.  A chunk's 310
// matrix instructions a warp (128 x 128, bf16) take 8.5 cycles each of a quarter of an SM,
// which bounds the workload above by 220 us; it takes 385 (states' pass 480): a warp's
// products follow from one another, and registers hold no more than two warps for each
// quarter.
template <class T, int DK, DeltaMode MODE>
__global__ void __launch_bounds__(384)
    k_delta_fwd(DeltaArgs a, DView<const T> q, DView<const T> k, DView<const T> v, DView<const T> gy, DView<T> y,
                int producers) {
  using Stage = ForwardStage<T, DK, MODE>;
  constexpr int NT = Stage::NT, IT = Stage::IT, lp = Stage::lp, plane = Stage::plane;
  // terms of what goes into y alone: 16 bits are stored of it, so two carry enough.  The
  // decays' gradients are sums of <grad_y, y> over many positions: all terms
  constexpr int NO = MODE == kForward && sizeof(T) == 2 ? 2 : NT;
  extern __shared__ __align__(128) unsigned char held[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int consumers = (blockDim.x >> 5) - producers, meeting = 32 * (consumers + 1);
  const int lv = consumers == 1 ? 1 : 32 - __clz(2 * consumers - 1), plane_v = (kChunk * 16) << lv;
  const int size = Stage::bytes(8 << lv);
  const int part = blockIdx.x % a.parts, pair = blockIdx.x / a.parts, seg = pair % a.segments, bh = pair / a.segments;
  const int nth = bh / a.heads, b = a.order ? a.order[nth] : nth, h = bh % a.heads, hk = h / a.share;
  const int first_v = part * 16 * consumers;
  const int len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk;
  // this segment's chunks; the last one that has any ends the sequence
  const int first = min(chunks, seg * a.span), end = min(chunks, first + a.span);
  const bool ends = seg == (chunks ? (chunks - 1) / a.span : 0);
  const int64_t head = (int64_t)b * a.heads + h;
  if (warp >= consumers) {
    const int p = warp - consumers, cols_v = max(0, min(16 * consumers, a.value_dim - first_v));
    unsigned char* st = held + p * size;
    for (int c = first + p; c < end; c += producers) {
      if (c >= first + producers) meet(1 + producers + p, meeting);
      const int t0 = c * kChunk, live = min(kChunk, len - t0);
      copy_record(st, a.work.record + (head * a.chunks + c) * Record::bytes, Record::forward_bytes, lane);
      const TileSource<T> kt{st + Stage::k, plane, lp, k.data + b * k.batch + t0 * k.time + hk * k.head, k.time,
                             a.key_dim, a.wide_qk};
      const TileSource<T> qt{st + Stage::q, plane, lp, q.data + b * q.batch + t0 * q.time + hk * q.head, q.time,
                             a.key_dim, a.wide_qk};
      const TileSource<T> vt{st + Stage::v, plane_v, lv, v.data + b * v.batch + t0 * v.time + h * v.head + first_v,
                             v.time, cols_v, a.wide_v};
      const TileSource<T> yt{st + Stage::v + IT * plane_v, plane_v, lv,
                             gy.data + b * gy.batch + t0 * gy.time + h * gy.head + first_v, gy.time, cols_v, a.wide_v};
      if constexpr (MODE == kStates) load_tiles<IT, 4, T>({kt, qt, vt, yt}, live, lane);
      else if constexpr (MODE == kForward) load_tiles<IT, 3, T>({kt, qt, vt}, live, lane);
      else load_tiles<IT, 2, T>({kt, vt}, live, lane);
      copies_done();
      arrive(1 + p, meeting);
    }
    return;
  }
  const int g = lane >> 2, t = lane & 3, e0 = first_v + 16 * warp;
  float S[DK / 8][4];   // S^T: channel e0 + g (+ 8), key columns 8 n + 2 t (+ 1)
#pragma unroll
  for (int n = 0; n < DK / 8; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
      if constexpr (MODE == kEffect)
        S[n][r] = e - 16 * a.warps == d ? 1.f : 0.f;
      else if (seg)
        S[n][r] = first < end ? a.work.between[((int64_t)pair * a.warps * 16 + e) * DK + d] : 0.f;
      else
        S[n][r] = a.state_in && d < a.key_dim && e < a.value_dim
                      ? a.state_in[(head * a.key_dim + d) * a.value_dim + e] : 0.f;
    }
  const int64_t warps = a.warps, mine = part * consumers + warp;
  const auto keep = [&](int c) {   // the state before chunk c, for the reverse pass
    const int64_t at = ((head * (a.chunks + 1) + c) * warps + mine) * (DK / 16) * 32 + lane;
    const bool all = c % kAgain == 0 || c == chunks;
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t x[3][4];
      left_of<3>(S, s, x);
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < kStateTerms<T> || all) a.work.s[j][at + s * 32] = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
    }
  };
  unsigned char* own = held + producers * size + warp * Stage::own;
  const uint32_t rows = right_rows(lane, lp), cols = right_cols(lane, lp);
  const uint32_t turned_v = next(left_cols(lane, lv), 0, warp, lv), low = right_rows(lane, 1);
  int stage = 0;
  for (int c = first; c < end; ++c) {
    unsigned char* st = held + stage * size;
    const uint32_t base = smem_of(st);
    if constexpr (MODE == kStates) keep(c);
    meet(1 + stage, meeting);
    const int t0 = c * kChunk, live = min(kChunk, len - t0);
    // K S0 and Q S0
    float Z[4][4], E[4][4], Y[4][4];
    zero(Z), zero(Y);
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t x[NT][4];
      left_of<NT>(S, s, x);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < IT; ++j) {
          uint32_t u[4], w[4];
          const uint32_t at = next(base + Stage::k + rows, p, s, lp) + j * plane;
          load_matrices<false>(u, at);
          if constexpr (MODE != kEffect) load_matrices<false>(w, at + IT * plane);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (i + j < NT) multiply(Z[2 * p], x[i], u[0], u[1]), multiply(Z[2 * p + 1], x[i], u[2], u[3]);
            if (MODE != kEffect && i + j < NO) multiply(Y[2 * p], x[i], w[0], w[1]), multiply(Y[2 * p + 1], x[i], w[2], w[3]);
          }
        }
    }
    // Z = V - exp(G) K S0
    load_turned<IT>(E, base + Stage::v + turned_v, plane_v, lv);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float2 f = pair_at(st, Record::since, n, t);
      Z[n][0] = E[n][0] - f.x * Z[n][0], Z[n][1] = E[n][1] - f.y * Z[n][1];
      Z[n][2] = E[n][2] - f.x * Z[n][2], Z[n][3] = E[n][3] - f.y * Z[n][3];
      times(Y[n], Y[n], make_float2(f.x * a.scale, f.y * a.scale));
    }
    const auto lower = [&](int tile, int p, int s, int j) {
      return base + low + tile + j * kLower + (p + s) * 512;
    };
    zero(E);
    product<2, 2, NT, NT, NT, false, 1>(
        E, [&](int s, uint32_t (&x)[NT][4]) { left_of<NT>(Z, s, x); },
        [&](int p, int s, int j) { return lower(Record::inverse, p, s, j); });
    if constexpr (MODE == kStates) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
        a.work.e[(((head * a.chunks + c) * warps + mine) * 4 + n) * 32 + lane] =
            make_float4(E[n][0], E[n][1], E[n][2], E[n][3]);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) times(E[n], E[n], pair_at(st, Record::beta, n, t));   // U
    if constexpr (MODE != kEffect) product<2, 2, NO, NO, NO, false, 1>(
        Y, [&](int s, uint32_t (&x)[NO][4]) { left_of<NO>(E, s, x); },
        [&](int p, int s, int j) { return lower(Record::a, p, s, j); });
    if constexpr (MODE == kStates) {
      // <grad_y, y> over the warp's channels
      float x[8];
      load_turned<IT>(Z, base + Stage::v + IT * plane_v + turned_v, plane_v, lv);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) x[2 * n + r] = Y[n][r] * Z[n][r] + Y[n][2 + r] * Z[n][2 + r];
      fold<8>(x, lane);
      a.work.sums[(mine * a.work.chunks + head * a.chunks + c) * kChunk + folded_column(lane)] = x[0];
    } else if constexpr (MODE == kForward) {
      // dead positions of the chunk too: 0
      if constexpr (sizeof(T) == 2) {
        const auto both = [](float lo, float hi) {
          Vec<T, 2> o;
          narrow2(o.e, make_float2(lo, hi));
          return *reinterpret_cast<const uint32_t*>(&o);
        };
#pragma unroll
        for (int s = 0; s < 2; ++s)
          store_matrices(next(smem_of(own) + left_cols(lane, 1), s, 0, 1), both(Y[2 * s][0], Y[2 * s][1]),
                         both(Y[2 * s][2], Y[2 * s][3]), both(Y[2 * s + 1][0], Y[2 * s + 1][1]),
                         both(Y[2 * s + 1][2], Y[2 * s + 1][3]));
        __syncwarp();
        store_turned(own, y.data + b * y.batch + (int64_t)t0 * y.time + h * y.head, y.time, e0, a.value_dim,
                     min(kChunk, a.len - t0), live, a.wide_y, lane);
      } else {
        float* turned = reinterpret_cast<float*>(own);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) turned[(8 * n + 2 * t + (r & 1)) * 17 + g + (r >> 1) * 8] = Y[n][r];
        __syncwarp();
        if (t0 + lane < a.len) {
          const bool on = lane < live;
          T* to = y.data + b * y.batch + (int64_t)(t0 + lane) * y.time + h * y.head + e0;
          const float* from = turned + lane * 17;
          if (a.wide_y && e0 + 16 <= a.value_dim) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              Vec<T, 4> o;
#pragma unroll
              for (int u = 0; u < 4; ++u) o.e[u] = on ? from[i + u] : 0.f;
              store_vec(to + i, o);
            }
          } else {
            for (int i = 0; i < 16 && e0 + i < a.value_dim; ++i) to[i] = on ? from[i] : 0.f;
          }
        }
      }
      __syncwarp();
    }
    // S1 = exp(G_31) S0 + K^T (exp(G_31 - G) U)
    const float whole = float_at(st, Record::since, kChunk - 1);
#pragma unroll
    for (int n = 0; n < 4; ++n) times(E[n], E[n], pair_at(st, Record::until, n, t));
#pragma unroll
    for (int n = 0; n < DK / 8; ++n) times(S[n], S[n], make_float2(whole, whole));
    product<2, DK / 16, NT, IT, NT, true, 0>(
        S, [&](int s, uint32_t (&x)[NT][4]) { left_of<NT>(E, s, x); },
        [&](int p, int s, int j) { return next(base + Stage::k + cols, s, p, lp) + j * plane; });
    if (c + producers < end) arrive(1 + producers + stage, meeting);
    stage = stage + 1 == producers ? 0 : stage + 1;
  }
  if constexpr (MODE == kEffect) {
    float* out = a.work.effect + ((int64_t)pair * (a.warps * 16 + DK) + e0 + g) * DK + 2 * t;
#pragma unroll
    for (int n = 0; n < DK / 8; ++n) {
      *reinterpret_cast<float2*>(out + 8 * n) = make_float2(S[n][0], S[n][1]);
      *reinterpret_cast<float2*>(out + 8 * DK + 8 * n) = make_float2(S[n][2], S[n][3]);
    }
  }
  if constexpr (MODE == kStates)
    if (ends) keep(chunks);
  if constexpr (MODE == kForward) {
    if (ends && a.state_out)
#pragma unroll
      for (int n = 0; n < DK / 8; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
          if (d < a.key_dim && e < a.value_dim) a.state_out[(head * a.key_dim + d) * a.value_dim + e] = S[n][r];
        }
    // positions past the last chunk, of this segment
    const int64_t from = (int64_t)kChunk * max(chunks, seg * a.span);
    const int64_t to = min((int64_t)a.len, (int64_t)kChunk * a.span * (seg + 1));
    for (int64_t i = from + (lane >> 4); i < to; i += 2)
      if (e0 + (lane & 15) < a.value_dim)
        y.data[b * y.batch + i * y.time + h * y.head + e0 + (lane & 15)] = from_f32<T>(0.f);
  }
}

// From segment to segment: S^T (rows are value channels) before each from what the one
// before makes of a state, S^T_p+1 = S^T_p M_p^T + N_p^T, with M^T and N^T as k_delta_fwd left them; or
// the gradients after each, dS^T_p-1 = dS^T_p M_p + N'_p^T.  A CTA has some rows; the
// next segment's M^T comes while this one's is used.  38 segments of 4 heads of 128 x 128:
// 76 us.
constexpr int chain_rows(int dk) { return dk == 128 ? 4 : 8; }
template <int DK, bool REVERSE>
__global__ void __launch_bounds__(256) k_delta_chain(DeltaArgs a) {
  constexpr int kRows = chain_rows(DK), G = 256 / DK, R = kRows / G, V = DK * DK / 1024;
  static_assert(R > 0 && G * R == kRows, "");
  extern __shared__ __align__(128) float chain[];
  float* m = chain;                // [DK][DK] M^T, groups of four exchanged by their row so that rows and columns are read alike
  float* x = chain + DK * DK;      // [kRows][DK]
  const int blocks = a.warps * 16 / kRows, rows0 = blockIdx.x % blocks * kRows, bh = blockIdx.x / blocks;
  const int b = bh / a.heads, len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk;
  const int last = chunks ? (chunks - 1) / a.span : 0, d = threadIdx.x % DK, r0 = threadIdx.x / DK * R;
  const float* given = REVERSE ? a.grad_last : a.state_in;
  // M^T follows N^T in a segment's effect of the forward; N'^T lies in another array of N^T's size
  const int64_t all = (int64_t)(a.warps * 16 + DK) * DK, some = (int64_t)a.warps * 16 * DK;
  const float* reversed = a.work.effect + (int64_t)a.batch * a.heads * a.segments * all;
  float4 next_m[V];
  float next_n[R];
  const auto fetch = [&](int p) {
    const int64_t pair = (int64_t)bh * a.segments + p;
    const float4* from = reinterpret_cast<const float4*>(a.work.effect + pair * all + some);
#pragma unroll
    for (int i = 0; i < V; ++i) next_m[i] = from[threadIdx.x + i * 256];
#pragma unroll
    for (int r = 0; r < R; ++r)
      next_n[r] = (REVERSE ? reversed + pair * some : a.work.effect + pair * all)[(int64_t)(rows0 + r0 + r) * DK + d];
  };
  if (last == 0) return;
  fetch(REVERSE ? last : 0);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = rows0 + r0 + r;
    x[(r0 + r) * DK + d] = given && d < a.key_dim && e < a.value_dim
                               ? given[((int64_t)bh * a.key_dim + d) * a.value_dim + e] : 0.f;
  }
  for (int n = 0; n < last; ++n) {
    const int p = REVERSE ? last - n : n, to = REVERSE ? p - 1 : p + 1;
    float acc[R];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = threadIdx.x + i * 256, row = u / (DK / 4), col = u % (DK / 4);
      *reinterpret_cast<float4*>(m + row * DK + ((col ^ (row & 7)) << 2)) = next_m[i];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = next_n[r];
    __syncthreads();
    if (n + 1 < last) fetch(to);
#pragma unroll 4
    for (int j = 0; j < DK; j += 4) {
      float w[4];
      if constexpr (REVERSE) {
        const float4 y = *reinterpret_cast<const float4*>(m + d * DK + (((j >> 2) ^ (d & 7)) << 2));
        w[0] = y.x, w[1] = y.y, w[2] = y.z, w[3] = y.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = m[(j + i) * DK + ((((d >> 2) ^ ((j + i) & 7)) << 2) | (d & 3))];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 y = *reinterpret_cast<const float4*>(x + (r0 + r) * DK + j);
        acc[r] += y.x * w[0] + y.y * w[1] + y.z * w[2] + y.w * w[3];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[(r0 + r) * DK + d] = acc[r];
      a.work.between[(((int64_t)bh * a.segments + to) * a.warps * 16 + rows0 + r0 + r) * DK + d] = acc[r];
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
//
// From the last chunk to the first, with dS the gradient of the state after the chunk,
// A^T dY and so on as above:
//   dU = A^T dY + diag(exp(G_31 - G)) K dS;  dE = diag(beta) dU;  dZ = (..)^-T dE = dV
//   dbeta = E . (dU - M^T dZ)                        (sums over the channels)
//   dS0 = exp(G_31) dS + Q^T (scale exp(G) dY) - K^T (exp(G) dZ)
// Value channels do not meet here either (k_delta_reverse, warps as in the forward).
// Then, all chunks at once (k_delta_gradients): dA = scale D o (dY U^T) and X = -D o (dZ
// U^T) below the diagonal,
//   dQ = scale exp(G) dY S0^T + dA K
//   dK = exp(G_31 - G) U dS^T - exp(G) dZ S0^T + dA^T Q + (X + X^T) K
// Decays: y and S1 are homogeneous in (S0, V), so dG_i = dY_i . Y_i - dV_i . V_i, and the
// gradient of g_t is their sum from t to the chunk's end and <dS, S1> there.  That number
// is the same sum over the chunks up to the next one where it is taken from the states:
// every sixteenth, before roundings add up.

template <class T, int DK>
struct ReverseStage {
  static constexpr int NR = 3, IT = Terms<T>::of(NR), lp = log_of(DK / 8), plane = kChunk * DK * 2;
  static constexpr int record = 0, k = (Record::bytes + 255) / 256 * 256, q = k + IT * plane, gy = q + IT * plane;
  static constexpr int bytes(int dvp) { return gy + 2 * IT * kChunk * dvp * 2; }   // grad_y and V
  static constexpr int own = sizeof(T) == 2 ? 1024 : 0;   // dV on its way to rows
};

// 378 matrix instructions a warp and chunk (128 x 128, bf16): 550 us of the workload above,
// where those alone would take 270.  EFFECT: only the gradient before a segment of a zero
// one after it.
template <class T, int DK, bool EFFECT>
__global__ void __launch_bounds__(384)
    k_delta_reverse(DeltaArgs a, DView<const T> q, DView<const T> k, DView<const T> v, DView<const T> gy, DView<T> gv,
                    int producers) {
  using Stage = ReverseStage<T, DK>;
  constexpr int IT = Stage::IT, lp = Stage::lp, plane = Stage::plane, NR = Stage::NR, NS = kStateTerms<T>;
  extern __shared__ __align__(128) unsigned char held[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int consumers = (blockDim.x >> 5) - producers, meeting = 32 * (consumers + 1);
  const int lv = consumers == 1 ? 1 : 32 - __clz(2 * consumers - 1), plane_v = (kChunk * 16) << lv;
  const int size = Stage::bytes(8 << lv);
  const int part = blockIdx.x % a.parts, pair = blockIdx.x / a.parts, seg = pair % a.segments, bh = pair / a.segments;
  const int nth = bh / a.heads, b = a.order ? a.order[nth] : nth, h = bh % a.heads, hk = h / a.share;
  const int first_v = part * 16 * consumers;
  const int len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk;
  const int first = min(chunks, seg * a.span), end = min(chunks, first + a.span);
  const bool ends = seg == (chunks ? (chunks - 1) / a.span : 0);
  const int64_t head = (int64_t)b * a.heads + h;
  if (warp >= consumers) {
    const int p = warp - consumers, cols_v = min(16 * consumers, a.value_dim - first_v);
    unsigned char* st = held + p * size;
    for (int n = p; n < end - first; n += producers) {
      if (n >= producers) meet(1 + producers + p, meeting);
      const int c = end - 1 - n, t0 = c * kChunk, live = min(kChunk, len - t0);
      copy_record(st, a.work.record + (head * a.chunks + c) * Record::bytes, Record::bytes, lane);
      const TileSource<T> kt{st + Stage::k, plane, lp, k.data + b * k.batch + t0 * k.time + hk * k.head, k.time,
                             a.key_dim, a.wide_qk};
      const TileSource<T> qt{st + Stage::q, plane, lp, q.data + b * q.batch + t0 * q.time + hk * q.head, q.time,
                             a.key_dim, a.wide_qk};
      const TileSource<T> yt{st + Stage::gy, plane_v, lv,
                             gy.data + b * gy.batch + t0 * gy.time + h * gy.head + first_v, gy.time, cols_v, a.wide_v};
      const TileSource<T> vt{st + Stage::gy + IT * plane_v, plane_v, lv,
                             v.data + b * v.batch + t0 * v.time + h * v.head + first_v, v.time, cols_v, a.wide_v};
      if constexpr (EFFECT) load_tiles<IT, 3, T>({kt, qt, yt}, live, lane);
      else load_tiles<IT, 4, T>({kt, qt, yt, vt}, live, lane);
      copies_done();
      arrive(1 + p, meeting);
    }
    return;
  }
  const int g = lane >> 2, t = lane & 3, e0 = first_v + 16 * warp;
  const int64_t warps = a.warps, mine = part * consumers + warp;
  float dS[DK / 8][4];
#pragma unroll
  for (int n = 0; n < DK / 8; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
      if constexpr (EFFECT)
        dS[n][r] = 0.f;
      else if (!ends)
        dS[n][r] = first < end ? a.work.between[((int64_t)pair * a.warps * 16 + e) * DK + d] : 0.f;
      else
        dS[n][r] = a.grad_last && d < a.key_dim && e < a.value_dim
                       ? a.grad_last[(head * a.key_dim + d) * a.value_dim + e] : 0.f;
    }
  const auto word = [](const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; };
  // <dS, S> before chunk c over the warp's channels
  const auto find_along = [&](int c) {
    const int64_t at = (head * (a.chunks + 1) + c) * warps + mine, from = at * (DK / 16) * 32 + lane;
    float x = 0.f;
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint4 u[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) u[j] = a.work.s[j][from + s * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f = unpack(word(u[2], i));
#pragma unroll
        for (int j = 1; j >= 0; --j) {
          const float2 w = unpack(word(u[j], i));
          f.x += w.x, f.y += w.y;
        }
        x += dS[2 * s + (i >> 1)][2 * (i & 1)] * f.x + dS[2 * s + (i >> 1)][2 * (i & 1) + 1] * f.y;
      }
    }
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    if (lane == 0) a.work.along[at] = x;
  };
  if (!EFFECT && ends) find_along(chunks);
  unsigned char* own = held + producers * size + warp * Stage::own;
  const uint32_t rows = right_rows(lane, lp), cols = right_cols(lane, lp);
  const uint32_t turned_v = next(left_cols(lane, lv), 0, warp, lv), low = right_cols(lane, 1);
  int stage = 0;
  for (int n0 = 0; n0 < end - first; ++n0) {
    const int c = end - 1 - n0, t0 = c * kChunk, live = min(kChunk, len - t0);
    unsigned char* st = held + stage * size;
    const uint32_t base = smem_of(st);
    const int64_t chunk = head * a.chunks + c, at_c = chunk * warps + mine;
    float4 e[4];   // E, from the states' pass
    float dots = 0.f;
    if constexpr (!EFFECT) {
#pragma unroll
      for (int n = 0; n < 4; ++n) e[n] = a.work.e[(at_c * 4 + n) * 32 + lane];
      dots = a.work.sums[(mine * a.work.chunks + chunk) * kChunk + folded_column(lane)];
    }
    meet(1 + stage, meeting);
    float dU[4][4], dZ[4][4], X[4][4];
    zero(dU);
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t x[NR][4];
      left_of<NR>(dS, s, x);
#pragma unroll
      for (int j = 0; j < (EFFECT ? 0 : NS); ++j)
        a.work.ds[j][at_c * (DK / 16) * 32 + s * 32 + lane] = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
#pragma unroll
      for (int j = 0; j < IT; ++j) {
        uint32_t u[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
          load_matrices<false>(u[p], next(base + Stage::k + rows, p, s, lp) + j * plane);
#pragma unroll
        for (int i = 0; i + j < NR; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            multiply(dU[2 * p], x[i], u[p][0], u[p][1]), multiply(dU[2 * p + 1], x[i], u[p][2], u[p][3]);
      }
    }
    const auto columns = [&](float (&x)[4][4], const float (&y)[4][4], int array) {   // x = y times a number a column
#pragma unroll
      for (int n = 0; n < 4; ++n) times(x[n], y[n], pair_at(st, array, n, t));
    };
    const auto lower = [&](int tile, int p, int s, int j) {
      return base + low + tile + j * kLower + (p + s) * 512;
    };
    columns(dU, dU, Record::until);
    product<2, 2, IT, NR, NR, true, 2>(
        dU,
        [&](int s, uint32_t (&x)[IT][4]) {
#pragma unroll
          for (int i = 0; i < IT; ++i)
            load_matrices<true>(x[i], next(base + Stage::gy + turned_v, s, 0, lv) + i * plane_v);
        },
        [&](int p, int s, int j) { return lower(Record::a, p, s, j); });
    columns(X, dU, Record::beta);
    zero(dZ);
    product<2, 2, NR, NR, NR, true, 2>(
        dZ, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(X, s, x); },
        [&](int p, int s, int j) { return lower(Record::inverse, p, s, j); });
    if constexpr (!EFFECT) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
      a.work.dz[(at_c * 4 + n) * 32 + lane] = make_float4(dZ[n][0], dZ[n][1], dZ[n][2], dZ[n][3]);
    zero(X);
    product<2, 2, NR, NR, NR, true, 2>(
        X, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(dZ, s, x); },
        [&](int p, int s, int j) { return lower(Record::m, p, s, j); });
    {
      float V[4][4];
      load_turned<IT>(V, base + Stage::gy + IT * plane_v + turned_v, plane_v, lv);
      float x[16];   // of a column: <grad_v, v>, grad_beta
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float E[4] = {e[n].x, e[n].y, e[n].z, e[n].w};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[4 * n + 2 * r] = dZ[n][r] * V[n][r] + dZ[n][2 + r] * V[n][2 + r];
          x[4 * n + 2 * r + 1] = E[r] * (dU[n][r] - X[n][r]) + E[2 + r] * (dU[n][2 + r] - X[n][2 + r]);
        }
      }
      fold<16>(x, lane);
      const int i = folded_column(lane);
      a.work.sums[((warps + mine) * a.work.chunks + chunk) * kChunk + i] = x[0];
      a.work.sums[((2 * warps + mine) * a.work.chunks + chunk) * kChunk + i] = x[1];
      float total = dots - x[0];   // a column each
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
      if (lane == 0) a.work.totals[at_c] = total;
    }
    // dV
    if constexpr (sizeof(T) == 2) {
      const auto both = [](float lo, float hi) {
        Vec<T, 2> o;
        narrow2(o.e, make_float2(lo, hi));
        return *reinterpret_cast<const uint32_t*>(&o);
      };
#pragma unroll
      for (int s = 0; s < 2; ++s)
        store_matrices(next(smem_of(own) + left_cols(lane, 1), s, 0, 1), both(dZ[2 * s][0], dZ[2 * s][1]),
                       both(dZ[2 * s][2], dZ[2 * s][3]), both(dZ[2 * s + 1][0], dZ[2 * s + 1][1]),
                       both(dZ[2 * s + 1][2], dZ[2 * s + 1][3]));
      __syncwarp();
      store_turned(own, gv.data + b * gv.batch + (int64_t)t0 * gv.time + h * gv.head, gv.time, e0, a.value_dim,
                   min(kChunk, a.len - t0), live, a.wide_y, lane);
      __syncwarp();
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
          if (t0 + i < a.len && e < a.value_dim)
            gv.data[b * gv.batch + (int64_t)(t0 + i) * gv.time + h * gv.head + e] = i < live ? dZ[n][r] : 0.f;
        }
    }
    }
    // the gradient of the state before the chunk
    const float whole = float_at(st, Record::since, kChunk - 1);
#pragma unroll
    for (int n = 0; n < DK / 8; ++n) times(dS[n], dS[n], make_float2(whole, whole));
    load_turned<IT>(X, base + Stage::gy + turned_v, plane_v, lv);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float2 f = pair_at(st, Record::since, n, t);
      times(X[n], X[n], make_float2(f.x * a.scale, f.y * a.scale));
      times(dZ[n], dZ[n], make_float2(-f.x, -f.y));
    }
    product<2, DK / 16, NR, IT, NR, true, 0>(
        dS, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(X, s, x); },
        [&](int p, int s, int j) { return next(base + Stage::q + cols, s, p, lp) + j * plane; });
    product<2, DK / 16, NR, IT, NR, true, 0>(
        dS, [&](int s, uint32_t (&x)[NR][4]) { left_of<NR>(dZ, s, x); },
        [&](int p, int s, int j) { return next(base + Stage::k + cols, s, p, lp) + j * plane; });
    if (n0 + producers < end - first) arrive(1 + producers + stage, meeting);
    stage = stage + 1 == producers ? 0 : stage + 1;
    if (!EFFECT && c % kAgain == 0 && c > 0) find_along(c);
  }
  if constexpr (EFFECT) {
    float* out = a.work.effect + (int64_t)a.batch * a.heads * a.segments * (a.warps * 16 + DK) * DK +
                 ((int64_t)pair * a.warps * 16 + e0 + g) * DK + 2 * t;
#pragma unroll
    for (int n = 0; n < DK / 8; ++n) {
      *reinterpret_cast<float2*>(out + 8 * n) = make_float2(dS[n][0], dS[n][1]);
      *reinterpret_cast<float2*>(out + 8 * DK + 8 * n) = make_float2(dS[n][2], dS[n][3]);
    }
  } else if (seg == 0 && a.grad_state) {
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 8 * n + 2 * t + (r & 1), e = e0 + g + (r >> 1) * 8;
        if (d < a.key_dim && e < a.value_dim) a.grad_state[(head * a.key_dim + d) * a.value_dim + e] = dS[n][r];
      }
  }
}

// The gradients of decays and betas: a warp a chunk, a lane a position.  The chunk's sums,
// and those of the chunks up to where <dS, S> is known.
static __global__ void __launch_bounds__(128) k_delta_numbers(DeltaArgs a) {
  const int lane = threadIdx.x & 31;
  const uint32_t chunk = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (chunk >= a.work.chunks) return;
  const uint32_t head = chunk / (uint32_t)a.chunks;
  const int c = (int)(chunk - head * a.chunks), b = (int)(head / (uint32_t)a.heads), h = (int)(head - b * (uint32_t)a.heads);
  const int len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk, W = a.warps;
  const int64_t i = (int64_t)c * kChunk + lane, stride = (int64_t)W * a.work.chunks * kChunk;
  float x = 0.f, gb = 0.f, g = 0.f;
  const bool on = i < len;
  if (c < chunks) {
    const float* sums = a.work.sums + (int64_t)chunk * kChunk + lane;
#pragma unroll 4
    for (int w = 0; w < W; ++w, sums += a.work.chunks * kChunk) x += sums[0] - sums[stride], gb += sums[2 * stride];
    if (on) g = a.decay.data[b * a.decay.batch + i * a.decay.time + h * a.decay.head];
    const int known = min(chunks, (c / kAgain + 1) * kAgain);
    float carry = 0.f;
    for (int n = (c + 1) * W + lane; n < known * W; n += 32) carry += a.work.totals[(int64_t)head * a.chunks * W + n];
    if (lane < W) carry += a.work.along[((int64_t)head * (a.chunks + 1) + known) * W + lane];
    for (int o = 16; o > 0; o >>= 1) carry += __shfl_xor_sync(kFull, carry, o);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(kFull, x, o);
      if (lane + o < 32) x += y;
    }
    x += carry;
  }
  if (i >= a.len) return;
  // where exp(g) is 0 so is its gradient, which the sums give to their rounding
  a.grad_decay.data[b * a.grad_decay.batch + i * a.grad_decay.time + h * a.grad_decay.head] =
      on && expf(g) != 0.f ? x : 0.f;
  a.grad_beta.data[b * a.grad_beta.batch + i * a.grad_beta.time + h * a.grad_beta.head] = on ? gb : 0.f;
}

// A CTA has a chunk of a key head and COLS of its channels.  In shared memory: S0 and dS
// [value channels][COLS], U and dZ [value channels][32], grad_y, K and Q, dA and X.  16-bit
// calls leave room for all channels; each CTA of a key head finds dA and X for itself.  630
// us of the workload above (reading 1.3 GB of states and intermediates, 190 us): loads,
// and the barriers around two short rounds of products, one CTA an SM.
template <class T, int DK>
struct GradientShared {
  static constexpr int COLS = DK == 128 && sizeof(T) == 4 ? 64 : DK, lc = log_of(COLS / 8);
  static constexpr int IT = Terms<T>::of(3), NS = kStateTerms<T>, NU = std::is_same_v<T, float> ? 3 : 2;
  static constexpr int warps = COLS / 8;   // 16 channels by 16 positions each
  static constexpr int plane = kChunk * COLS * 2;
  int s, ds, u, dz, gy, k, q, da, x, bytes;
  __host__ __device__ GradientShared(int W, int dvp) {
    s = 768;   // the record's numbers first
    ds = s + NS * W * 16 * COLS * 2;
    u = ds + NS * W * 16 * COLS * 2;
    dz = u + NU * W * 1024;
    gy = dz + NU * W * 1024;
    k = gy + IT * kChunk * dvp * 2;
    q = k + IT * plane;
    da = q + IT * plane;
    x = da + NU * kLower;
    bytes = x + NU * kLower;
  }
};

template <class T, int DK>
__global__ void __launch_bounds__(32 * GradientShared<T, DK>::warps, 16 / GradientShared<T, DK>::warps)
    k_delta_gradients(DeltaArgs a, DView<const T> q, DView<const T> k, DView<const T> gy, DView<T> gq, DView<T> gk,
                      DView<T> gv) {
  using Shared = GradientShared<T, DK>;
  constexpr int IT = Shared::IT, NS = Shared::NS, NU = Shared::NU, COLS = Shared::COLS, lc = Shared::lc,
                plane = Shared::plane, kWarps = Shared::warps, kThreads = 32 * kWarps;
  extern __shared__ __align__(128) unsigned char held[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int W = a.warps, lv = W == 1 ? 1 : 32 - __clz(2 * W - 1), plane_v = (kChunk * 16) << lv;
  const Shared at(W, 8 << lv);
  const int J = a.heads / a.share;
  const uint32_t job = blockIdx.x / (DK / COLS), bj = job / (uint32_t)a.chunks;
  const int col0 = (int)(blockIdx.x % (DK / COLS)) * COLS;
  const int c = (int)(job - bj * a.chunks), b = (int)(bj / (uint32_t)J), hk = (int)(bj - b * (uint32_t)J);
  const int len = length_of(a, b), chunks = (len + kChunk - 1) / kChunk, t0 = c * kChunk;
  const int live = min(kChunk, len - t0), there = min(kChunk, a.len - t0);
  if (live <= 0) {   // past the entry's end
    for (int i = warp; i < there; i += kWarps) {
      T* tq = gq.data + b * gq.batch + (int64_t)(t0 + i) * gq.time + hk * gq.head;
      T* tk = gk.data + b * gk.batch + (int64_t)(t0 + i) * gk.time + hk * gk.head;
      for (int d = col0 + lane; d < min(a.key_dim, col0 + COLS); d += 32) tq[d] = tk[d] = from_f32<T>(0.f);
      if (col0) continue;
      for (int h = hk * a.share; h < (hk + 1) * a.share; ++h) {
        T* to = gv.data + b * gv.batch + (int64_t)(t0 + i) * gv.time + h * gv.head;
        for (int e = lane; e < a.value_dim; e += 32) to[e] = from_f32<T>(0.f);
      }
    }
    return;
  }
  const uint32_t sh = smem_of(held);
  // this warp's part of dQ and dK: positions 16 m .., channels col0 + 16 p ..
  const int m = warp & 1, p = warp >> 1;
  float sq[2][4], sk[2][4];
  zero(sq), zero(sk);
  const int cols = min(COLS, max(0, a.key_dim - col0));
  // K and Q: a stripe of the rows for each warp
  for (int w = 0; w < 2; ++w) {
    const DView<const T>& x = w ? q : k;
    const T* rows = x.data + b * x.batch + t0 * x.time + hk * x.head + col0;
    unsigned char* tile = held + (w ? at.q : at.k);
    for (int u = threadIdx.x; u < kChunk << lc; u += kThreads) {
      const int r = u >> lc, n = u & ((1 << lc) - 1);
      const bool on = r < live && n * 8 < cols;
      if constexpr (std::is_same_v<T, __nv_bfloat16>)
        if (a.wide_qk) {
          copy_async(smem_of(tile) + piece(r, n, lc), on ? rows + r * x.time + n * 8 : rows, on);
          continue;
        }
      put_eight<T, IT>(tile + piece(r, n, lc), plane, rows + r * x.time + n * 8, on ? cols - n * 8 : 0, a.wide_qk);
    }
  }
  for (int hs = 0; hs < a.share; ++hs) {
    const int h = hk * a.share + hs;
    const int64_t head = (int64_t)b * a.heads + h, chunk = head * a.chunks + c;
    if (hs) __syncthreads();   // every warp is through with the head before
    const unsigned char* record = a.work.record + chunk * Record::bytes;
    if (threadIdx.x < 40) copy_async(sh + threadIdx.x * 16, record + threadIdx.x * 16, true);
    for (int u = threadIdx.x; u < kChunk << lv; u += kThreads) {
      const int r = u >> lv, n = u & ((1 << lv) - 1);
      const bool on = r < live && n * 8 < a.value_dim;
      const T* rows = gy.data + b * gy.batch + t0 * gy.time + h * gy.head;
      if constexpr (std::is_same_v<T, __nv_bfloat16>)
        if (a.wide_v) {
          copy_async(sh + at.gy + piece(r, n, lv), on ? rows + r * gy.time + n * 8 : rows, on);
          continue;
        }
      put_eight<T, IT>(held + at.gy + piece(r, n, lv), plane_v, rows + r * gy.time + n * 8, on ? a.value_dim - n * 8 : 0,
                       a.wide_v);
    }
    // E and dZ, and the states, a lane's four words of 16 channels by 16 key channels: as many of
    // a thread's loads as registers hold are in flight before the first is stored
    constexpr int UE = 2, US = NS == 1 ? 4 : NS == 2 ? 2 : 1;
    float4 e[UE], z[UE];
    float2 f[UE];
    const auto load_e = [&](int u0) {
#pragma unroll
      for (int n = 0; n < UE; ++n) {
        const int u = u0 + n * kThreads;
        if (u >= W * 128) continue;
        e[n] = a.work.e[chunk * W * 128 + u];
        z[n] = a.work.dz[chunk * W * 128 + u];
        f[n] = *reinterpret_cast<const float2*>(record + Record::beta + (8 * ((u >> 5) & 3) + 2 * (u & 3)) * 4);
      }
    };
    load_e(threadIdx.x);
    for (int u0 = threadIdx.x; u0 < W * (COLS / 16) * 32; u0 += US * kThreads) {
      uint4 x[2][US][NS];
#pragma unroll
      for (int n = 0; n < US; ++n) {
        const int u = u0 + n * kThreads, l = u & 31, s = (u >> 5) % (COLS / 16), w = (u >> 5) / (COLS / 16);
        if (u >= W * (COLS / 16) * 32) continue;
        const int64_t of = (int64_t)(w * (DK / 16) + col0 / 16 + s) * 32 + l;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          x[0][n][j] = a.work.s[j][(head * (a.chunks + 1) + c) * W * (DK / 16) * 32 + of];
          x[1][n][j] = a.work.ds[j][chunk * W * (DK / 16) * 32 + of];
        }
      }
#pragma unroll
      for (int n = 0; n < US; ++n) {
        const int u = u0 + n * kThreads, l = u & 31, s = (u >> 5) % (COLS / 16), w = (u >> 5) / (COLS / 16);
        if (u >= W * (COLS / 16) * 32) continue;
        // words of rows 8 apart and of neighbouring pieces
        const uint32_t first = element_at(16 * w + (l >> 2), 16 * s + 2 * (l & 3), lc), second = first ^ 16u;
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            unsigned char* to = held + (k ? at.ds : at.s) + j * W * 16 * COLS * 2;
            *reinterpret_cast<uint32_t*>(to + first) = x[k][n][j].x;
            *reinterpret_cast<uint32_t*>(to + first + 16 * COLS) = x[k][n][j].y;
            *reinterpret_cast<uint32_t*>(to + second) = x[k][n][j].z;
            *reinterpret_cast<uint32_t*>(to + second + 16 * COLS) = x[k][n][j].w;
          }
      }
    }
    for (int u0 = threadIdx.x; u0 < W * 128; u0 += UE * kThreads) {
      if (u0 != threadIdx.x) load_e(u0);
#pragma unroll
      for (int n = 0; n < UE; ++n) {
        const int u = u0 + n * kThreads, l = u & 31, col = 8 * ((u >> 5) & 3) + 2 * (l & 3), row = 16 * (u >> 7) + (l >> 2);
        if (u >= W * 128) continue;
        const uint32_t r0 = element_at(row, col, 2), r1 = r0 + 512;
        put_pair<NU>(held + at.u + r0, W * 1024, e[n].x * f[n].x, e[n].y * f[n].y);
        put_pair<NU>(held + at.u + r1, W * 1024, e[n].z * f[n].x, e[n].w * f[n].y);
        put_pair<NU>(held + at.dz + r0, W * 1024, z[n].x, z[n].y);
        put_pair<NU>(held + at.dz + r1, W * 1024, z[n].z, z[n].w);
      }
    }
    copies_done();
    __syncthreads();
    // dA and X, a 16 x 16 block at a time
    for (int u = warp; u < 6; u += kWarps) {
      const bool is_x = u >= 3;
      const int blk = is_x ? u - 3 : u, mi = (blk + 1) >> 1, pj = blk >> 1;
      float acc[2][4];
      zero(acc);
      const uint32_t right = next(sh + at.u + right_cols(lane, 2), 0, pj, 2);
      const uint32_t left = is_x ? next(sh + at.dz + left_cols(lane, 2), 0, mi, 2) : next(sh + at.gy + left_rows(lane, lv), mi, 0, lv);
      for (int s = 0; s < W; ++s) {
        uint32_t y[NU][4];
#pragma unroll
        for (int j = 0; j < NU; ++j) load_matrices<true>(y[j], next(right, s, 0, 2) + j * W * 1024);
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          uint32_t x[4];
          if (is_x) load_matrices<true>(x, next(left, s, 0, 2) + i * W * 1024);
          else if (i < IT) load_matrices<false>(x, next(left, 0, s, lv) + i * plane_v);
          else continue;
#pragma unroll
          for (int j = 0; j + i < NU; ++j) multiply(acc[0], x, y[j][0], y[j][1]), multiply(acc[1], x, y[j][2], y[j][3]);
        }
      }
      uint32_t out[4][NU];   // pairs of rows g and g + 8, of columns 2 t and 8 + 2 t
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * mi + g + 8 * r, j = 16 * pj + 8 * n + 2 * t;
          float x = i >= j ? acc[n][2 * r] * between(held, i, j) : 0.f;
          float y = i > j ? acc[n][2 * r + 1] * between(held, i, j + 1) : 0.f;
          if (is_x) x = i > j ? -x : 0.f, y = i > j + 1 ? -y : 0.f;
          else x *= a.scale, y *= a.scale;
          split<NU>(x, y, out[2 * n + r]);
        }
#pragma unroll
      for (int w = 0; w < NU; ++w)
        store_rows(sh + (is_x ? at.x : at.da) + w * kLower + blk * 512 + left_rows(lane, 1), out[0][w], out[1][w],
                   out[2][w], out[3][w]);
    }
    {
      float aq[2][4], ak[2][4], az[2][4];
      zero(aq), zero(ak), zero(az);
      const uint32_t states = next(sh + at.s + right_cols(lane, lc), 0, p, lc);
      const uint32_t us = next(sh + at.u + left_cols(lane, 2), 0, m, 2);
      const uint32_t ys = next(sh + at.gy + left_rows(lane, lv), m, 0, lv);
      for (int s = 0; s < W; ++s) {
        uint32_t bs[NS][4], bd[NS][4];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const uint32_t to = next(states, s, 0, lc) + j * W * 16 * COLS * 2;
          load_matrices<true>(bs[j], to);
          load_matrices<true>(bd[j], to + at.ds - at.s);
        }
        const uint32_t to = next(us, s, 0, 2);
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          uint32_t x[4];
          if (i < IT) {
            load_matrices<false>(x, next(ys, 0, s, lv) + i * plane_v);
#pragma unroll
            for (int j = 0; j < NS && i + j < NU; ++j)
              multiply(aq[0], x, bs[j][0], bs[j][1]), multiply(aq[1], x, bs[j][2], bs[j][3]);
          }
          load_matrices<true>(x, to + i * W * 1024 + at.dz - at.u);
#pragma unroll
          for (int j = 0; j < NS && i + j < NU; ++j)
            multiply(az[0], x, bs[j][0], bs[j][1]), multiply(az[1], x, bs[j][2], bs[j][3]);
          load_matrices<true>(x, to + i * W * 1024);
#pragma unroll
          for (int j = 0; j < NS && i + j < NU; ++j)
            multiply(ak[0], x, bd[j][0], bd[j][1]), multiply(ak[1], x, bd[j][2], bd[j][3]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * m + g + (r >> 1) * 8;
        const float since = float_at(held, Record::since, i), until = float_at(held, Record::until, i);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          sq[n][r] += a.scale * since * aq[n][r];
          sk[n][r] += until * ak[n][r] - since * az[n][r];
        }
      }
    }
    __syncthreads();   // dA and X are there
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t bk[IT][4], bq[IT][4];
#pragma unroll
      for (int j = 0; j < IT; ++j) {
        const uint32_t to = next(sh + at.k + right_cols(lane, lc), s, p, lc) + j * plane;
        load_matrices<true>(bk[j], to);
        load_matrices<true>(bq[j], to + IT * plane);
      }
      const auto add = [&](float (&acc)[2][4], const uint32_t (&x)[4], const uint32_t (&y)[IT][4], int i) {
#pragma unroll
        for (int j = 0; j < IT; ++j)
          if (i + j < NU) multiply(acc[0], x, y[j][0], y[j][1]), multiply(acc[1], x, y[j][2], y[j][3]);
      };
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        uint32_t x[4];
        const uint32_t to = sh + at.da + i * kLower + (m + s) * 512;
        if (s <= m) {
          load_matrices<false>(x, to + left_rows(lane, 1));
          add(sq, x, bk, i);
          load_matrices<false>(x, to + at.x - at.da + left_rows(lane, 1));
          add(sk, x, bk, i);
        }
        if (s >= m) {
          load_matrices<true>(x, to + left_cols(lane, 1));
          add(sk, x, bq, i);
          load_matrices<true>(x, to + at.x - at.da + left_cols(lane, 1));
          add(sk, x, bk, i);
        }
      }
    }
  }
  // to rows by way of shared memory, so that whole sectors leave
  __syncthreads();
  constexpr int V = 16 / sizeof(T), pieces = COLS / V;
  const auto place = [](int row, int p) { return (row * pieces + (p ^ (row & (pieces < 8 ? pieces - 1 : 7)))) * 16; };
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int col = 16 * p + 8 * n + 2 * t;
        Vec<T, 2> o;
        narrow2(o.e, w ? make_float2(sk[n][2 * r], sk[n][2 * r + 1]) : make_float2(sq[n][2 * r], sq[n][2 * r + 1]));
        store_vec(reinterpret_cast<T*>(held + w * kChunk * COLS * sizeof(T) + place(16 * m + g + 8 * r, col / V)) + col % V, o);
      }
  __syncthreads();
  for (int u = threadIdx.x; u < 2 * kChunk * pieces; u += kThreads) {
    const int w = u / (kChunk * pieces), i = u / pieces % kChunk, n = u % pieces, d = col0 + n * V;
    if (i >= there || d >= a.key_dim) continue;
    Vec<T, V> o = load_vec<T, V>(reinterpret_cast<const T*>(held + w * kChunk * COLS * sizeof(T) + place(i, n)));
    if (i >= live)
#pragma unroll
      for (int e = 0; e < V; ++e) o.e[e] = from_f32<T>(0.f);
    const DView<T>& to = w ? gk : gq;
    T* at = to.data + b * to.batch + (int64_t)(t0 + i) * to.time + hk * to.head + d;
    if (a.wide_gy) {
      store_vec(at, o);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (d + e < a.key_dim) at[e] = o.e[e];
    }
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

template <class T, int DK>
cudaError_t launch_delta_prepare(const DeltaArgs& a, const DeltaViews& w, bool backward, cudaStream_t stream) {
  if (a.work.chunks == 0) return cudaSuccess;
  const int most = kMostShared / PrepareShared<T, DK>::bytes, warps = most < 4 ? most : 4;
  const int smem = warps * PrepareShared<T, DK>::bytes;
  const auto kernel = k_delta_prepare<T, DK>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)((a.work.chunks + warps - 1) / warps), 32 * warps, smem, stream>>>(
      a, dview<const T>(w.q), dview<const T>(w.k), backward);
  return cudaGetLastError();
}

// CTAs, warps and stages of the kernels that walk along time, over `blocks` of 16 channels.
struct DeltaShape {
  int consumers, producers, smem;
  unsigned ctas;
};
template <class Stage>
DeltaShape walk_shape(const emb_delta_s* h, DeltaArgs& a, int blocks) {
  const int64_t pairs = (int64_t)a.batch * a.heads * a.segments;
  // channels over several CTAs where there are fewer than two sequences for an SM (a CTA's
  // warps are faster alone, so the last ones do not last: 256 heads of 128 x 128 forward 431
  // us in one CTA each, 385 in two, 450 in four, which copy keys and queries as often), and
  // where there are more than eight warps' of them
  a.parts = 1;
  for (int d = 2; d <= blocks && (pairs * a.parts < 2 * h->sm_count || blocks / a.parts > 8); ++d)
    if (blocks % d == 0) a.parts = d;
  DeltaShape s;
  const auto shape = [&](int most_producers) {
    s.consumers = blocks / a.parts;
    s.ctas = (unsigned)(pairs * a.parts);
    int dvp = 16;
    while (dvp < 16 * s.consumers) dvp *= 2;
    const int own = s.consumers * Stage::own;
    // a producer without a chunk would hold shared memory that another CTA can have (886 x 3
    // positions of 8 heads of 123 x 16 fp32, forward 459 us with two, 215 with one)
    s.producers = most_producers < a.span ? most_producers : a.span;
    while (s.producers > 1 && s.producers * Stage::bytes(dvp) + own > kMostShared) --s.producers;
    s.smem = s.producers * Stage::bytes(dvp) + own;
  };
  // six or eight warps' channels over two CTAs also where there are many sequences, if an SM
  // has shared memory for both: one's start and end then lie beside the other's chunks
  // (1024 heads of 64 x 128 fp16, 300 positions, forward + backward 2184 us in one, 1882 in
  // two; fp32 of 128 x 128, where only one fits, 4578 and 5503)
  if (a.parts == 1 && blocks >= 6 && blocks % 2 == 0) {
    a.parts = 2;
    shape(2);
    if (2 * s.smem > kMostShared) a.parts = 1;
  }
  shape(pairs * a.parts > h->sm_count ? 2 : 4);
  return s;
}

// Long sequences of few heads go in segments, all at once: first what each makes of any
// state (twice a walk's work), then from one to the next, then the walk itself.
template <int DK>
void cut_segments(const emb_delta_s* h, DeltaArgs& a) {
  a.segments = 1, a.span = a.chunks > 0 ? a.chunks : 1;
  const int64_t heads = (int64_t)a.batch * a.heads;
  if (heads * 4 > h->sm_count || a.chunks < kLeastChunks || !h->effect) return;
  // an SM each, but no more than the way from one to the next makes up for: a step of that
  // takes 2.7 us and a walk's chunk 4.3 (1024 chunks of 4 heads of 128 bf16, forward + backward:
  // 38 segments 1.49 ms, 19 1.72)
  int64_t n = h->sm_count / heads;
  while (2 * n * n > 3 * (int64_t)a.chunks) --n;
  if (n * heads > h->max_pairs) n = h->max_pairs / heads;
  if (n < 2) return;
  a.span = (int)((a.chunks + n - 1) / n);
  a.segments = (a.chunks + a.span - 1) / a.span;
}

template <class T, int DK, DeltaMode MODE>
cudaError_t launch_walk(const emb_delta_s* h, DeltaArgs a, const DeltaViews& w, cudaStream_t stream) {
  const int blocks = a.warps + (MODE == kEffect ? DK / 16 : 0);
  const DeltaShape s = walk_shape<ForwardStage<T, DK, MODE>>(h, a, blocks);
  const auto kernel = k_delta_fwd<T, DK, MODE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem);
  if (e != cudaSuccess) return e;
  kernel<<<s.ctas, 32 * (s.consumers + s.producers), s.smem, stream>>>(
      a, dview<const T>(w.q), dview<const T>(w.k), dview<const T>(w.v), dview<const T>(w.gy), dview<T>(w.y),
      s.producers);
  return cudaGetLastError();
}

template <int DK, bool REVERSE>
cudaError_t launch_chain(const DeltaArgs& a, cudaStream_t stream) {
  constexpr int smem = (DK + chain_rows(DK)) * DK * 4;
  const auto kernel = k_delta_chain<DK, REVERSE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(a.batch * a.heads * (a.warps * 16 / chain_rows(DK))), 256, smem, stream>>>(a);
  return cudaGetLastError();
}

template <class T, int DK, DeltaMode MODE>
cudaError_t launch_delta_fwd(const emb_delta_s* h, DeltaArgs& a, const DeltaViews& w, cudaStream_t stream) {
  cut_segments<DK>(h, a);
  if (a.offsets && a.len > kChunk && a.batch <= kMostOrdered && (int64_t)a.batch * a.heads > h->sm_count) {
    k_delta_order<<<(a.batch + 255) / 256, 256, 0, stream>>>(a, h->order);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    a.order = h->order;
  }
  cudaError_t e = launch_delta_prepare<T, DK>(a, w, MODE == kStates, stream);
  if (e == cudaSuccess && a.segments > 1) e = launch_walk<T, DK, kEffect>(h, a, w, stream);
  if (e == cudaSuccess && a.segments > 1) e = launch_chain<DK, false>(a, stream);
  return e == cudaSuccess ? launch_walk<T, DK, MODE>(h, a, w, stream) : e;
}

template <class T, int DK, bool EFFECT>
cudaError_t launch_reverse(const emb_delta_s* h, DeltaArgs a, const DeltaViews& w, cudaStream_t stream) {
  const DeltaShape s = walk_shape<ReverseStage<T, DK>>(h, a, a.warps);
  const auto kernel = k_delta_reverse<T, DK, EFFECT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem);
  if (e != cudaSuccess) return e;
  kernel<<<s.ctas, 32 * (s.consumers + s.producers), s.smem, stream>>>(
      a, dview<const T>(w.q), dview<const T>(w.k), dview<const T>(w.v), dview<const T>(w.gy), dview<T>(w.gv),
      s.producers);
  return cudaGetLastError();
}

template <class T, int DK>
cudaError_t launch_delta_bwd(const emb_delta_s* h, DeltaArgs a, const DeltaViews& w, cudaStream_t stream) {
  cudaError_t e = launch_delta_fwd<T, DK, kStates>(h, a, w, stream);
  if (e == cudaSuccess && a.segments > 1) e = launch_reverse<T, DK, true>(h, a, w, stream);
  if (e == cudaSuccess && a.segments > 1) e = launch_chain<DK, true>(a, stream);
  if (e == cudaSuccess) e = launch_reverse<T, DK, false>(h, a, w, stream);
  if (e != cudaSuccess || a.chunks == 0) return e;
  k_delta_numbers<<<(unsigned)((a.work.chunks + 3) / 4), 128, 0, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  using Shared = GradientShared<T, DK>;
  int dvp = 16;
  while (dvp < 16 * a.warps) dvp *= 2;
  const int smem = Shared(a.warps, dvp).bytes;
  const auto gradients = k_delta_gradients<T, DK>;
  e = cudaFuncSetAttribute(gradients, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  gradients<<<(unsigned)(a.work.chunks / a.share * (DK / Shared::COLS)), 32 * Shared::warps, smem, stream>>>(
      a, dview<const T>(w.q), dview<const T>(w.k), dview<const T>(w.gy), dview<T>(w.gq), dview<T>(w.gk),
      dview<T>(w.gv));
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_delta(const emb_delta_s* h, const DeltaArgs& call, const DeltaViews& w, bool backward, cudaStream_t s) {
  const auto of = [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    DeltaArgs a = call;
    return backward ? launch_delta_bwd<T, DK>(h, a, w, s) : launch_delta_fwd<T, DK, kForward>(h, a, w, s);
  };
  if (call.key_dim <= 32) return of(std::integral_constant<int, 32>());
  if (call.key_dim <= 64) return of(std::integral_constant<int, 64>());
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
