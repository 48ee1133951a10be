// scan.cu -- gated linear recurrence over padded sequences, forward, backward
// and one position at a time (scan_* in emb.h).
#include <atomic>
#include <new>

#include "rows.cuh"

namespace emb {

// Words the tiles of one call share.  The last CTA of a call leaves ticket,
// done and fail at zero and counts the epoch up, so a call needs no clearing.
struct ScanShared {
  uint32_t ticket;   // next tile
  uint32_t done;     // CTAs that found no more tiles
  uint32_t epoch;    // calls so far: the tag of this call's records
  uint32_t fail;     // a wait ran out: the others stop waiting
};

}  // namespace emb

struct emb_scan_s {
  int32_t dim = 0, max_batch = 0, max_len = 0;
  int sm_count = 0, device = 0;
  int64_t max_records = 0;
  uint32_t* status_d = nullptr;
  emb::ScanShared* shared_d = nullptr;
  ulonglong2* records_d = nullptr;   // [tiles][channels] what a tile does to a state (below)
};

namespace emb {

constexpr int kScanThreads = 256;
constexpr unsigned kScanSpins = 1u << 21;   // rounds a wait takes at most (about a second)
constexpr int kJoin = 8;                    // lanes of a channel in a chained call
constexpr int kCtasPerSm = 2;

// V channels of a thread.  Pairs go through the packed fp32 instructions: the
// recurrence is bound by instruction issue where elements are 16 bits.
template <int V>
struct Lanes {
  float v[V];
};
template <int V>
__device__ __forceinline__ Lanes<V> all_of(float x) {
  Lanes<V> o;
#pragma unroll
  for (int i = 0; i < V; ++i) o.v[i] = x;
  return o;
}
#define LANES_OP(name, args, one, two)                          \
  template <int V>                                              \
  __device__ __forceinline__ Lanes<V> name args {               \
    Lanes<V> o;                                                 \
    if constexpr (V == 1) {                                     \
      o.v[0] = one;                                             \
    } else {                                                    \
      _Pragma("unroll") for (int i = 0; i < V; i += 2) {        \
        const float2 r = two;                                   \
        o.v[i] = r.x, o.v[i + 1] = r.y;                         \
      }                                                         \
    }                                                           \
    return o;                                                   \
  }
#define PAIR(x) make_float2((x).v[i], (x).v[i + 1])
LANES_OP(add, (const Lanes<V>& a, const Lanes<V>& b), __fadd_rn(a.v[0], b.v[0]), __fadd2_rn(PAIR(a), PAIR(b)))
LANES_OP(sub, (const Lanes<V>& a, const Lanes<V>& b), __fsub_rn(a.v[0], b.v[0]),
         __ffma2_rn(PAIR(b), make_float2(-1.f, -1.f), PAIR(a)))
LANES_OP(mul, (const Lanes<V>& a, const Lanes<V>& b), __fmul_rn(a.v[0], b.v[0]), __fmul2_rn(PAIR(a), PAIR(b)))
LANES_OP(mad, (const Lanes<V>& a, const Lanes<V>& b, const Lanes<V>& c), __fmaf_rn(a.v[0], b.v[0], c.v[0]),
         __ffma2_rn(PAIR(a), PAIR(b), PAIR(c)))
#undef PAIR
#undef LANES_OP

template <class T, int V>
__device__ __forceinline__ Lanes<V> widen(const Vec<T, V>& x) {
  Lanes<V> o;
  if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      float2 r;
      if constexpr (std::is_same_v<T, __half>) {
        r = __half22float2(*reinterpret_cast<const __half2*>(&x.e[i]));
      } else {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&x.e[i]);
        r = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
      }
      o.v[i] = r.x, o.v[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = to_f32(x.e[i]);
  }
  return o;
}
template <class T, int V>
__device__ __forceinline__ Vec<T, V> narrow(const Lanes<V>& x) {
  Vec<T, V> o;
  if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (std::is_same_v<T, __half>)
        *reinterpret_cast<__half2*>(&o.e[i]) = __floats2half2_rn(x.v[i], x.v[i + 1]);
      else
        *reinterpret_cast<__nv_bfloat162*>(&o.e[i]) = __floats2bfloat162_rn(x.v[i], x.v[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(x.v[i]);
  }
  return o;
}

// sigmoid(g) and sigmoid(-g) from one exponential: with e = exp(-g), a = 1 /
// (1 + e) and 1 - a = e a keeps every digit where the gate saturates.  Gates
// stop at -87 (they would leave less than 2^-125 of the state), so e is
// finite; above 87 e counts as 0; NaN goes through.  A gate of +infinity gives
// exactly (1, 0): positions that are not there.  The flushing forms of the
// two approximations are single instructions, the others scale around them.
__device__ __forceinline__ float exp2_flush(float x) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ float inverse_flush(float x) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ void gates(float g, float& a, float& na) {
  asm("max.NaN.f32 %0, %0, 0fC2AE0000;" : "+f"(g));
  const float e = exp2_flush(g * -1.44269504f);
  a = inverse_flush(1.f + e);
  na = e * a;
}
template <class T, int V>
__device__ __forceinline__ void gates(const Vec<T, V>& g, Lanes<V>& a, Lanes<V>& na) {
  Lanes<V> x;
  if constexpr (sizeof(T) == 2 && V > 1) {
    Vec<T, V> c;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (std::is_same_v<T, __half>)
        *reinterpret_cast<__half2*>(&c.e[i]) =
            __hmax2_nan(*reinterpret_cast<const __half2*>(&g.e[i]), __float2half2_rn(-87.f));
      else
        *reinterpret_cast<__nv_bfloat162*>(&c.e[i]) =
            __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&g.e[i]), __float2bfloat162_rn(-87.f));
    }
    x = widen(c);
  } else {
    x = widen(g);
#pragma unroll
    for (int i = 0; i < V; ++i) asm("max.NaN.f32 %0, %0, 0fC2AE0000;" : "+f"(x.v[i]));
  }
  Lanes<V> e = mul(x, all_of<V>(-1.44269504f));
#pragma unroll
  for (int i = 0; i < V; ++i) e.v[i] = exp2_flush(e.v[i]);
  a = add(e, all_of<V>(1.f));
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = inverse_flush(a.v[i]);
  na = mul(e, a);
}

// `wide`: every column vector of the view can be moved in one access.  The
// others are moved element by element by the same threads, so results do not
// depend on strides and alignment.
template <class T>
struct View {
  T* p;
  int64_t bs, ts;
  bool wide;
  __device__ T* at(int64_t b, int64_t t, int64_t d) const { return p + (b * bs + t * ts + d); }
};

// Where a thread's stretch starts.  In the WIDE variant all views of a call
// have the same strides: one offset serves them all.
template <bool WIDE>
struct Start {
  int64_t o = 0;
  int b = 0, d = 0, t = 0;
  template <class T>
  __device__ Start(const View<T>& w, int b, int d, int t) : b(b), d(d), t(t) {
    if (WIDE) o = b * w.bs + t * w.ts + d;
  }
  template <class T>
  __device__ T* of(const View<T>& w) const {
    return WIDE ? w.p + o : w.at(b, t, d);
  }
};

template <int V, class T>
__device__ __forceinline__ Vec<T, V> get(const T* p, bool wide) {
  if (wide) return load_vec<T, V>(p);
  Vec<T, V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) r.e[v] = p[v];
  return r;
}

template <int V, class T>
__device__ __forceinline__ void put(T* p, bool wide, const Vec<T, V>& r) {
  if (wide) {
    store_vec(p, r);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = r.e[v];
  }
}

// Writes one thread's R column vectors; positions past n are 0, past `len` not
// there.
template <bool WIDE, int V, int R, class T>
__device__ __forceinline__ void put_stretch(const View<T>& w, T* p, const Vec<T, V> (&o)[R], int t0, int n, int len) {
  if (t0 + R <= n) {
#pragma unroll
    for (int r = 0; r < R; ++r, p += w.ts) put<V>(p, WIDE || w.wide, o[r]);
  } else {
    Vec<T, V> z;
#pragma unroll
    for (int v = 0; v < V; ++v) z.e[v] = from_f32<T>(0.f);
    for (int r = 0; r < R; ++r, p += w.ts)
      if (t0 + r < len) {
        Vec<T, V> x = z;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i == r && t0 + r < n) x = o[i];
        put<V>(p, WIDE || w.wide, x);
      }
  }
}

// A call's shape.  A tile is TT = (256 / cx) * R positions of cx column vectors
// of V channels; a column vector is V neighbouring channels of one batch entry.
struct ScanArgs {
  int32_t batch, len, dim;
  int32_t cx_log;        // column vectors of a tile, log2
  int32_t tiles;         // along time
  uint32_t total;        // tiles in all (chained calls)
  int64_t vecs;          // column vectors in all: batch * dim / V
  DivMagic32 per;        // by dim / V: a column vector's batch entry
  DivMagic32 groups;     // by the tiles across (chained calls)
  DivMagic32 tile;       // by the positions of a tile
  const int32_t* offsets;
  uint32_t* status;
  ScanShared* shared;
  ulonglong2* records;   // [tiles][pitch] (chained calls)
  ulonglong2* states;    // [groups of tiles + 1][pitch]
  uint32_t pitch;        // channels in all: a chained call has few
  int32_t group_log;     // log2 of the tiles of a chain's group
};

__device__ __forceinline__ int live_len(const ScanArgs& s, int b) {
  if (!s.offsets) return s.len;
  const int64_t n = (int64_t)__ldg(s.offsets + b + 1) - __ldg(s.offsets + b);
  if (n < 0) latch(s.status, EMB_ERR_BAD_INDEX);
  return n < 0 ? 0 : n > s.len ? s.len : (int)n;
}

// What a stretch of positions does to the state before it: h -> a h + b.
struct Affine {
  float a, b;
};
__device__ __forceinline__ Affine after(const Affine& later, const Affine& earlier) {
  return {later.a * earlier.a, fmaf(later.a, earlier.b, later.b)};
}

// Records of the chain.  Each 64-bit half carries the tag, so a reader that
// sees the wanted tag in both has both values of one write: no fence is needed.
__device__ __forceinline__ void put_record(ulonglong2* p, Affine f, uint32_t tag) {
  const uint64_t x = (uint64_t)tag << 32 | __float_as_uint(f.a), y = (uint64_t)tag << 32 | __float_as_uint(f.b);
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(x), "l"(y) : "memory");
}
__device__ __forceinline__ uint32_t get_record(const ulonglong2* p, Affine& f) {
  uint64_t x, y;
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "l"(p) : "memory");
  f = {__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)y)};
  const uint32_t tx = (uint32_t)(x >> 32), ty = (uint32_t)(y >> 32);
  return tx == ty ? tx : 0u;
}
// The state before tile `i` of one channel's chain.  The chain is cut into
// groups of tiles.  A tile writes its own effect for the later tiles of its
// group, and a group's last tile the state after the group; a tile joins the
// effects ahead of it in its group, which the channel's kJoin lanes read, behind
// the state before the group.  Along a sequence only the groups wait for one
// another in turn (one write and read in L2 per group), and the order of every
// join is fixed: results repeat bit for bit.  `all`: what this tile does;
// `next`: a later tile needs to know; state0: the state before tile 0.  All
// lanes of the warp call; the arguments are uniform over a channel's lanes.
__device__ __forceinline__ float chain_state(const ScanArgs& s, int64_t col, int i, bool want, bool next, Affine all,
                                             float state0, uint32_t epoch) {
  const auto row = [&](uint32_t r) { return (uint64_t)r * s.pitch; };
  const int each_log = s.group_log - 3, last = (1 << s.group_log) - 1;   // a lane's records
  const int j = threadIdx.x & (kJoin - 1), m = i >> s.group_log, at = i & last, first = j << each_log;
  ulonglong2* own = s.records + (row(i - at) + col);   // the group's first tile
  ulonglong2* states = s.states + (row(m) + col);
  if (want && next && j == 0 && at != last) put_record(own + row(at), all, epoch);
  own += row(first);
  Affine sum{1.f, 0.f}, st{0.f, state0};
  bool have_state = !want || m == 0 || j != 0;
  unsigned spins = 0;
  for (int u = 0;; ++u) {
    bool have = !want || first + u >= at;
    Affine f{1.f, 0.f};
    const bool ends = (u + 1) >> each_log != 0;
    for (;; ++spins) {
      if (!have) have = get_record(own, f) == epoch;
      if (!have_state) have_state = get_record(states, st) == epoch;
      if (__all_sync(kFull, have && (have_state || !ends))) break;
      if (spins >= kScanSpins) {
        latch(s.status, EMB_ERR_TIMEOUT);
        *(volatile uint32_t*)&s.shared->fail = 1u;
        break;
      }
      if ((spins & 255u) == 255u && __any_sync(kFull, *(volatile uint32_t*)&s.shared->fail != 0u)) spins = kScanSpins;
    }
    sum = after(f, sum);
    own += s.pitch;
    if (ends) break;
  }
#pragma unroll
  for (int o = 1; o < kJoin; o <<= 1) {
    const Affine e{__shfl_down_sync(kFull, sum.a, o, kJoin), __shfl_down_sync(kFull, sum.b, o, kJoin)};
    sum = after(e, sum);   // the upper lanes' sums are not used
  }
  const float h = __shfl_sync(kFull, fmaf(sum.a, st.b, sum.b), 0, kJoin);
  if (want && next && j == 0 && at == last) put_record(states + s.pitch, {0.f, fmaf(all.a, h, all.b)}, epoch);
  return h;
}
// Small groups wait for fewer tiles, large ones for fewer groups in turn; with
// few channels the turns bound the call.  us forward with groups of 8, 16 and
// 32: 4 x 32768 x 512 bf16 (64 tiles across) 105, 113, 128; 65536 x 320 bf16
// (10) 46, 47, 52; 65536 x 128 fp32 (4) 36, 32, 33; 131072 x 16 bf16 (1) 39,
// 24, 19.
constexpr int kLeastGroup = 8;
constexpr int group_log(int64_t across) { return across >= 8 ? 3 : across >= 3 ? 4 : 5; }

// A CTA's place: its threads as column vectors by stretches of R positions,
// and again as channels by J lanes, for joining the stretches.
template <int V, int R>
struct Place {
  int cx, ty, TT;            // column vector in the tile, stretch, positions of a tile
  int ch, j, j_log, pitch;   // channel in the tile, lane of it
  __device__ explicit Place(const ScanArgs& s) {
    const int tid = threadIdx.x;
    cx = tid & ((1 << s.cx_log) - 1);
    ty = tid >> s.cx_log;
    TT = (kScanThreads >> s.cx_log) * R;
    j_log = max(31 - __clz(kScanThreads / V) - s.cx_log, 0);
    j = tid & ((1 << j_log) - 1);
    ch = tid >> j_log;
    pitch = (V << s.cx_log) + 1;   // the lanes of a channel then read different banks
  }
};

// Joins the stretches of a tile for one channel: lane j takes stretches j V ..
// j V + V - 1 of (a, b) in shared memory, `back` in descending order.
// ex: what the stretches before this lane's do; all: what the whole tile does.
template <int V, class P>
__device__ __forceinline__ void join_stretches(const P& p, const float* sa, const float* sb, bool back, Affine (&f)[V],
                                               Affine& ex, Affine& all) {
  const int J = 1 << p.j_log;
  Affine m{1.f, 0.f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int y = p.j * V + i, at = (back ? J * V - 1 - y : y) * p.pitch + p.ch;
    f[i] = {sa[at], sb[at]};
    m = after(f[i], m);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o < J) {
      const Affine e{__shfl_up_sync(kFull, m.a, o, J), __shfl_up_sync(kFull, m.b, o, J)};
      if (p.j >= o) m = after(m, e);
    }
  }
  ex = {__shfl_up_sync(kFull, m.a, 1, J), __shfl_up_sync(kFull, m.b, 1, J)};
  if (p.j == 0) ex = {1.f, 0.f};
  all = {__shfl_sync(kFull, m.a, J - 1, J), __shfl_sync(kFull, m.b, J - 1, J)};
}

// The next tile of a chained call: tickets go to the tiles of one stretch of
// time, then of the next, so a tile comes after the one it waits for.
__device__ __forceinline__ uint32_t take_ticket(const ScanArgs& s) { return atomicAdd(&s.shared->ticket, 1u); }

// Called by one thread of a CTA that found no more tiles.
__device__ __forceinline__ void leave(const ScanArgs& s) {
  if (atomicAdd(&s.shared->done, 1u) != gridDim.x - 1) return;
  s.shared->ticket = 0;
  s.shared->done = 0;
  s.shared->fail = 0;
  s.shared->epoch = s.shared->epoch == 0xffffffffu ? 1u : s.shared->epoch + 1;
}

// Channel v of a column vector.
struct Channel {
  bool ok;
  int b, d, n;
  int64_t col;   // b * dim + d
};
template <int V>
__device__ __forceinline__ Channel channel_of(const ScanArgs& s, int64_t vec, int v) {
  Channel c;
  c.ok = vec < s.vecs;
  const uint32_t i = c.ok ? (uint32_t)vec : 0u;
  c.b = (int)div_magic32(i, s.per);
  c.d = (int)(i - (uint32_t)c.b * s.per.d) * V + v;
  c.n = c.ok ? live_len(s, c.b) : 0;
  c.col = (int64_t)i * V + v;
  return c;
}

// A thread's R column vectors of one input, staged in shared memory: only the
// thread itself reads what it copied, so no barrier is needed.  Copies are
// asynchronous where the view allows it; otherwise the vectors are loaded
// when they are due (`now`).  Positions at or past n hold `dead`.
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <class T, int V, int R, bool WIDE>
struct Staged {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr bool kAlways = WIDE && kBytes >= 4;
  Vec<T, V>* at;   // + r * kScanThreads
  __device__ bool async(const View<const T>& w) const { return kAlways || (kBytes >= 4 && w.wide); }
  __device__ static void copy(Vec<T, V>* to, const T* p) {
    const unsigned d = (unsigned)__cvta_generic_to_shared(to);
    if constexpr (kBytes == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(p) : "memory");
    else if constexpr (kBytes >= 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(p), "n"(kBytes) : "memory");
  }
  __device__ void fill(const View<const T>& w, const T* p, int t0, int n, float dead, bool now) const {
    if (kAlways ? now : async(w) == now) return;
    Vec<T, V> z;
#pragma unroll
    for (int v = 0; v < V; ++v) z.e[v] = from_f32<T>(dead);
    if (kAlways || !now) {
      if (t0 + R <= n) {
#pragma unroll
        for (int r = 0; r < R; ++r, p += w.ts) copy(at + r * kScanThreads, p);
      } else {
        for (int r = 0; r < R; ++r, p += w.ts) {
          if (t0 + r < n) copy(at + r * kScanThreads, p);
          else at[r * kScanThreads] = z;
        }
      }
    } else if constexpr (!kAlways) {
      Vec<T, V> got[R];
#pragma unroll
      for (int r = 0; r < R; ++r, p += w.ts) {
        got[r] = z;
        if (t0 + r < n) got[r] = get<V>(p, WIDE || w.wide);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) at[r * kScanThreads] = got[r];
    }
  }
};

#define SCAN_DEAD_GATE __int_as_float(0x7f800000)

// Forward.  A thread keeps R positions of V channels as (a, (1 - a) x) in
// registers, so x and gate are read once.  Its stretch's effect goes to shared
// memory, the channels' lanes join the stretches behind the state before the
// tile, and each thread then runs its positions from its own first state.  The
// next tile's inputs are copied meanwhile.  fp32 is bound by memory (16 x 8192
// x 512 walking 129 us, 6.2 TB/s); 16 bits by instruction issue and the latency
// between a tile's steps (128 x 1024 x 512 bf16 81 us, 5.0 TB/s; 19 instructions
// an element), chained also by the waits (131072 x 512 bf16 120 us, 10 of them
// waiting for records).
// CHAIN: a CTA takes tiles by ticket and finds the state before its tile in the
// records of the tiles ahead; otherwise it walks along time with the state in
// hand.  cx = 256: a thread is a whole stretch of its own, nothing is joined.
template <class T, int V, int R, bool CHAIN, bool WIDE>
__global__ void __launch_bounds__(kScanThreads, kCtasPerSm) k_scan_fwd(ScanArgs s, View<const T> x, View<const T> g,
                                                                       View<T> y, const float* __restrict__ state_in,
                                                                       float* __restrict__ state_out) {
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t slot;
  const Place<V, R> p(s);
  const bool whole = s.cx_log == 8;
  const Staged<T, V, R, WIDE> sx{(Vec<T, V>*)raw + threadIdx.x}, sg{sx.at + R * kScanThreads};
  float* sa = (float*)(raw + 2 * R * kScanThreads * sizeof(Vec<T, V>));
  float* sb = sa + (kScanThreads >> s.cx_log) * p.pitch;
  const uint32_t epoch = CHAIN ? *(volatile uint32_t*)&s.shared->epoch : 0;
  uint32_t tile = 0, next = 0;
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) slot = take_ticket(s);
    __syncthreads();
    tile = slot;
  }
  int k = CHAIN ? (int)div_magic32(tile, s.groups) : 0;
  int64_t gi = CHAIN ? tile - (uint32_t)k * s.groups.d : blockIdx.x;
  Channel c = channel_of<V>(s, (gi << s.cx_log) + p.cx, 0);
  auto fill = [&](const Channel& c, int k, bool now) {
    const int t0 = k * p.TT + p.ty * R;
    const Start<WIDE> at(x, c.b, c.d, t0);
    sx.fill(x, at.of(x), t0, c.n, 0.f, now);
    sg.fill(g, at.of(g), t0, c.n, SCAN_DEAD_GATE, now);
    return at.o;
  };
  int64_t o = 0, o1 = 0;   // WIDE: this tile's and the next one's start
  if (!CHAIN || tile < s.total) o = fill(c, k, false);
  float held = 0.f;          // walking: the channel's state
  Channel q{};               // walking: the same all along (16 x 8192 x 512 bf16 95 -> 89 us, backward 176 -> 167)
  if (!CHAIN && !whole) q = channel_of<V>(s, (gi << s.cx_log) + p.ch / V, p.ch % V);
  Lanes<V> own;              // whole: the thread's states
  while (CHAIN ? tile < s.total : k < s.tiles) {
    const int t0 = k * p.TT + p.ty * R;
    fill(c, k, true);
    copies_done();
    Lanes<V> a[R], b[R], fa = all_of<V>(1.f), fb = all_of<V>(0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Lanes<V> na;
      gates(sg.at[r * kScanThreads], a[r], na);
      b[r] = mul(na, widen(sx.at[r * kScanThreads]));
      fa = mul(fa, a[r]);
      fb = mad(a[r], fb, b[r]);
    }
    // The staged inputs are in registers: copy the next tile's.  A chained call
    // draws its ticket only when this tile has waited for the state before it:
    // a tile held by a CTA that still waits would make later ones wait for it
    // (drawn before the join: 131072 x 512 fp32 177 us forward, after: 157).
    int k1 = k + 1;
    int64_t gi1 = gi;
    Channel c1 = c;
    auto ahead = [&] {
      if constexpr (CHAIN) {
        next = slot;
        k1 = (int)div_magic32(next, s.groups);
        gi1 = next - (uint32_t)k1 * s.groups.d;
        if (next >= s.total) return;
        c1 = channel_of<V>(s, (gi1 << s.cx_log) + p.cx, 0);
      } else if (k1 >= s.tiles) {
        return;
      }
      o1 = fill(c1, k1, false);
    };
    Lanes<V> h;
    if (whole) {
      ahead();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == 0) own.v[v] = state_in && c.ok ? state_in[c.col + v] : 0.f;
        h.v[v] = own.v[v];
        own.v[v] = fmaf(fa.v[v], own.v[v], fb.v[v]);
        if (state_out && c.ok && k == s.tiles - 1) state_out[c.col + v] = own.v[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sa[p.ty * p.pitch + p.cx * V + v] = fa.v[v];
        sb[p.ty * p.pitch + p.cx * V + v] = fb.v[v];
      }
      __syncthreads();
      if (!CHAIN) ahead();
      if constexpr (CHAIN) q = channel_of<V>(s, (gi << s.cx_log) + p.ch / V, p.ch % V);
      Affine f[V], ex, all;
      join_stretches<V>(p, sa, sb, false, f, ex, all);
      const int end = (k + 1) * p.TT;
      const bool live = q.ok && (k * p.TT < q.n || k == 0);
      if constexpr (CHAIN) {
        const float state0 = live && k >> s.group_log == 0 && state_in ? state_in[q.col] : 0.f;
        held = chain_state(s, q.col, k, live, end < q.n, all, state0, epoch);
      } else if (k == 0) {
        held = state_in && q.ok ? state_in[q.col] : 0.f;
      }
      float st = fmaf(ex.a, held, ex.b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sb[(p.j * V + i) * p.pitch + p.ch] = st;
        st = fmaf(f[i].a, st, f[i].b);
      }
      held = fmaf(all.a, held, all.b);
      if (state_out && live && p.j == 0 && end >= q.n) state_out[q.col] = held;
      if (CHAIN && threadIdx.x == 0) slot = take_ticket(s);
      __syncthreads();
      if (CHAIN) ahead();
#pragma unroll
      for (int v = 0; v < V; ++v) h.v[v] = sb[p.ty * p.pitch + p.cx * V + v];
    }
    Vec<T, V> out[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h = mad(a[r], h, b[r]);
      out[r] = narrow<T>(h);
    }
    put_stretch<WIDE, V, R>(y, WIDE ? y.p + o : y.at(c.b, t0, c.d), out, t0, c.n, c.ok ? s.len : 0);
    c = c1, k = k1, gi = gi1, o = o1;
    tile = next;
  }
  if (CHAIN && threadIdx.x == 0) leave(s);
}

// The backward of 16-bit elements finds the fp32 states before its tiles again.
// k_scan_effects reduces each tile to what it does to a state, all tiles at
// once; k_scan_states runs along each channel's tiles.  Both leave their numbers
// in the first rows of the tile's gradients, the upper half of an fp32 in one
// and the lower in the other, which that tile's CTA reads and overwrites: no
// workspace.  Only whole tiles with live positions behind them are looked at.
// 131072 x 512 bf16: 45 us, the inputs read a second time at 5.9 TB/s, and 11 us,
// the latency of strided rows (one CTA for 32 channels: 32); 128 x 1024 x 512 41
// and 10 us.  As a chain of tiles like the forward's they took 139 us and 68.
template <class T, int V>
__device__ __forceinline__ void put_halves(const View<T>& up, const View<T>& low, int b, int t, int d,
                                           const Lanes<V>& x) {
  Vec<T, V> u, l;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t w = __float_as_uint(x.v[v]);
    *reinterpret_cast<uint16_t*>(&u.e[v]) = (uint16_t)(w >> 16);
    *reinterpret_cast<uint16_t*>(&l.e[v]) = (uint16_t)w;
  }
  put<V>(up.at(b, t, d), up.wide, u);
  put<V>(low.at(b, t, d), low.wide, l);
}
template <int V, class T>
__device__ __forceinline__ Lanes<V> get_halves(const View<T>& up, const View<T>& low, int b, int t, int d) {
  const Vec<T, V> u = get<V>((const T*)up.at(b, t, d), up.wide), l = get<V>((const T*)low.at(b, t, d), low.wide);
  Lanes<V> x;
#pragma unroll
  for (int v = 0; v < V; ++v)
    x.v[v] = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(&u.e[v]) << 16 |
                             *reinterpret_cast<const uint16_t*>(&l.e[v]));
  return x;
}

// A CTA takes 32 column vectors of one tile, its warps a part of the tile's
// positions each; a call of several tiles has them of 128 or 160 positions.
constexpr int kEffectWarps = 4, kEffectRows = 8;
template <class T, int V>
__global__ void __launch_bounds__(kEffectWarps * 32) k_scan_effects(const __grid_constant__ ScanArgs s,
                                                                    View<const T> x, View<const T> g, View<T> gx,
                                                                    View<T> gg) {
  __shared__ Lanes<V> sa[kEffectWarps][32], sb[kEffectWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, TT = (int)s.tile.d;
  const uint32_t k = div_magic32(blockIdx.x, s.groups);
  const Channel c = channel_of<V>(s, (int64_t)(blockIdx.x - k * s.groups.d) * 32 + lane, 0);
  const int t0 = (int)k * TT, part = TT / kEffectWarps;
  const bool live = t0 + TT < c.n;
  Lanes<V> a = all_of<V>(1.f), b = all_of<V>(0.f);
  if (live) {
    const T *px = x.at(c.b, t0 + warp * part, c.d), *pg = g.at(c.b, t0 + warp * part, c.d);
    for (int t = 0; t < part; t += kEffectRows) {
      Vec<T, V> xv[kEffectRows], gv[kEffectRows];
#pragma unroll
      for (int r = 0; r < kEffectRows; ++r, px += x.ts, pg += g.ts)
        xv[r] = get<V>(px, x.wide), gv[r] = get<V>(pg, g.wide);
#pragma unroll
      for (int r = 0; r < kEffectRows; ++r) {
        Lanes<V> e, ne;
        gates(gv[r], e, ne);
        a = mul(a, e);
        b = mad(e, b, mul(ne, widen(xv[r])));
      }
    }
  }
  sa[warp][lane] = a, sb[warp][lane] = b;
  __syncthreads();
  if (warp != 0 || !live) return;
#pragma unroll
  for (int w = 1; w < kEffectWarps; ++w) {
    b = mad(sa[w][lane], b, sb[w][lane]);
    a = mul(sa[w][lane], a);
  }
  put_halves<T, V>(gx, gg, c.b, t0, c.d, a);
  put_halves<T, V>(gx, gg, c.b, t0 + 1, c.d, b);
}

// A cluster takes 32 channels, the warps of its CTAs `each` neighbouring tiles:
// up to 2048 tiles are then read once, all loads in flight.  Effects of the CTAs
// ahead are read from their shared memory.
constexpr int kStateWarps = 32, kStateRows = 8, kStateCtas = 8;
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ Affine of_cta(const Affine* p, uint32_t rank) {   // the same variable of another CTA
  uint32_t a;
  Affine f;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(f.a), "=f"(f.b) : "r"(a) : "memory");
  return f;
}
template <class T>
__global__ void __launch_bounds__(kStateWarps * 32) k_scan_states(const __grid_constant__ ScanArgs s, int each,
                                                                  View<T> gx, View<T> gg,
                                                                  const float* __restrict__ state_in) {
  __shared__ Affine part[kStateWarps][32];
  __shared__ alignas(8) Affine cta[32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, TT = (int)s.tile.d;
  const uint32_t rank = cluster_rank(), ctas = cluster_ctas();
  const Channel c = channel_of<1>(s, (int64_t)(blockIdx.x / ctas) * 32 + lane, 0);
  const int whole = c.n > 0 ? (int)div_magic32((uint32_t)c.n - 1, s.tile) : 0;   // tiles with live positions behind them
  const int lo = min(((int)rank * warps + warp) * each, whole), hi = min(lo + each, whole);
  Affine f[kStateRows];
  const auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kStateRows; ++i) {
      f[i] = {1.f, 0.f};
      if (k0 + i < hi)
        f[i] = {get_halves<1>(gx, gg, c.b, (k0 + i) * TT, c.d).v[0],
                get_halves<1>(gx, gg, c.b, (k0 + i) * TT + 1, c.d).v[0]};
    }
  };
  Affine all{1.f, 0.f}, before = all;
  for (int k0 = lo; k0 == lo || k0 < hi; k0 += kStateRows) {
    load(k0);
#pragma unroll
    for (int i = 0; i < kStateRows; ++i) all = after(f[i], all);
  }
  part[warp][lane] = all;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = after(part[w][lane], before);
  if (warp == warps - 1) cta[lane] = after(all, before);
  float h = state_in && c.ok ? state_in[c.col] : 0.f;
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
    for (uint32_t r = 0; r < rank; ++r) {
      const Affine e = of_cta(&cta[lane], r);
      h = fmaf(e.a, h, e.b);
    }
    cluster_arrive();   // no CTA leaves before the others have read its effects
  }
  h = fmaf(before.a, h, before.b);
  for (int k0 = lo; k0 < hi; k0 += kStateRows) {   // effects are read before states take their places
    if (each > kStateRows) load(k0);
#pragma unroll
    for (int i = 0; i < kStateRows; ++i) {
      if (k0 + i < hi && k0 + i > 0) put_halves<T, 1>(gx, gg, c.b, (k0 + i) * TT, c.d, all_of<1>(h));
      h = fmaf(f[i].a, h, f[i].b);
    }
  }
  if (hi > lo && hi == whole) put_halves<T, 1>(gx, gg, c.b, whole * TT, c.d, all_of<1>(h));
  if (ctas > 1) cluster_wait();
}

template <class T>
__device__ __forceinline__ float get_state(const View<T>& up, const View<T>& low, int b, int t, int d) {
  return get_halves<1>(View<T>{up.p, up.bs, up.ts, true}, View<T>{low.p, low.bs, low.ts, true}, b, t, d).v[0];
}

// Backward, from the last position to the first: C_t = a_t (grad_y_t + C_{t+1})
// is what position t passes back.  The gate's gradient needs the state before
// each position, in fp32: a tile runs forward from the state before it, and
// both joins use the same products of gates.  fp32 elements: that state is y just
// before the tile, one row of y instead of all of them.  16 bits: y is rounded,
// and h - x may be far smaller than h; so the states are found again from x and
// gate (k_scan_effects, k_scan_states) and y is not read.
// Bound as the forward is: 16 x 8192 x 512 fp32 208 us, 6.4 TB/s; 128 x 1024 x
// 512 bf16 156 us, 131072 x 512 bf16 206 us, with the states before the tiles
// 215 and 270 (from y as it is rounded 154 and 202: every position's y read, and
// the gate's gradient as far off as h's rounding is beside h - x).
template <class T, int V, int R, bool CHAIN, bool WIDE>
__global__ void __launch_bounds__(kScanThreads, kCtasPerSm) k_scan_bwd(ScanArgs s, View<const T> x, View<const T> g,
                                                                       View<const T> y, View<const T> gy,
                                                                       const float* __restrict__ state_in,
                                                                       const float* __restrict__ grad_out, View<T> gx,
                                                                       View<T> gg, float* __restrict__ grad_in) {
  constexpr bool HALF = sizeof(T) == 2;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t slot;
  const Place<V, R> p(s);
  const bool whole = !HALF && s.cx_log == 8;   // 16 bits: such lengths are held whole (k_scan_short_bwd)
  const int area = (kScanThreads >> s.cx_log) * p.pitch;
  const Staged<T, V, R, WIDE> sx{(Vec<T, V>*)raw + threadIdx.x}, sg{sx.at + R * kScanThreads},
      sd{sg.at + R * kScanThreads};
  float* sa = (float*)(raw + 3 * R * kScanThreads * sizeof(Vec<T, V>));
  float *sb = sa + area, *sc = sb + area;
  if constexpr (HALF) pdl_wait();
  const uint32_t epoch = CHAIN ? *(volatile uint32_t*)&s.shared->epoch : 0;
  uint32_t tile = 0, next = 0;
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) slot = take_ticket(s);
    __syncthreads();
    tile = slot;
  }
  int k = s.tiles - 1 - (CHAIN ? (int)div_magic32(tile, s.groups) : 0);
  int64_t gi = CHAIN ? tile - (uint32_t)(s.tiles - 1 - k) * s.groups.d : blockIdx.x;
  Channel c = channel_of<V>(s, (gi << s.cx_log) + p.cx, 0);
  auto fill = [&](const Channel& c, int k, bool now) {
    const int t0 = k * p.TT + p.ty * R;
    const Start<WIDE> at(x, c.b, c.d, t0);
    sx.fill(x, at.of(x), t0, c.n, 0.f, now);
    sg.fill(g, at.of(g), t0, c.n, SCAN_DEAD_GATE, now);
    sd.fill(gy, at.of(gy), t0, c.n, 0.f, now);
    return at.o;
  };
  int64_t o = 0, o1 = 0;
  if (!CHAIN || tile < s.total) o = fill(c, k, false);
  float held = 0.f;
  // fp32 with four channels has no registers to keep it in
  constexpr bool kHeld = !CHAIN && !(!HALF && V == 4);
  Channel q{};
  if (kHeld && !whole) q = channel_of<V>(s, (gi << s.cx_log) + p.ch / V, p.ch % V);
  Lanes<V> own;
  while (CHAIN ? tile < s.total : k >= 0) {
    const int t0 = k * p.TT + p.ty * R;
    fill(c, k, true);
    copies_done();
    Lanes<V> a[R], na[R], xv[R];   // xv: x, then the gate's factor of G
    Vec<T, V> dy[R];               // as it is stored: 16 bits take half the registers
    Lanes<V> fa = all_of<V>(1.f), fb = all_of<V>(0.f), fc = all_of<V>(0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      gates(sg.at[r * kScanThreads], a[r], na[r]);
      xv[r] = widen(sx.at[r * kScanThreads]);
      dy[r] = sd.at[r * kScanThreads];
      fa = mul(fa, a[r]);
      fb = mad(a[r], fb, mul(na[r], xv[r]));
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) fc = mul(a[r], add(widen(dy[r]), fc));
    // the next tile's inputs (as in the forward)
    int k1 = k - 1;
    int64_t gi1 = gi;
    Channel c1 = c;
    auto ahead = [&] {
      if constexpr (CHAIN) {
        next = slot;
        const int back = (int)div_magic32(next, s.groups);
        k1 = s.tiles - 1 - back;
        gi1 = next - (uint32_t)back * s.groups.d;
        if (next >= s.total) return;
        c1 = channel_of<V>(s, (gi1 << s.cx_log) + p.cx, 0);
      } else if (k1 < 0) {
        return;
      }
      o1 = fill(c1, k1, false);
    };
    Lanes<V> h, C;
    if (whole) {
      ahead();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == s.tiles - 1) own.v[v] = grad_out && c.ok ? grad_out[c.col + v] : 0.f;
        C.v[v] = own.v[v];
        own.v[v] = fmaf(fa.v[v], own.v[v], fc.v[v]);
        if (grad_in && c.ok && k == 0) grad_in[c.col + v] = own.v[v];
        h.v[v] = 0.f;
        if (c.ok && t0 == 0) h.v[v] = state_in ? state_in[c.col + v] : 0.f;
        else if (t0 < c.n) h.v[v] = to_f32(*y.at(c.b, t0 - 1, c.d + v));
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sa[p.ty * p.pitch + p.cx * V + v] = fa.v[v];
        sb[p.ty * p.pitch + p.cx * V + v] = fb.v[v];
        sc[p.ty * p.pitch + p.cx * V + v] = fc.v[v];
      }
      if constexpr (!kHeld) q = channel_of<V>(s, (gi << s.cx_log) + p.ch / V, p.ch % V);
      const int start = k * p.TT;
      const bool live = q.ok && (start < q.n || k == 0);
      float first = 0.f;
      if (live && k == 0) first = state_in ? state_in[q.col] : 0.f;
      else if (live) first = HALF ? get_state(gx, gg, q.b, start, q.d) : to_f32(*y.at(q.b, start - 1, q.d));
      __syncthreads();
      if (!CHAIN) ahead();
      Affine f[V], ex, all;
      join_stretches<V>(p, sa, sb, false, f, ex, all);
      float st = fmaf(ex.a, first, ex.b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sb[(p.j * V + i) * p.pitch + p.ch] = st;
        st = fmaf(f[i].a, st, f[i].b);
      }
      join_stretches<V>(p, sa, sc, true, f, ex, all);
      // the chain of a channel begins at the tile of its last position
      const int last = q.n > 0 ? (int)div_magic32((uint32_t)q.n - 1, s.tile) : 0;
      if constexpr (CHAIN) {
        const int i = live ? last - k : 0;
        const float state0 = live && i >> s.group_log == 0 && grad_out ? grad_out[q.col] : 0.f;
        held = chain_state(s, q.col, i, live, k > 0, all, state0, epoch);
      } else if (k == last) {
        held = grad_out && q.ok ? grad_out[q.col] : 0.f;
      }
      st = fmaf(ex.a, held, ex.b);
      const int J = 1 << p.j_log;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sc[(J * V - 1 - (p.j * V + i)) * p.pitch + p.ch] = st;
        st = fmaf(f[i].a, st, f[i].b);
      }
      if (live) held = fmaf(all.a, held, all.b);
      if (grad_in && live && p.j == 0 && k == 0) grad_in[q.col] = held;
      if (CHAIN && threadIdx.x == 0) slot = take_ticket(s);
      __syncthreads();
      if (CHAIN) ahead();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h.v[v] = sb[p.ty * p.pitch + p.cx * V + v];
        C.v[v] = sc[p.ty * p.pitch + p.cx * V + v];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Lanes<V> before = h;
      h = mad(a[r], h, mul(na[r], xv[r]));
      xv[r] = mul(mul(a[r], na[r]), sub(before, xv[r]));
    }
    Vec<T, V> ox[R], og[R];
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const Lanes<V> G = add(widen(dy[r]), C);
      ox[r] = narrow<T>(mul(na[r], G));
      og[r] = narrow<T>(mul(xv[r], G));
      C = mul(a[r], G);
    }
    put_stretch<WIDE, V, R>(gx, WIDE ? gx.p + o : gx.at(c.b, t0, c.d), ox, t0, c.n, c.ok ? s.len : 0);
    put_stretch<WIDE, V, R>(gg, WIDE ? gg.p + o : gg.at(c.b, t0, c.d), og, t0, c.n, c.ok ? s.len : 0);
    c = c1, k = k1, gi = gi1, o = o1;
    tile = next;
  }
  if (CHAIN && threadIdx.x == 0) leave(s);
}

// Short sequences, of at most U positions: a thread holds a whole column vector
// in registers, so the backward runs forward from the first state and needs no
// y.  The tiles above would leave most of their positions empty (20000 x 2 x
// 75 fp16: 47 us forward, 8 here).  Bound by memory where a vector fills an
// access (50000 x 4 x 256 fp32 7.0 TB/s in either direction, 100000 x 7 x 50
// fp16 6.4), by instruction issue for single channels of 16 bits (3.9).
template <class T, int V, int U, bool WIDE>
__global__ void __launch_bounds__(128) k_scan_short_fwd(const __grid_constant__ ScanArgs s, View<const T> x,
                                                        View<const T> g, View<T> y,
                                                        const float* __restrict__ state_in,
                                                        float* __restrict__ state_out) {
  const Channel c = channel_of<V>(s, blockIdx.x * 128ll + threadIdx.x, 0);
  if (!c.ok) return;
  Vec<T, V> xr[U], gr[U];
  const Start<WIDE> at(x, c.b, c.d, 0);
  const T *px = at.of(x), *pg = at.of(g);
#pragma unroll
  for (int t = 0; t < U; ++t, px += x.ts, pg += g.ts)
    if (t < c.n) {
      xr[t] = get<V>(px, WIDE || x.wide);
      gr[t] = get<V>(pg, WIDE || g.wide);
    }
  Lanes<V> h = all_of<V>(0.f);
  if (state_in) {
#pragma unroll
    for (int v = 0; v < V; ++v) h.v[v] = state_in[c.col + v];
  }
  T* py = at.of(y);
#pragma unroll
  for (int t = 0; t < U; ++t, py += y.ts) {
    Vec<T, V> o;
    if (t < c.n) {
      Lanes<V> a, na;
      gates(gr[t], a, na);
      h = mad(a, h, mul(na, widen(xr[t])));
      o = narrow<T>(h);
    } else {
      o = narrow<T>(all_of<V>(0.f));
    }
    if (t < s.len) put<V>(py, WIDE || y.wide, o);
  }
  if (state_out) {
#pragma unroll
    for (int v = 0; v < V; ++v) state_out[c.col + v] = h.v[v];
  }
}

template <class T, int V, int U, bool WIDE>
__global__ void __launch_bounds__(128) k_scan_short_bwd(const __grid_constant__ ScanArgs s, View<const T> x,
                                                        View<const T> g, View<const T> gy,
                                                        const float* __restrict__ state_in,
                                                        const float* __restrict__ grad_out, View<T> gx, View<T> gg,
                                                        float* __restrict__ grad_in) {
  const Channel c = channel_of<V>(s, blockIdx.x * 128ll + threadIdx.x, 0);
  if (!c.ok) return;
  Vec<T, V> xr[U], gr[U], dr[U];
  const Start<WIDE> at(x, c.b, c.d, 0);
  const T *px = at.of(x), *pg = at.of(g), *pd = at.of(gy);
#pragma unroll
  for (int t = 0; t < U; ++t, px += x.ts, pg += g.ts, pd += gy.ts)
    if (t < c.n) {
      xr[t] = get<V>(px, WIDE || x.wide);
      gr[t] = get<V>(pg, WIDE || g.wide);
      dr[t] = get<V>(pd, WIDE || gy.wide);
    }
  Lanes<V> h = all_of<V>(0.f), C = all_of<V>(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (state_in) h.v[v] = state_in[c.col + v];
    if (grad_out) C.v[v] = grad_out[c.col + v];
  }
  Lanes<V> a[U], na[U], w[U];   // w: the gate's factor of G
#pragma unroll
  for (int t = 0; t < U; ++t)
    if (t < c.n) {
      gates(gr[t], a[t], na[t]);
      const Lanes<V> xv = widen(xr[t]);
      w[t] = mul(mul(a[t], na[t]), sub(h, xv));
      h = mad(a[t], h, mul(na[t], xv));
    }
  T *pgx = at.of(gx) + (U - 1) * gx.ts, *pgg = at.of(gg) + (U - 1) * gg.ts;
#pragma unroll
  for (int t = U - 1; t >= 0; --t, pgx -= gx.ts, pgg -= gg.ts) {
    Vec<T, V> ox = narrow<T>(all_of<V>(0.f)), og = ox;
    if (t < c.n) {
      const Lanes<V> G = add(widen(dr[t]), C);
      ox = narrow<T>(mul(na[t], G));
      og = narrow<T>(mul(w[t], G));
      C = mul(a[t], G);
    }
    if (t < s.len) {
      put<V>(pgx, WIDE || gx.wide, ox);
      put<V>(pgg, WIDE || gg.wide, og);
    }
  }
  if (grad_in) {
#pragma unroll
    for (int v = 0; v < V; ++v) grad_in[c.col + v] = C.v[v];
  }
}

// One position per session: a thread takes V channels of one row, each value is
// read and written once.  Bound by memory (100000 x 256 bf16 56 us, 6.4 TB/s),
// few sessions by their launch (192 x 256: 1.6 us); widths that only pairs or
// single channels divide by instruction issue (100000 x 50 fp16 17 us).
template <class T, int V>
__global__ void __launch_bounds__(128) k_scan_step(int64_t n, DivMagic vecs, const T* __restrict__ x, int64_t xs,
                                                   const T* __restrict__ g, int64_t gs,
                                                   const int64_t* __restrict__ rows, float* __restrict__ states,
                                                   int64_t num_rows, T* __restrict__ y, int64_t ys) {
  const int64_t per = (int64_t)vecs.d, dim = per * V;
  for (int64_t i = blockIdx.x * 128ll + threadIdx.x; i < n * per; i += gridDim.x * 128ll) {
    const int64_t row = (int64_t)div_magic((uint64_t)i, vecs), d = (i - row * per) * V;
    const int64_t at = rows[row];
    Lanes<V> h = all_of<V>(0.f);
    if (at >= 0 && at < num_rows) {
      const Vec<T, V> gv = load_vec<T, V>(g + row * gs + d), xv = load_vec<T, V>(x + row * xs + d);
      Vec<float, V>* s = reinterpret_cast<Vec<float, V>*>(states + at * dim + d);
      Lanes<V> a, na;
      gates(gv, a, na);
      h = mad(a, widen(*s), mul(na, widen(xv)));
      *s = narrow<float>(h);
    }
    store_vec(y + row * ys + d, narrow<T>(h));
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


template <class T, int V>
View<T> as_view(const scan_view* v) {
  return View<T>{(T*)v->data, v->batch_stride, v->time_stride,
                 aligned_to(v->data, V * sizeof(T)) && v->batch_stride % V == 0 && v->time_stride % V == 0};
}

bool call_ok(emb_scan h, int32_t batch, int32_t len, int32_t dtype) {
  return h && batch >= 0 && batch <= h->max_batch && len >= 0 && len <= h->max_len && dtype_size(dtype) != 0 &&
         on_device(h->device);
}

// How a call is cut.  R: positions of a thread.
struct Cut {
  ScanArgs args;
  bool chain, fits;
  bool follows;   // launched as the dependant of the kernel ahead of it
  unsigned grid;
  int device;
};

// Positions of a thread, as many as its registers hold, for V = 4, 2 and 1
// channels.  Fewer tiles wait for one another where there are more, so a
// chained backward of 16-bit elements, whose gradients of y take half the
// registers, has five (131072 x 512 bf16: 206 us);
// walking, tiles of 160 positions fit sequences worse (1024 x 512 x 128 bf16:
// 160 us with four, 169 with five).
template <int V>
constexpr int fwd_positions() { return V == 4 ? 8 : V == 2 ? 16 : 24; }
template <class T, int V, bool CHAIN>
constexpr int bwd_positions() {
  if (V == 4) return sizeof(T) == 2 && CHAIN ? 5 : 4;
  if (V == 2) return 8;
  return sizeof(T) == 2 ? 16 : 8;
}
// log2 of the column vectors of a tile where sequences are long: 32 channels
// (chained with 16: 131072 x 512 bf16 138 us forward against 122; with 64: 127)
template <int V>
constexpr int long_cx() { return V == 4 ? 3 : V == 2 ? 4 : 5; }

int channels_at_once(int32_t dim) { return dim % 4 == 0 ? 4 : dim % 2 == 0 ? 2 : 1; }

// Positions of the smallest tile that a chained call has, forward or backward,
// and the records of one whose tiles have TT positions: one of each tile, one
// of each group of tiles, for every channel.
template <int V>
constexpr int least_tile() {
  constexpr int f = fwd_positions<V>(), b4 = bwd_positions<float, V, true>(), b2 = bwd_positions<__half, V, true>();
  constexpr int b = b4 < b2 ? b4 : b2;
  return (kScanThreads >> long_cx<V>()) * (f < b ? f : b);
}
int64_t chain_records(int TT, int64_t cols, int64_t len) {
  const int64_t tiles = (len + TT - 1) / TT;
  return (tiles + tiles / kLeastGroup + 1) * cols;
}

// A call whose last round of walking CTAs would leave more than two fifths of
// the GPU's places idle is chained, if it is long enough for a chain to start:
// the more CTAs walk side by side, the more.  us forward, walking and chained,
// on 304 places: 176 tiles across, 11 x 8192 x 512 bf16, 94 and 74; 256 tiles 97
// and 107; 430 of 2400 positions fp32 69 and 79; 100 of 600, 1200 and 2400
// positions bf16 8.4 and 10.4, 12.6 and 12.9, 22 and 19; 800 x 512 10.4 and 8.1.
// chain_r, walk_r: positions of a thread in either case.
bool idle_enough(int64_t wide, int64_t slots) { return wide * 5 < (wide + slots - 1) / slots * slots * 3; }
// The tiles of 32 channels across the widest call that is chained: under 6/5 of
// the places (under 3/5 of one round of them, of two, and never of three).
int64_t most_chained(int64_t slots) { return (6 * slots - 1) / 5; }
template <int V>
Cut cut_call(const emb_scan_s* h, int32_t batch, int32_t len, const int32_t* offsets, int chain_r, int walk_r) {
  Cut c{};
  ScanArgs& a = c.args;
  a.batch = batch;
  a.len = len;
  a.dim = h->dim;
  a.vecs = (int64_t)batch * h->dim / V;
  a.offsets = offsets;
  a.status = h->status_d;
  a.shared = h->shared_d;
  a.records = h->records_d;
  a.per = make_div_magic32((uint32_t)(h->dim / V));
  constexpr int kCx = long_cx<V>();
  static_assert((kScanThreads / V >> kCx) == kJoin, "the lanes of a channel read its group's records");
  const int64_t slots = (int64_t)h->sm_count * kCtasPerSm;
  const auto across = [&](int cx_log) { return (a.vecs + (1 << cx_log) - 1) >> cx_log; };
  const int64_t wide = across(kCx), places = (wide + slots - 1) / slots * slots;
  c.chain = idle_enough(wide, slots) && len * places > (kScanThreads >> kCx) * chain_r * (2 * places + 10 * wide);
  const int R = c.chain ? chain_r : walk_r;
  if (c.chain) {
    a.cx_log = kCx;
  } else {
    // stretches that a sequence fills, rounded up to a power of two
    int ty_log = 0;
    while (ty_log < 8 - kCx && (R << ty_log) < len) ++ty_log;
    a.cx_log = 8 - ty_log;
    // fewer than V stretches, or V that would fill the GPU side by side: a thread walks alone
    constexpr int kAlone = V == 4 ? 6 : V == 2 ? 7 : 8;
    if (a.cx_log > kAlone || (a.cx_log == kAlone && (a.vecs >> 8) >= h->sm_count)) a.cx_log = 8;
    // tiles of 128 positions rather than of 256 where both fill the GPU: less of the last one is past the end
    if (V == 4 && a.cx_log == kCx && R == 8 && across(kCx + 1) >= slots) ++a.cx_log;
  }
  const int64_t groups = across(a.cx_log);
  const int TT = (kScanThreads >> a.cx_log) * R;
  a.tiles = len > TT ? (len + TT - 1) / TT : 1;
  a.tile = make_div_magic32((uint32_t)TT);
  if (c.chain) {
    a.groups = make_div_magic32((uint32_t)groups);
    a.total = (uint32_t)(groups * a.tiles);
    a.pitch = (uint32_t)(batch * h->dim);
    a.group_log = group_log(groups);
    a.states = a.records + (int64_t)a.tiles * a.pitch;
  }
  // the records were sized for this call when the handle was made; a cut that does not fit them is not launched
  c.fits = !c.chain || chain_records(TT, a.pitch, len) <= h->max_records;
  const int64_t all = groups * a.tiles;
  c.device = h->device;
  c.grid = (unsigned)(c.chain && all >= slots ? slots : c.chain ? all : groups);
  return c;
}

// Sequences that single threads hold whole (k_scan_short_*): how long they may
// be, the positions that a thread of V channels has registers for, and the
// channels of a thread.  Measured, held whole and in tiles: 50000 x 9 x 64 bf16
// forward 30 and 47 us, with 16 positions 47 and 52; backward of 8 positions 77
// and 98 us; fp32 forward of 9 61 and 59; pairs of 50000 x 9 x 50 fp16 backward
// 59, single channels 75.  16-bit backwards of 9 to 16 positions are held whole,
// in pairs, so that no state before a tile is needed (50000 x 9 x 64 85 us, of 16
// 106).
constexpr int kShort = 16;
template <class T>
int32_t short_len(int32_t dim) {
  return channels_at_once(dim) == 4 && sizeof(T) == 4 ? 8 : 16;
}
template <class T, bool BACKWARD, int V>
constexpr int short_positions() {
  return V > 1 && sizeof(T) == 2 && (V == 2 || !BACKWARD) ? 2 * kShort / V : kShort / V;
}
template <class T, bool BACKWARD>
int32_t short_channels(int32_t dim, int32_t len) {
  const int V = channels_at_once(dim);
  if (V == 4 && len <= short_positions<T, BACKWARD, 4>()) return 4;
  return V > 1 && len <= short_positions<T, BACKWARD, 2>() ? 2 : 1;
}
unsigned short_grid(const Cut& c) { return (unsigned)((c.args.vecs + 127) / 128); }

// `staged`: bytes of the inputs' copies; `areas`: shared arrays of the joins.
template <int V, auto kernel, class... A>
cudaError_t launch(const Cut& c, size_t staged, int areas, cudaStream_t stream, A... a) {
  constexpr int kMostShared = 100 << 10;   // of each of the CTAs that share an SM
  // the limit is set once per kernel and device (one bit each), when it has been set
  static std::atomic<uint64_t> set{0};
  const uint64_t mine = c.device < 64 ? uint64_t(1) << c.device : 0;
  if (!(set.load(std::memory_order_relaxed) & mine)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e != cudaSuccess) return e;
    set.fetch_or(mine, std::memory_order_relaxed);
  }
  const size_t smem = staged + (size_t)areas * (kScanThreads >> c.args.cx_log) * ((V << c.args.cx_log) + 1) *
                                   sizeof(float);
  if (!c.fits || smem > kMostShared) return cudaErrorNotSupported;
  if (c.follows) return launch_dependent(kernel, c.grid, kScanThreads, smem, stream, c.args, a...);
  kernel<<<c.grid, kScanThreads, smem, stream>>>(c.args, a...);
  return cudaGetLastError();
}

// The states before a backward's tiles, where it has several.
template <class T, int V>
cudaError_t find_states(const Cut& c, View<const T> x, View<const T> g, View<T> gx, View<T> gg, const float* state_in,
                        cudaStream_t stream, std::integral_constant<int, V>) {
  ScanArgs a = c.args;
  const int64_t groups = (a.vecs + 31) / 32, most = a.tiles - 1;
  if (!c.fits) return cudaErrorNotSupported;
  if (most == 0) return cudaSuccess;
  a.groups = make_div_magic32((uint32_t)groups);
  k_scan_effects<T, V><<<(unsigned)(groups * most), kEffectWarps * 32, 0, stream>>>(a, x, g, gx, gg);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  a.vecs = (int64_t)a.batch * a.dim;
  a.per = make_div_magic32((uint32_t)a.dim);
  int warps = 1, ctas = 1;   // about four tiles each, and no more than are read at once if there are warps enough
  while (warps < kStateWarps && warps * 4 < most) warps *= 2;
  while (ctas < kStateCtas && ctas * kStateWarps * kStateRows < most) ctas *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.vecs + 31) / 32 * ctas));
  cfg.blockDim = dim3(warps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const int64_t parts = warps * ctas;
  return cudaLaunchKernelEx(&cfg, k_scan_states<T>, a, (int)((most + parts - 1) / parts), gx, gg, state_in);
}

// All views wide, with the first one's strides: the kernels of this variant
// have no other path.
template <int V, class... W>
bool all_wide(int size, const scan_view* first, const W*... w) {
  const auto same = [&](const scan_view* v) {
    return aligned_to(v->data, V * size) && v->batch_stride == first->batch_stride &&
           v->time_stride == first->time_stride;
  };
  return first->batch_stride % V == 0 && first->time_stride % V == 0 && same(first) && (same(w) && ...);
}

// Calls f with the channels that a thread takes as a constant.
template <class F>
cudaError_t with_channels(int32_t dim, F f) {
  switch (channels_at_once(dim)) {
    case 4: return f(std::integral_constant<int, 4>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, 1>());
  }
}
// Calls f with truth values as constants.
template <class F>
auto with_flag(bool a, F f) {
  return a ? f(std::true_type()) : f(std::false_type());
}
template <class F>
auto with_flags(bool a, bool b, F f) {
  return with_flag(a, [&](auto x) { return with_flag(b, [&](auto y) { return f(x, y); }); });
}

}  // namespace emb

using namespace emb;

extern "C" emb_status scan_create(int32_t dim, int32_t max_batch, int32_t max_len, emb_scan* out) {
  if (!out) return EMB_ERR_INVALID_ARG;
  *out = nullptr;
  if (dim < 1 || max_batch < 1 || max_len < 1) return EMB_ERR_INVALID_ARG;
  if (dim > 65536 || max_len > (1 << 30)) return EMB_ERR_UNSUPPORTED;
  emb_scan_s* h = new (std::nothrow) emb_scan_s();
  if (!h) return EMB_ERR_OOM;
  h->dim = dim;
  h->max_batch = max_batch;
  h->max_len = max_len;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) {
    const int64_t slots = (int64_t)h->sm_count * kCtasPerSm, most = most_chained(slots) * 32;
    const int64_t all = (int64_t)max_batch * dim;
    const int V = channels_at_once(dim), TT = V == 4 ? least_tile<4>() : V == 2 ? least_tile<2>() : least_tile<1>();
    h->max_records = chain_records(TT, all < most ? all : most, max_len);
    e = dev_alloc((void**)&h->status_d, sizeof(uint32_t));
  }
  if (e == cudaSuccess) e = dev_alloc((void**)&h->shared_d, sizeof(ScanShared));
  if (e == cudaSuccess) e = dev_alloc((void**)&h->records_d, sizeof(ulonglong2) * h->max_records);
  if (e == cudaSuccess) e = cudaMemset(h->status_d, 0, sizeof(uint32_t));
  const ScanShared first{0, 0, 1, 0};   // epoch 0 is what cleared records hold
  if (e == cudaSuccess) e = cudaMemcpy(h->shared_d, &first, sizeof(first), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemset(h->records_d, 0, sizeof(ulonglong2) * h->max_records);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    dev_free(h->status_d);
    dev_free(h->shared_d);
    dev_free(h->records_d);
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
  dev_free(h->shared_d);
  dev_free(h->records_d);
  delete h;
  return cuda_status(e);
}

extern "C" emb_status scan_get_device_status(emb_scan h, void* stream) {
  if (!h) return EMB_ERR_INVALID_ARG;
  // read and cleared in the stream's own order: a clear on another stream could
  // come after the next call has latched an error
  uint32_t st = 0;
  EMB_CUDA_TRY(cudaMemcpyAsync(&st, h->status_d, sizeof(uint32_t), cudaMemcpyDeviceToHost, (cudaStream_t)stream));
  EMB_CUDA_TRY(cudaMemsetAsync(h->status_d, 0, sizeof(uint32_t), (cudaStream_t)stream));
  EMB_CUDA_TRY(cudaStreamSynchronize((cudaStream_t)stream));
  return (emb_status)st;
}

extern "C" emb_status scan_forward(emb_scan h, int32_t batch, int32_t len, int32_t dtype, const scan_view* x,
                                   const scan_view* gate, const int32_t* offsets, const float* state_in,
                                   const scan_view* y, float* state_out, void* stream) {
  if (!call_ok(h, batch, len, dtype) || !view_ok(x, dtype, batch, len, h->dim, false) ||
      !view_ok(gate, dtype, batch, len, h->dim, false) || !view_ok(y, dtype, batch, len, h->dim, true))
    return EMB_ERR_INVALID_ARG;
  if (batch == 0) return EMB_OK;
  if ((int64_t)batch * h->dim >= (int64_t(1) << 32)) return EMB_ERR_UNSUPPORTED;
  return cuda_status(with_element(dtype, [&](auto* e) {
    using T = std::remove_pointer_t<decltype(e)>;
    if (len <= short_len<T>(h->dim))
      return with_channels(short_channels<T, false>(h->dim, len), [&](auto v) {
        constexpr int V = decltype(v)::value, U = kShort / V, most = short_positions<T, false, V>();
        const Cut c = cut_call<V>(h, batch, len, offsets, 1, 1);
        const auto kernel = with_flag(all_wide<V>(sizeof(T), x, gate, y), [&](auto wide) {
          constexpr bool W = decltype(wide)::value;
          return len <= 2   ? k_scan_short_fwd<T, V, 2, W>
                 : len <= U ? k_scan_short_fwd<T, V, U, W>
                            : k_scan_short_fwd<T, V, most, W>;
        });
        kernel<<<short_grid(c), 128, 0, (cudaStream_t)stream>>>(
            c.args, as_view<const T, V>(x), as_view<const T, V>(gate), as_view<T, V>(y), state_in, state_out);
        return cudaGetLastError();
      });
    return with_channels(h->dim, [&](auto v) {
      constexpr int V = decltype(v)::value, R = fwd_positions<V>();
      const Cut c = cut_call<V>(h, batch, len, offsets, R, R);
      return with_flags(c.chain, all_wide<V>(sizeof(T), x, gate, y), [&](auto chain, auto wide) {
        return launch<V, k_scan_fwd<T, V, R, decltype(chain)::value, decltype(wide)::value>>(
            c, 2 * R * kScanThreads * V * sizeof(T), 2, (cudaStream_t)stream, as_view<const T, V>(x),
            as_view<const T, V>(gate), as_view<T, V>(y), state_in, state_out);
      });
    });
  }));
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
  if ((int64_t)batch * h->dim >= (int64_t(1) << 32)) return EMB_ERR_UNSUPPORTED;
  return cuda_status(with_element(dtype, [&](auto* e) {
    using T = std::remove_pointer_t<decltype(e)>;
    if (len <= short_len<T>(h->dim))
      return with_channels(short_channels<T, true>(h->dim, len), [&](auto v) {
        constexpr int V = decltype(v)::value, U = kShort / V, most = short_positions<T, true, V>();
        const Cut c = cut_call<V>(h, batch, len, offsets, 1, 1);
        const auto kernel = with_flag(all_wide<V>(sizeof(T), x, gate, grad_y, grad_x, grad_gate), [&](auto wide) {
          constexpr bool W = decltype(wide)::value;
          return len <= 2   ? k_scan_short_bwd<T, V, 2, W>
                 : len <= U ? k_scan_short_bwd<T, V, U, W>
                            : k_scan_short_bwd<T, V, most, W>;
        });
        kernel<<<short_grid(c), 128, 0, (cudaStream_t)stream>>>(
            c.args, as_view<const T, V>(x), as_view<const T, V>(gate), as_view<const T, V>(grad_y), state_in,
            grad_state_out, as_view<T, V>(grad_x), as_view<T, V>(grad_gate), grad_state_in);
        return cudaGetLastError();
      });
    return with_channels(h->dim, [&](auto v) {
      constexpr int V = decltype(v)::value;
      Cut c = cut_call<V>(h, batch, len, offsets, bwd_positions<T, V, true>(), bwd_positions<T, V, false>());
      if constexpr (sizeof(T) == 2) {
        const cudaError_t e = find_states(c, as_view<const T, V>(x), as_view<const T, V>(gate),
                                          as_view<T, V>(grad_x), as_view<T, V>(grad_gate), state_in,
                                          (cudaStream_t)stream, std::integral_constant<int, V>());
        if (e != cudaSuccess) return e;
        c.follows = c.args.tiles > 1;
      }
      const bool same = all_wide<V>(sizeof(T), x, gate, grad_y, grad_x, grad_gate);   // of y: single elements
      return with_flags(c.chain, same, [&](auto chain, auto wide) {
        constexpr int R = bwd_positions<T, V, decltype(chain)::value>();
        return launch<V, k_scan_bwd<T, V, R, decltype(chain)::value, decltype(wide)::value>>(
            c, 3 * R * kScanThreads * V * sizeof(T), 3, (cudaStream_t)stream,
            as_view<const T, V>(x), as_view<const T, V>(gate), as_view<const T, V>(y), as_view<const T, V>(grad_y),
            state_in, grad_state_out, as_view<T, V>(grad_x), as_view<T, V>(grad_gate), grad_state_in);
      });
    });
  }));
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
  const auto fits = [&](int v) {
    return dim % v == 0 && x_stride % v == 0 && gate_stride % v == 0 && y_stride % v == 0 && aligned_to(x, v * size) &&
           aligned_to(gate, v * size) && aligned_to(y, v * size) && aligned_to(states, v * sizeof(float));
  };
  const int v = fits(4) ? 4 : fits(2) ? 2 : 1, vecs = dim / v;
  const int64_t need = (n * vecs + 127) / 128;
  const unsigned grid = (unsigned)(need < (1 << 20) ? need : (1 << 20));
  with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    auto kernel = v == 4 ? k_scan_step<T, 4> : v == 2 ? k_scan_step<T, 2> : k_scan_step<T, 1>;
    kernel<<<grid, 128, 0, (cudaStream_t)stream>>>(n, make_div_magic((uint64_t)vecs), (const T*)x, x_stride,
                                                  (const T*)gate, gate_stride, rows, states, num_rows, (T*)y,
                                                  y_stride);
  });
  return cuda_status(cudaGetLastError());
}

// A sequence of four tiles of which only the last is handed out.
extern "C" emb_status scan_selftest_timeout(uint32_t* latched, uint32_t* latched_after, float* wait_ms) {
  if (!latched || !latched_after) return EMB_ERR_INVALID_ARG;
  constexpr int dim = 32, len = 4 * (kScanThreads >> long_cx<4>()) * fwd_positions<4>();
  emb_scan h = nullptr;
  emb_status st = scan_create(dim, 1, len, &h);
  if (st != EMB_OK) return st;
  float* buf = nullptr;   // x, gate and y
  cudaEvent_t a = nullptr, b = nullptr;
  cudaError_t e = dev_alloc((void**)&buf, sizeof(float) * dim * len * 3);
  if (e == cudaSuccess) e = cudaMemset(buf, 0, sizeof(float) * dim * len * 3);
  if (e == cudaSuccess) e = cudaEventCreate(&a);
  if (e == cudaSuccess) e = cudaEventCreate(&b);
  const uint32_t last = 3;
  if (e == cudaSuccess) e = cudaMemcpy(&h->shared_d->ticket, &last, sizeof(last), cudaMemcpyHostToDevice);
  const scan_view x{buf, dim * len, dim}, g{buf + dim * len, dim * len, dim}, y{buf + 2 * dim * len, dim * len, dim};
  for (uint32_t* out : {latched, latched_after}) {
    if (e != cudaSuccess) break;
    e = cudaEventRecord(a, nullptr);
    if (e == cudaSuccess) st = scan_forward(h, 1, len, EMB_DT_F32, &x, &g, nullptr, nullptr, &y, nullptr, nullptr);
    if (e == cudaSuccess && st == EMB_OK) e = cudaEventRecord(b, nullptr);
    if (e == cudaSuccess && st == EMB_OK) *out = (uint32_t)scan_get_device_status(h, nullptr);
    if (e == cudaSuccess && st == EMB_OK && out == latched && wait_ms) e = cudaEventElapsedTime(wait_ms, a, b);
    if (st != EMB_OK) break;
  }
  if (a) cudaEventDestroy(a);
  if (b) cudaEventDestroy(b);
  dev_free(buf);
  scan_destroy(h);
  return st != EMB_OK ? st : cuda_status(e);
}
