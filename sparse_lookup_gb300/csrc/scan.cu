// scan.cu -- gated linear recurrence over padded sequences, forward, backward
// and one position at a time (scan_* in emb.h).
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
  int sm_count = 0;
  int64_t max_records = 0;
  uint32_t* status_d = nullptr;
  emb::ScanShared* shared_d = nullptr;
  ulonglong2* records_d = nullptr;   // [tiles][channels] what a tile does to a state (below)
};

namespace emb {

constexpr int kScanThreads = 256;
constexpr unsigned kScanSpins = 1u << 21;   // rounds a wait takes at most (about a second)
constexpr int kGroup = 32;                  // tiles of a chain's group
constexpr int kAhead = 4;                   // records of a group that one lane reads
constexpr int kCtasPerSm = 2;

// sigmoid(g) and sigmoid(-g) from one exponential: with e = exp(-g), a = 1 /
// (1 + e) and 1 - a = e a keeps every digit where the gate saturates.  e stops
// at 2^126 (gates below -87 then leave 2^-126 of the state); NaN goes through.
// A gate of +infinity gives exactly (1, 0): positions that are not there.
__device__ __forceinline__ void gates(float g, float& a, float& na) {
  float e;
  asm("min.NaN.f32 %0, %1, 0f42FC0000;" : "=f"(e) : "f"(g * -1.44269504f));
  asm("ex2.approx.f32 %0, %0;" : "+f"(e));
  asm("rcp.approx.f32 %0, %1;" : "=f"(a) : "f"(1.f + e));
  na = e * a;
}

// `wide`: every column vector of the view can be moved in one access.  The
// others are moved element by element by the same threads, so results do not
// depend on strides and alignment.
template <class T>
struct View {
  T* p;
  int64_t bs, ts;
  bool wide;
  __device__ T* at(int64_t b, int64_t t, int64_t d) const { return p + b * bs + t * ts + d; }
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

// A call's shape.  A tile is TT = (256 / cx) * R positions of cx column vectors
// of V channels; a column vector is V neighbouring channels of one batch entry.
struct ScanArgs {
  int32_t batch, len, dim;
  int32_t cx_log;        // column vectors of a tile, log2
  int32_t tiles;         // along time
  uint32_t total;        // tiles in all (chained calls)
  int64_t vecs;          // column vectors in all: batch * dim / V
  DivMagic per;          // by dim / V: a column vector's batch entry
  DivMagic32 groups;     // by the tiles across (chained calls)
  const int32_t* offsets;
  uint32_t* status;
  ScanShared* shared;
  ulonglong2* records;
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
// groups of kGroup tiles.  A tile writes its own effect for the later tiles of
// its group, and a group's last tile the state after the group; a tile joins
// the effects ahead of it in its group, read at once by the channel's J =
// kGroup / kAhead lanes, behind the state before the group.  Along a sequence
// only the groups wait for one another in turn (one write and read in L2 per
// kGroup tiles), and the order of every join is fixed: results repeat bit for
// bit.  `all`: what this tile does; `next`: a later tile needs to know; state0:
// the state before tile 0.  All lanes of the warp call; the arguments are
// uniform over a channel's lanes.
__device__ __forceinline__ float chain_state(const ScanArgs& s, int64_t col, int i, bool want, bool next, Affine all,
                                             float state0, uint32_t epoch) {
  constexpr int J = kGroup / kAhead;
  const int64_t pitch = (int64_t)s.batch * s.dim;
  ulonglong2 *own = s.records + col, *states = s.records + s.tiles * pitch + col;
  const int j = threadIdx.x & (J - 1), m = i / kGroup, at = i % kGroup;
  if (want && next && j == 0 && at != kGroup - 1) put_record(own + i * pitch, all, epoch);
  Affine f[kAhead], st{0.f, state0};
  bool have[kAhead], have_state = !want || m == 0 || j != 0;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    f[u] = {1.f, 0.f};
    have[u] = !want || j * kAhead + u >= at;
  }
  for (unsigned spins = 0;; ++spins) {
    bool all_here = true;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (!have[u]) have[u] = get_record(own + (m * kGroup + j * kAhead + u) * pitch, f[u]) == epoch;
    if (!have_state) have_state = get_record(states + m * pitch, st) == epoch;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) all_here = all_here && have[u];
    if (__all_sync(kFull, all_here && have_state)) break;
    if (spins >= kScanSpins) {
      latch(s.status, EMB_ERR_TIMEOUT);
      *(volatile uint32_t*)&s.shared->fail = 1u;
      break;
    }
    if ((spins & 255u) == 255u && __any_sync(kFull, *(volatile uint32_t*)&s.shared->fail != 0u)) break;
  }
  Affine sum = f[0];
#pragma unroll
  for (int u = 1; u < kAhead; ++u) sum = after(f[u], sum);
#pragma unroll
  for (int o = 1; o < J; o <<= 1) {
    const Affine e{__shfl_down_sync(kFull, sum.a, o, J), __shfl_down_sync(kFull, sum.b, o, J)};
    sum = after(e, sum);   // the upper lanes' sums are not used
  }
  const float h = __shfl_sync(kFull, fmaf(sum.a, st.b, sum.b), 0, J);
  if (want && next && j == 0 && at == kGroup - 1)
    put_record(states + (m + 1) * pitch, {0.f, fmaf(all.a, h, all.b)}, epoch);
  return h;
}

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
  if (!c.ok) vec = 0;
  c.b = (int)div_magic((uint64_t)vec, s.per);
  c.d = (int)(vec - (int64_t)c.b * (int64_t)s.per.d) * V + v;
  c.n = c.ok ? live_len(s, c.b) : 0;
  c.col = vec * V + v;
  return c;
}

// A thread's R column vectors of one input, staged in shared memory: only the
// thread itself reads what it copied, so no barrier is needed.  Copies are
// asynchronous where the view allows it; otherwise the vectors are loaded
// when they are due (`now`).  Positions at or past n hold `dead`.
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <class T, int V, int R>
struct Staged {
  static constexpr int kBytes = V * (int)sizeof(T);
  Vec<T, V>* at;   // + r * kScanThreads
  __device__ bool async(const View<const T>& w) const { return kBytes >= 4 && w.wide; }
  __device__ void fill(const View<const T>& w, const T* p, int t0, int first, int n, float dead, bool now) const {
    if (async(w) == now) return;
    Vec<T, V> z;
#pragma unroll
    for (int v = 0; v < V; ++v) z.e[v] = from_f32<T>(dead);
    if constexpr (kBytes >= 4) {
      if (!now) {
#pragma unroll
        for (int r = 0; r < R; ++r, p += w.ts) {
          Vec<T, V>* to = at + r * kScanThreads;
          if (t0 + r >= first && t0 + r < n) {
            const unsigned d = (unsigned)__cvta_generic_to_shared(to);
            if constexpr (kBytes == 16)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(p) : "memory");
            else
              asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(p), "n"(kBytes) : "memory");
          } else {
            *to = z;
          }
        }
        return;
      }
    }
    Vec<T, V> got[R];
#pragma unroll
    for (int r = 0; r < R; ++r, p += w.ts) {
      got[r] = z;
      if (t0 + r >= first && t0 + r < n) got[r] = get<V>(p, w.wide);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) at[r * kScanThreads] = got[r];
  }
};

#define SCAN_DEAD_GATE __int_as_float(0x7f800000)

// Forward.  A thread keeps R positions of V channels as (a, (1 - a) x) in
// registers, so x and gate are read once.  Its stretch's effect goes to shared
// memory, the channels' lanes join the stretches behind the state before the
// tile, and each thread then runs its positions from its own first state.  The
// next tile's inputs are copied meanwhile.
// CHAIN: a CTA takes tiles by ticket and finds the state before its tile in the
// records of the tiles ahead; otherwise it walks along time with the state in
// hand.  cx = 256: a thread is a whole stretch of its own, nothing is joined.
template <class T, int V, int R, bool CHAIN>
__global__ void __launch_bounds__(kScanThreads, kCtasPerSm) k_scan_fwd(ScanArgs s, View<const T> x, View<const T> g,
                                                                       View<T> y, const float* __restrict__ state_in,
                                                                       float* __restrict__ state_out) {
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t slot;
  const Place<V, R> p(s);
  const bool whole = s.cx_log == 8;
  const Staged<T, V, R> sx{(Vec<T, V>*)raw + threadIdx.x}, sg{sx.at + R * kScanThreads};
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
    sx.fill(x, x.at(c.b, t0, c.d), t0, 0, c.n, 0.f, now);
    sg.fill(g, g.at(c.b, t0, c.d), t0, 0, c.n, SCAN_DEAD_GATE, now);
  };
  if (!CHAIN || tile < s.total) fill(c, k, false);
  float held = 0.f;          // walking: the channel's state
  float own[V];              // whole: the thread's states
  while (CHAIN ? tile < s.total : k < s.tiles) {
    const int t0 = k * p.TT + p.ty * R;
    fill(c, k, true);
    copies_done();
    uint32_t ticket = 0;
    if (CHAIN && threadIdx.x == 0) ticket = take_ticket(s);
    float a[R][V], b[R][V], fa[V], fb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) fa[v] = 1.f, fb[v] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Vec<T, V> xr = sx.at[r * kScanThreads], gr = sg.at[r * kScanThreads];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float na;
        gates(to_f32(gr.e[v]), a[r][v], na);
        b[r][v] = na * to_f32(xr.e[v]);
        fa[v] *= a[r][v];
        fb[v] = fmaf(a[r][v], fb[v], b[r][v]);
      }
    }
    // the staged inputs are in registers: copy the next tile's.  Its ticket was
    // drawn when this tile's inputs had come, not before: a CTA that drew two
    // neighbours would publish the second only after the first's own wait.
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
      fill(c1, k1, false);
    };
    float h[V];
    if (whole) {
      ahead();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == 0) own[v] = state_in && c.ok ? state_in[c.col + v] : 0.f;
        h[v] = own[v];
        own[v] = fmaf(fa[v], own[v], fb[v]);
        if (state_out && c.ok && k == s.tiles - 1) state_out[c.col + v] = own[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sa[p.ty * p.pitch + p.cx * V + v] = fa[v];
        sb[p.ty * p.pitch + p.cx * V + v] = fb[v];
      }
      if (CHAIN && threadIdx.x == 0) slot = ticket;
      __syncthreads();
      ahead();
      const Channel q = channel_of<V>(s, (gi << s.cx_log) + p.ch / V, p.ch % V);
      Affine f[V], ex, all;
      join_stretches<V>(p, sa, sb, false, f, ex, all);
      const int end = (k + 1) * p.TT;
      const bool live = q.ok && (k * p.TT < q.n || k == 0);
      if constexpr (CHAIN) {
        const float state0 = live && k < kGroup && state_in ? state_in[q.col] : 0.f;
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
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = sb[p.ty * p.pitch + p.cx * V + v];
    }
    T* to = y.at(c.b, t0, c.d);
#pragma unroll
    for (int r = 0; r < R; ++r, to += y.ts) {
      const int t = t0 + r;
      Vec<T, V> o;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = fmaf(a[r][v], h[v], b[r][v]);
        o.e[v] = from_f32<T>(t < c.n ? h[v] : 0.f);
      }
      if (c.ok && t < s.len) put<V>(to, y.wide, o);
    }
    c = c1, k = k1, gi = gi1;
    tile = next;
  }
  if (CHAIN && threadIdx.x == 0) leave(s);
}

// Backward, from the last position to the first: C_t = a_t (grad_y_t + C_{t+1})
// is what position t passes back.  The gate's gradient needs the state before
// each position.  fp32: a tile runs forward from y just before it, which costs
// one row of y instead of all of them; both joins use the same products of
// gates.  16 bits: y is read at every position (RERUN false) -- a rerun would
// carry the rounding of the one row it starts from into states that are
// smaller than that row, where y itself is off by half a unit of its own.
template <class T, int V, int R, bool CHAIN>
__global__ void __launch_bounds__(kScanThreads, kCtasPerSm) k_scan_bwd(ScanArgs s, View<const T> x, View<const T> g,
                                                                       View<const T> y, View<const T> gy,
                                                                       const float* __restrict__ state_in,
                                                                       const float* __restrict__ grad_out, View<T> gx,
                                                                       View<T> gg, float* __restrict__ grad_in) {
  constexpr bool RERUN = sizeof(T) == 4;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t slot;
  const Place<V, R> p(s);
  const bool whole = s.cx_log == 8;
  const int area = (kScanThreads >> s.cx_log) * p.pitch;
  const Staged<T, V, R> sx{(Vec<T, V>*)raw + threadIdx.x}, sg{sx.at + R * kScanThreads},
      sd{sg.at + R * kScanThreads}, sy{sd.at + R * kScanThreads};
  float* sa = (float*)(raw + (RERUN ? 3 : 4) * R * kScanThreads * sizeof(Vec<T, V>));
  float *sb = sa + area, *sc = sb + area;
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
    sx.fill(x, x.at(c.b, t0, c.d), t0, 0, c.n, 0.f, now);
    sg.fill(g, g.at(c.b, t0, c.d), t0, 0, c.n, SCAN_DEAD_GATE, now);
    sd.fill(gy, gy.at(c.b, t0, c.d), t0, 0, c.n, 0.f, now);
    if (!RERUN) sy.fill(y, y.at(c.b, (int64_t)t0 - 1, c.d), t0, 1, c.n, 0.f, now);
  };
  if (!CHAIN || tile < s.total) fill(c, k, false);
  float held = 0.f;
  float own[V];
  while (CHAIN ? tile < s.total : k >= 0) {
    const int t0 = k * p.TT + p.ty * R;
    fill(c, k, true);
    copies_done();
    uint32_t ticket = 0;
    if (CHAIN && threadIdx.x == 0) ticket = take_ticket(s);
    float a[R][V], na[R][V], xv[R][V], dy[R][V];   // xv: x, then the gate's factor of G
    float fa[V], fb[V], fc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) fa[v] = 1.f, fb[v] = 0.f, fc[v] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Vec<T, V> xr = sx.at[r * kScanThreads], gr = sg.at[r * kScanThreads], dr = sd.at[r * kScanThreads];
      Vec<T, V> yr;
      if (!RERUN) yr = sy.at[r * kScanThreads];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gates(to_f32(gr.e[v]), a[r][v], na[r][v]);
        xv[r][v] = to_f32(xr.e[v]);
        dy[r][v] = to_f32(dr.e[v]);
        if (!RERUN) {
          float before = to_f32(yr.e[v]);
          if (r == 0 && t0 == 0) before = state_in && c.ok ? state_in[c.col + v] : 0.f;
          xv[r][v] = a[r][v] * na[r][v] * (before - xv[r][v]);
        }
        fa[v] *= a[r][v];
        if (RERUN) fb[v] = fmaf(a[r][v], fb[v], na[r][v] * xv[r][v]);
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
#pragma unroll
      for (int v = 0; v < V; ++v) fc[v] = a[r][v] * (dy[r][v] + fc[v]);
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
      fill(c1, k1, false);
    };
    float h[V], C[V];
    if (whole) {
      ahead();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == s.tiles - 1) own[v] = grad_out && c.ok ? grad_out[c.col + v] : 0.f;
        C[v] = own[v];
        own[v] = fmaf(fa[v], own[v], fc[v]);
        if (grad_in && c.ok && k == 0) grad_in[c.col + v] = own[v];
        h[v] = 0.f;
        if (!RERUN) continue;
        if (c.ok && t0 == 0) h[v] = state_in ? state_in[c.col + v] : 0.f;
        else if (t0 < c.n) h[v] = to_f32(*y.at(c.b, t0 - 1, c.d + v));
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sa[p.ty * p.pitch + p.cx * V + v] = fa[v];
        if (RERUN) sb[p.ty * p.pitch + p.cx * V + v] = fb[v];
        sc[p.ty * p.pitch + p.cx * V + v] = fc[v];
      }
      const Channel q = channel_of<V>(s, (gi << s.cx_log) + p.ch / V, p.ch % V);
      const int start = k * p.TT;
      const bool live = q.ok && (start < q.n || k == 0);
      float first = 0.f;
      if (RERUN && live) first = k == 0 ? (state_in ? state_in[q.col] : 0.f) : to_f32(*y.at(q.b, start - 1, q.d));
      if (CHAIN && threadIdx.x == 0) slot = ticket;
      __syncthreads();
      ahead();
      Affine f[V], ex, all;
      float st;
      if (RERUN) {
        join_stretches<V>(p, sa, sb, false, f, ex, all);
        st = fmaf(ex.a, first, ex.b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sb[(p.j * V + i) * p.pitch + p.ch] = st;
          st = fmaf(f[i].a, st, f[i].b);
        }
      }
      join_stretches<V>(p, sa, sc, true, f, ex, all);
      // the chain of a channel begins at the tile of its last position
      const int last = q.n > 0 ? (q.n - 1) / p.TT : 0;
      if constexpr (CHAIN) {
        const int i = live ? last - k : 0;
        const float state0 = live && i < kGroup && grad_out ? grad_out[q.col] : 0.f;
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
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (RERUN) h[v] = sb[p.ty * p.pitch + p.cx * V + v];
        C[v] = sc[p.ty * p.pitch + p.cx * V + v];
      }
    }
    if (RERUN) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float before = h[v];
          h[v] = fmaf(a[r][v], before, na[r][v] * xv[r][v]);
          xv[r][v] = a[r][v] * na[r][v] * (before - xv[r][v]);
        }
    }
    T *tx = gx.at(c.b, (int64_t)t0 + R - 1, c.d), *tg = gg.at(c.b, (int64_t)t0 + R - 1, c.d);
#pragma unroll
    for (int r = R - 1; r >= 0; --r, tx -= gx.ts, tg -= gg.ts) {
      const int t = t0 + r;
      Vec<T, V> ox, og;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float G = dy[r][v] + C[v];
        const bool on = t < c.n;
        ox.e[v] = from_f32<T>(on ? na[r][v] * G : 0.f);
        og.e[v] = from_f32<T>(on ? xv[r][v] * G : 0.f);
        C[v] = a[r][v] * G;
      }
      if (c.ok && t < s.len) {
        put<V>(tx, gx.wide, ox);
        put<V>(tg, gg.wide, og);
      }
    }
    c = c1, k = k1, gi = gi1;
    tile = next;
  }
  if (CHAIN && threadIdx.x == 0) leave(s);
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


template <class T, int V>
View<T> as_view(const scan_view* v) {
  return View<T>{(T*)v->data, v->batch_stride, v->time_stride,
                 aligned_to(v->data, V * sizeof(T)) && v->batch_stride % V == 0 && v->time_stride % V == 0};
}

bool call_ok(emb_scan h, int32_t batch, int32_t len, int32_t dtype) {
  return h && batch >= 0 && batch <= h->max_batch && len >= 0 && len <= h->max_len && dtype_size(dtype) != 0;
}

// How a call is cut.  R: positions of a thread.
struct Cut {
  ScanArgs args;
  bool chain;
  unsigned grid;
  size_t smem;
};

constexpr int kWideV = 4, kFwdR = 8, kBwdR = 4;   // V = 1: twice the positions, for as many bytes in flight
constexpr int kChainCx = 3, kWalkCx = 5;          // log2 of the column vectors of a tile
int64_t chain_records(int64_t dim, int64_t batch, int64_t len, int V, int R, int sms) {
  const int64_t cols = batch * dim;
  (void)sms;
  const int TT = (kScanThreads >> (V == 1 ? 5 : kChainCx)) * R;
  const int64_t tiles = (len + TT - 1) / TT;
  return (tiles + tiles / kGroup + 1) * cols;
}

Cut cut_call(const emb_scan_s* h, int32_t batch, int32_t len, const int32_t* offsets, int V, int R, int areas,
             size_t staged) {
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
  const int64_t slots = (int64_t)h->sm_count * kCtasPerSm;
  c.chain = (a.vecs >> kWalkCx) < slots;
  a.cx_log = c.chain ? (V == 1 ? 5 : kChainCx) : kWalkCx;
  const int TT = (kScanThreads >> a.cx_log) * R;
  a.tiles = (len + TT - 1) / TT;
  if (a.tiles < 1) a.tiles = 1;
  const int64_t groups = (a.vecs + (1 << a.cx_log) - 1) >> a.cx_log;
  if (a.tiles == 1) c.chain = false;
  a.per = make_div_magic((uint64_t)(h->dim / V));
  if (c.chain) {
    a.groups = make_div_magic32((uint32_t)groups);
    a.total = (uint32_t)(groups * a.tiles);
  }
  const int64_t all = groups * a.tiles;
  c.grid = (unsigned)(c.chain ? (all < slots ? all : slots) : groups);
  c.smem = staged + (size_t)areas * (kScanThreads >> a.cx_log) * ((V << a.cx_log) + 1) * sizeof(float);
  return c;
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
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) {
    const int64_t cols = (int64_t)h->sm_count * kCtasPerSm * (kWideV << kWalkCx) + dim;   // a call with more walks
    const int64_t batch = (int64_t)max_batch * dim < cols ? max_batch : cols / dim + 1;
    for (int V : {1, kWideV})
      for (int R : {kFwdR, kBwdR}) {
        const int64_t n = chain_records(dim, batch, max_len, V, V == 1 ? 2 * R : R, h->sm_count);
        if (n > h->max_records) h->max_records = n;
      }
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
  uint32_t st = 0;
  EMB_CUDA_TRY(cudaStreamSynchronize((cudaStream_t)stream));
  EMB_CUDA_TRY(cudaMemcpy(&st, h->status_d, sizeof(uint32_t), cudaMemcpyDeviceToHost));
  EMB_CUDA_TRY(cudaMemset(h->status_d, 0, sizeof(uint32_t)));
  return (emb_status)st;
}

template <class K>
static cudaError_t allow_shared(K kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 << 10);
}

template <class T, int V, int R>
static cudaError_t launch_fwd(const emb_scan_s* h, int32_t batch, int32_t len, const scan_view* x, const scan_view* gate,
                       const int32_t* offsets, const float* state_in, const scan_view* y, float* state_out,
                       cudaStream_t stream) {
  const Cut c = cut_call(h, batch, len, offsets, V, R, 2, 2 * R * kScanThreads * V * sizeof(T));
  auto kernel = c.chain ? k_scan_fwd<T, V, R, true> : k_scan_fwd<T, V, R, false>;
  static const cudaError_t room[2] = {allow_shared(k_scan_fwd<T, V, R, false>), allow_shared(k_scan_fwd<T, V, R, true>)};
  if (room[c.chain] != cudaSuccess) return room[c.chain];
  kernel<<<c.grid, kScanThreads, c.smem, stream>>>(c.args, as_view<const T, V>(x), as_view<const T, V>(gate), as_view<T, V>(y),
                                                  state_in, state_out);
  return cudaGetLastError();
}

template <class T, int V, int R>
static cudaError_t launch_bwd(const emb_scan_s* h, int32_t batch, int32_t len, const scan_view* x, const scan_view* gate,
                       const int32_t* offsets, const float* state_in, const scan_view* y, const scan_view* grad_y,
                       const float* grad_state_out, const scan_view* grad_x, const scan_view* grad_gate,
                       float* grad_state_in, cudaStream_t stream) {
  const Cut c = cut_call(h, batch, len, offsets, V, R, 3, (sizeof(T) == 4 ? 3 : 4) * R * kScanThreads * V * sizeof(T));
  auto kernel = c.chain ? k_scan_bwd<T, V, R, true> : k_scan_bwd<T, V, R, false>;
  static const cudaError_t room[2] = {allow_shared(k_scan_bwd<T, V, R, false>), allow_shared(k_scan_bwd<T, V, R, true>)};
  if (room[c.chain] != cudaSuccess) return room[c.chain];
  kernel<<<c.grid, kScanThreads, c.smem, stream>>>(c.args, as_view<const T, V>(x), as_view<const T, V>(gate),
                                                  as_view<const T, V>(y), as_view<const T, V>(grad_y), state_in,
                                                  grad_state_out, as_view<T, V>(grad_x), as_view<T, V>(grad_gate),
                                                  grad_state_in);
  return cudaGetLastError();
}

extern "C" emb_status scan_forward(emb_scan h, int32_t batch, int32_t len, int32_t dtype, const scan_view* x,
                                   const scan_view* gate, const int32_t* offsets, const float* state_in,
                                   const scan_view* y, float* state_out, void* stream) {
  if (!call_ok(h, batch, len, dtype) || !view_ok(x, dtype, batch, len, h->dim, false) ||
      !view_ok(gate, dtype, batch, len, h->dim, false) || !view_ok(y, dtype, batch, len, h->dim, true))
    return EMB_ERR_INVALID_ARG;
  if (batch == 0) return EMB_OK;
  const bool vec = h->dim % kWideV == 0;
  return cuda_status(with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    auto launch = vec ? launch_fwd<T, kWideV, kFwdR> : launch_fwd<T, 1, 2 * kFwdR>;
    return launch(h, batch, len, x, gate, offsets, state_in, y, state_out, (cudaStream_t)stream);
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
  const bool vec = h->dim % kWideV == 0;
  return cuda_status(with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    auto launch = vec ? launch_bwd<T, kWideV, kBwdR> : launch_bwd<T, 1, 2 * kBwdR>;
    return launch(h, batch, len, x, gate, offsets, state_in, y, grad_y, grad_state_out, grad_x, grad_gate,
                  grad_state_in, (cudaStream_t)stream);
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
  const unsigned grid = (unsigned)(n < (1 << 20) ? n : (1 << 20));
  with_element(dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_scan_step<T><<<grid, 256, 0, (cudaStream_t)stream>>>(n, dim, (const T*)x, x_stride, (const T*)gate, gate_stride,
                                                         rows, states, num_rows, (T*)y, y_stride);
  });
  return cuda_status(cudaGetLastError());
}
