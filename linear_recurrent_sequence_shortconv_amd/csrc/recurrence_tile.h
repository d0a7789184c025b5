// Tiles of the gated recurrence and of its backward pass.
//
// Memory bound at the copy's rate if every value is read and written once, so
// the tokens are divided although each needs the state of the one before:
// a workgroup takes a tile of W strips of R rows and 64 V channels, a strip a
// wave, V channels a lane.  A strip's effect on the state is h -> A h + U (A the
// product of its decays, U what it leaves of a state of 0), so a wave sweeps its
// strip twice, in registers: for (A, U), and, from the state that enters it, for
// the results.  Between the sweeps the strips of a tile are joined through LDS,
// and the tiles of a sequence through one 64-bit word (A, U) a channel: a tile
// writes its own (A, U) there as soon as it has it, and (0, h) once it knows the
// state h behind it.  A tile reads the words of up to LOOK tiles before it and
// carries the state on from the nearest word with A = 0, by the same operations
// in the same order whichever word that is, so that results do not depend on
// timing.  Workgroups take their tiles in order from a counter: a tile waits for
// tiles alone whose workgroups run already, down to the first, which waits for
// none, so every wait ends.
//
// Rows of a batch follow one another through the tiles; where a sequence starts,
// A is 0 and the state h0.  The backward pass goes through rows and tiles in
// reverse, its state the gradient a_t g_t that a token hands to the one before.
//
// bf16, gates by power with an input gate, 2048 channels: one sequence of 16384 tokens
// 66 us, 4.0 TB/s, backward of 8 x 2048 tokens 129 us, 4.2 TB/s.  fp32, 8 x 1024 tokens:
// 72 us, 3.7 TB/s, bound by the vector units (99 instructions a value for the bf16
// kernel's 33, in three quarters of the cycles).  In the middle of a
// launch tiles move 4.7 to 4.9 TB/s; the rest is the kernel that readies the words
// (5 us), the first workgroups, which load before any computes, and the last.
#pragma once

#include "recurrence_kernel.h"
#include "tile_place.h"

namespace prism {

// Words of the tiles (nullptr: no tile needs another's), the counter, and the
// states to start from.
struct TileArgs {
  unsigned long long* words;   // [tiles][slices * 64 V]
  unsigned* counter;
  int tiles, slices;
  const float* first;          // h0, or dhT (nullptr: zeros)
  int flat;                    // the batches' rows follow one another in every tensor
};

constexpr unsigned NOT_YET = 0xffffffffu;   // of a word's A: nothing written so far
// Looks at the words before a wait ends by itself, with a state that is not a
// number: about a second, where waits of a correct call end within milliseconds.
// (Two calls at the same time on one workspace, which is an error, could otherwise
// wait for ever.)
constexpr int MOST_LOOKS = 1 << 20;
constexpr unsigned long long NO_STATE = 0x7fc00000ull << 32;   // (0, not a number)
// Words a tile reads at once, and waves a SIMD has registers for: with few tiles
// in all, the state goes from tile to tile faster if they look further; with many,
// their registers and reads cost more (figures at the choice).
constexpr int LOOK = 4, WAVES = 4, LOOK_FAR = 16, WAVES_FAR = 2;
constexpr int FAR_TILES = 512, FAR_CHAIN = 32;   // tiles at most in all, at least in a sequence

__device__ inline float through(float A, float U, float h) { return A == 0.f ? U : fmaf(A, h, U); }

__device__ inline void publish(unsigned long long* w, float A, float U) {
  unsigned a = __float_as_uint(A);
  if (a == NOT_YET) a = 0x7fc00000u;   // (one NaN for another)
  const unsigned long long v = (unsigned long long)__float_as_uint(U) << 32 | a;
  __hip_atomic_store(w, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state behind tile `tile - step` (step 1: forward, -1: backward) for the
// lane's V channels, by a whole wave; `left` tiles lie before this one.
template <int V, int L>
__device__ inline void look_back(const unsigned long long* words, long stride, int tile, int step, int left,
                                 float (&h)[V]) {
  unsigned long long w[L][V];
  auto load = [&](int k, int v) {
    return __hip_atomic_load(words + (tile - step * (k + 1)) * stride + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
#pragma unroll
  for (int k = 0; k < L; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) w[k][v] = k < left ? load(k, v) : 0;
  for (int looks = 0;; ++looks) {
    // whether all are written, and whether those between the tile and a state are
    bool written = true, known = true, found[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      found[v] = false;
#pragma unroll
      for (int k = 0; k < L; ++k) {
        const bool there = (unsigned)w[k][v] != NOT_YET;
        written = written && there;
        known = known && (found[v] || there);
        found[v] = found[v] || __uint_as_float((unsigned)w[k][v]) == 0.f;
      }
      known = known && found[v];
    }
    if (__all(known)) break;
    if (__all(written)) {   // (left >= L then: no word is a state, and the furthest will be)
      while (true) {
        bool state = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          w[L - 1][v] = ++looks < MOST_LOOKS ? load(L - 1, v) : NO_STATE;
          state = state && (found[v] || __uint_as_float((unsigned)w[L - 1][v]) == 0.f);
        }
        if (__all(state)) break;
      }
      break;
    }
    __builtin_amdgcn_s_sleep(1);
#pragma unroll
    for (int k = 0; k < L; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((unsigned)w[k][v] == NOT_YET) w[k][v] = looks < MOST_LOOKS ? load(k, v) : NO_STATE;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = 0.f;
#pragma unroll
    for (int k = L - 1; k >= 0; --k)
      h[v] = through(__uint_as_float((unsigned)w[k][v]), __uint_as_float((unsigned)(w[k][v] >> 32)), h[v]);
  }
}

// Rows a strip and waves a tile, forward and backward: the most rows whose values
// fit the registers of 4 waves a SIMD (backward keeps five values a row where
// forward keeps two), and a tile that lasts longer than a state takes from one to
// the next.
constexpr int REC_R = 16, REC_W = 8, REC_BWD_R = 8, REC_BWD_W = 8;

// Which rows of a strip start and end a sequence and which belong to one, as
// bits, and the sequence of row k in lane k.
struct Strip {
  int row, n;
  unsigned first, last, in;
  int b;
  __device__ inline int batch(int k) const { return __builtin_amdgcn_readlane(b, k); }
};
template <int R>
__device__ inline Strip strip_of(const RecurrenceArgs& a, int row) {
  Strip s;
  s.row = min(row, a.rows - 1);
  s.n = min(max(a.rows - row, 0), R);
  s.first = s.last = s.in = 0;
  s.b = 0;
  if (s.n == 0) return s;
  const int lane = threadIdx.x & (WAVE - 1);
  if (!a.cu) {
    const int b = row / a.T, t = row - b * a.T;
    s.b = b;
    for (int k = t ? a.T - t : a.T; k < s.n; k += a.T) s.b += lane >= k;
    for (int k = t ? a.T - t : 0; k < s.n; k += a.T) s.first |= 1u << k;
    for (int k = a.T - 1 - t; k < s.n; k += a.T) s.last |= 1u << k;
    s.in = (1u << s.n) - 1;
  } else {
    const int end = row + s.n;
    for (int at = row; at < end;) {
      const Sequence q = find_sequence(a.cu, a.B, a.T, a.rows, at);
      const int stop = min(q.end, end);
      if (q.b >= 0 && q.b < a.B) {
        s.in |= ((1u << (stop - at)) - 1) << (at - row);
        if (q.start == at) s.first |= 1u << (at - row);
        if (q.end == stop) s.last |= 1u << (stop - 1 - row);
        if (lane >= at - row) s.b = q.b;
      }
      at = stop;
    }
  }
  return s;
}

// All rows are one sequence's, which may start with the first and end with the last.
template <int R>
__device__ inline bool plain_strip(const Strip& s) {
  return s.in == (1u << R) - 1 && !(s.first >> 1) && !(s.last & ((1u << (R - 1)) - 1));
}

// Walks a tensor's rows of a strip; rows past its end are its last.  EVEN: a full
// strip whose rows are one step apart.
template <typename E, bool EVEN>
struct RowWalk {
  const E* p;
  long step, jump;
  __device__ inline RowWalk(const void* base, const TokenSteps& s, const RecurrenceArgs& a, const TileArgs& g, int row) {
    step = s.t;
    if (g.flat) {
      p = static_cast<const E*>(base) + row * s.t;
      jump = 0;
    } else {
      const int b = row / a.T;
      p = static_cast<const E*>(base) + (b * s.b + (row - b * a.T) * s.t);
      jump = s.b - a.T * s.t;
    }
  }
  __device__ inline void next(const Strip& s, int k) {   // from row k to k + 1
    if (EVEN) {
      p += step;
    } else if (k + 1 < s.n) {
      p += step;
      if (s.first >> (k + 1) & 1) p += jump;
    }
  }
  __device__ inline void back(const Strip& s, int k) {   // from row k to k - 1
    if (EVEN) {
      p -= step;
    } else if (k > 0 && k < s.n) {
      p -= step;
      if (s.first >> k & 1) p -= jump;
    }
  }
};

// A lane's values of a row: the row's address is the wave's, the offset of 32 bits
// the lane's, which one instruction adds by itself.
template <typename E, int V>
__device__ inline typename VecIo<E, V>::raw load_raw(const E* p, int c) {
  return *reinterpret_cast<const typename VecIo<E, V>::raw*>(reinterpret_cast<const char*>(p) +
                                                             (unsigned)c * (unsigned)sizeof(E));
}
template <typename E, int V>
__device__ inline void store_values(const E* p, int c, const float (&x)[V]) {
  *reinterpret_cast<typename VecIo<E, V>::raw*>(const_cast<char*>(reinterpret_cast<const char*>(p)) +
                                                (unsigned)c * (unsigned)sizeof(E)) = VecIo<E, V>::pack(x);
}

// Values that enter each strip, from the strips' (A, U) in LDS and, where the
// tile's first row (backward: last) goes on from another tile, from its words.
// `strip` counts in the direction of the pass.
template <int V, int W, int L>
__device__ inline void enter_strip(const TileArgs& g, int tile, int slice, int step, int left, bool open, int strip,
                                   const float (&A)[V], const float (&U)[V], float (&h)[V]) {
  __shared__ float sA[W][V][WAVE], sU[W][V][WAVE], s0[V][WAVE];
  const int lane = threadIdx.x & (WAVE - 1);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sA[strip][v][lane] = A[v];
    sU[strip][v][lane] = U[v];
  }
  __syncthreads();
  if (strip == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (g.words) {
      float At[V], Ut[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        At[v] = 1.f;
        Ut[v] = 0.f;
        for (int k = 0; k < W; ++k) {
          Ut[v] = through(sA[k][v][lane], sU[k][v][lane], Ut[v]);
          At[v] = sA[k][v][lane] == 0.f ? 0.f : At[v] * sA[k][v][lane];
        }
      }
      const long stride = (long)g.slices * WAVE * V;
      unsigned long long* w = g.words + tile * stride + (slice * WAVE + lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) publish(w + v, open ? At[v] : 0.f, Ut[v]);
      if (open) {
        look_back<V, L>(g.words + (slice * WAVE + lane) * V, stride, tile, step, left, h);
#pragma unroll
        for (int v = 0; v < V; ++v) publish(w + v, 0.f, through(At[v], Ut[v], h[v]));
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s0[v][lane] = h[v];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = s0[v][lane];
    for (int k = 0; k < strip; ++k) h[v] = through(sA[k][v][lane], sU[k][v][lane], h[v]);
  }
}

// The workgroup's place in the order of tiles and slices.
__device__ inline TilePlace take_tile(const TileArgs& g) {
  if (!g.words) return tile_place(blockIdx.x, g.tiles, g.slices);
  __shared__ unsigned taken;
  if (threadIdx.x == 0)
    taken = __hip_atomic_fetch_add(g.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return tile_place(__builtin_amdgcn_readfirstlane(taken), g.tiles, g.slices);
}

// A lane's values of a state [B, D] (nullptr: zeros).
template <int V>
__device__ inline void load_state(const float* p, int b, int D, int c, float (&h)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = p ? p[(long)b * D + c + v] : 0.f;
}
template <int V>
__device__ inline void store_state(float* p, int b, int D, int c, const float (&h)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) p[(long)b * D + c + v] = h[v];
}

// A strip's part of a pass: its values in registers, the sweep for (A, U), and the
// sweep from the state that enters it.  PLAIN: a plain strip with channels for all
// lanes; EVEN: its rows are one step apart.
template <typename E, int V, int G, bool INP, int R>
struct ForwardStrip {
  typedef typename VecIo<E, V>::raw raw;
  typedef VecIo<E, V> IO;
  float lam[V], av[R][V], uv[R][V], start[V];   // start: before the first sequence that starts here

  template <bool PLAIN, bool EVEN>
  __device__ inline void first_sweep(const RecurrenceArgs& a, const TileArgs& g, const Strip& s, int c, float (&A)[V],
                                     float (&U)[V]) {
    raw rx[R], rf[R], ri[R];
    const int f0 = s.first ? __builtin_ctz(s.first) : 0;
    if (s.first) load_state<V>(g.first, s.batch(f0), a.D, c, start);
    RowWalk<E, EVEN> px(a.x, a.sx, a, g, s.row), pf(a.f, a.sf, a, g, s.row),
        pi(INP ? a.i : a.x, INP ? a.si : a.sx, a, g, s.row);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      rx[k] = load_raw<E, V>(px.p, c);
      rf[k] = load_raw<E, V>(pf.p, c);
      if (INP) ri[k] = load_raw<E, V>(pi.p, c);
      px.next(s, k);
      pf.next(s, k);
      if (INP) pi.next(s, k);
    }
    if (PLAIN && s.first) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] = 0.f;
        U[v] = start[v];
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float x[V], f[V], i[V];
      IO::unpack(rx[k], x);
      IO::unpack(rf[k], f);
      if (INP) IO::unpack(ri[k], i);
#pragma unroll
      for (int v = 0; v < V; ++v) gate_inputs<E, G, INP>(x[v], f[v], INP ? i[v] : 0.f, lam[v], av[k][v], uv[k][v]);
      if (!PLAIN && (s.first >> k & 1)) {
        float h0[V];
        if (k == f0) {
#pragma unroll
          for (int v = 0; v < V; ++v) h0[v] = start[v];
        } else {
          load_state<V>(g.first, s.batch(k), a.D, c, h0);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          uv[k][v] = fmaf(av[k][v], h0[v], uv[k][v]);
          A[v] = 0.f;
          U[v] = uv[k][v];
        }
      } else if (PLAIN || (s.in >> k & 1)) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          U[v] = fmaf(av[k][v], U[v], uv[k][v]);
          A[v] *= av[k][v];
        }
      }
    }
  }

  template <bool PLAIN, bool EVEN>
  __device__ inline void second_sweep(const RecurrenceArgs& a, const TileArgs& g, const Strip& s, int c, bool on,
                                      float (&h)[V]) const {
    RowWalk<E, EVEN> ph(a.h, a.sh, a, g, s.row);
    if (PLAIN && s.first) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = start[v];
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (PLAIN || (s.in >> k & 1)) {
        const bool first = !PLAIN && (s.first >> k & 1);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = first ? uv[k][v] : fmaf(av[k][v], h[v], uv[k][v]);
        if (PLAIN || on) store_values<E, V>(ph.p, c, h);
        if (a.hT && (PLAIN ? k == R - 1 && s.last : (s.last >> k & 1)) && (PLAIN || on))
          store_state<V>(a.hT, s.batch(k), a.D, c, h);
      }
      ph.next(s, k);
    }
  }
};

template <typename E, int V, int G, bool INP, int R, int W, bool FAR>
__global__ __launch_bounds__(W * WAVE, FAR ? WAVES_FAR : WAVES) void recurrence_tile_kernel(const RecurrenceArgs a,
                                                                                           const TileArgs g) {
  const TilePlace place = take_tile(g);
  if (place.turn < 0) return;
  const int tile = place.turn, slice = place.slice;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), lane = threadIdx.x & (WAVE - 1);
  int c = (slice * WAVE + lane) * V;
  const bool on = c < a.D;
  if (!on) c = 0;
  ForwardStrip<E, V, G, INP, R> strip;
#pragma unroll
  for (int v = 0; v < V; ++v) strip.lam[v] = G == GATE_POWER ? a.lam[c + v] : 0.f;   // (loads return in order)
  const Strip s = strip_of<R>(a, tile * (R * W) + wave * R);
  const bool plain = plain_strip<R>(s) && (slice + 1) * WAVE * V <= a.D;
  const bool even = s.n == R && (g.flat || !(s.first >> 1));
  float A[V], U[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.f;
    U[v] = 0.f;
  }
  if (plain)
    strip.template first_sweep<true, true>(a, g, s, c, A, U);
  else if (even)
    strip.template first_sweep<false, true>(a, g, s, c, A, U);
  else
    strip.template first_sweep<false, false>(a, g, s, c, A, U);
  // (the tile goes on from the one before it unless a sequence starts with it; the
  // first strip knows)
  bool open = false;
  if (wave == 0 && tile > 0) open = !(s.first & 1);
  enter_strip<V, W, FAR ? LOOK_FAR : LOOK>(g, tile, slice, 1, tile, open, wave, A, U, h);
  if (plain)
    strip.template second_sweep<true, true>(a, g, s, c, on, h);
  else if (even)
    strip.template second_sweep<false, true>(a, g, s, c, on, h);
  else
    strip.template second_sweep<false, false>(a, g, s, c, on, h);
}

// Rows from the last to the first.  before = h_{t-1} is the row of h before, or
// h0 at a sequence's first token.
template <typename E, int V, int G, bool INP, int R>
struct BackwardStrip {
  typedef typename VecIo<E, V>::raw raw;
  typedef VecIo<E, V> IO;
  raw rx[R], ri[R], rb[R], rg[R];
  GateValue gv[R][V];
  float lam[V], dlam[V], h0[V], end[V];   // of the last sequence that starts here, of the last that ends
  bool low;   // (power gates) whether 1 - a^2 of a value is below the normal numbers

  // Whether one of them is of a nearly shut gate: neither shut altogether, as gates of
  // padding may be, nor of a rate of 0.
  __device__ inline bool shut() const {
    if (!__any(low)) return false;
    bool any = false;
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) any = any || nearly_shut(lam[v], gate_rcp<E>(1.f + gv[k][v].k));
    return __any(any);
  }

  template <bool PLAIN, bool EVEN>
  __device__ inline void first_sweep(const RecurrenceArgs& a, const TileArgs& g, const Strip& s, int c, float (&A)[V],
                                     float (&U)[V]) {
    raw rf[R];
    const int l1 = s.last ? 31 - __builtin_clz(s.last) : 0, f1 = s.first ? 31 - __builtin_clz(s.first) : 0;
    if (s.last) load_state<V>(g.first, s.batch(l1), a.D, c, end);
    if (s.first) load_state<V>(a.h0, s.batch(f1), a.D, c, h0);
    const int row = s.row + max(s.n - 1, 0);
    RowWalk<E, EVEN> pf(a.f, a.sf, a, g, row), pg(a.dh, a.sdh, a, g, row);
#pragma unroll
    for (int k = R - 1; k >= 0; --k) {
      rf[k] = load_raw<E, V>(pf.p, c);
      rg[k] = load_raw<E, V>(pg.p, c);
      pf.back(s, k);
      pg.back(s, k);
    }
    RowWalk<E, EVEN> px(a.x, a.sx, a, g, row), pi(INP ? a.i : a.x, INP ? a.si : a.sx, a, g, row),
        pb(a.h, a.sh, a, g, row);
#pragma unroll
    for (int k = R - 1; k >= 0; --k) {
      rx[k] = load_raw<E, V>(px.p, c);
      if (INP) ri[k] = load_raw<E, V>(pi.p, c);
      // (a row that starts a sequence, or is of none, has no row before it)
      const bool inner = PLAIN ? k > 0 || !s.first : (s.in >> k & 1) && !(s.first >> k & 1);
      rb[k] = load_raw<E, V>(pb.p - (inner ? pb.step : 0), c);
      px.back(s, k);
      if (INP) pi.back(s, k);
      pb.back(s, k);
    }
    if (PLAIN && s.last) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] = 0.f;
        U[v] = end[v];
      }
    }
#pragma unroll
    for (int k = R - 1; k >= 0; --k) {
      float f[V];
      IO::unpack(rf[k], f);
#pragma unroll
      for (int v = 0; v < V; ++v) gv[k][v] = gate_value<E, G>(f[v], lam[v]);
      if (!PLAIN && (s.last >> k & 1)) {
        if (k == l1) {
#pragma unroll
          for (int v = 0; v < V; ++v) U[v] = end[v];
        } else {
          load_state<V>(g.first, s.batch(k), a.D, c, U);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 0.f;
      }
      if (PLAIN || (s.in >> k & 1)) {
        float d[V];
        IO::unpack(rg[k], d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          U[v] = gv[k][v].a * (d[v] + U[v]);
          A[v] *= gv[k][v].a;
        }
      }
    }
  }

  // SHUT: once more, for the values of nearly shut gates alone (apart from the
  // sweep that all take, which keeps its registers, its time and its other results).
  template <bool PLAIN, bool EVEN, bool SHUT>
  __device__ inline void second_sweep(const RecurrenceArgs& a, const TileArgs& g, const Strip& s, int c, bool on,
                                      float (&carry)[V]) {
    const int row = s.row + max(s.n - 1, 0);
    RowWalk<E, EVEN> px(a.dx, a.sdx, a, g, row), pf(a.df, a.sdf, a, g, row),
        pi(INP ? a.di : a.dx, INP ? a.sdi : a.sdx, a, g, row);
    const int l1 = s.last ? 31 - __builtin_clz(s.last) : 0, f1 = s.first ? 31 - __builtin_clz(s.first) : 0;
    if (PLAIN && s.last) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = end[v];
    }
#pragma unroll
    for (int k = R - 1; k >= 0; --k) {
      if (!PLAIN && (s.last >> k & 1)) {
        if (k == l1) {
#pragma unroll
          for (int v = 0; v < V; ++v) carry[v] = end[v];
        } else {
          load_state<V>(g.first, s.batch(k), a.D, c, carry);
        }
      }
      if (PLAIN || (s.in >> k & 1)) {
        float x[V], i[V], b[V], d[V], dx[V], df[V], di[V];
        IO::unpack(rx[k], x);
        if (INP) IO::unpack(ri[k], i);
        IO::unpack(rb[k], b);
        IO::unpack(rg[k], d);
        const bool first = PLAIN ? k == 0 && s.first : (s.first >> k & 1);
        if (first) {
          if (PLAIN || k == f1) {
#pragma unroll
            for (int v = 0; v < V; ++v) b[v] = h0[v];
          } else {
            load_state<V>(a.h0, s.batch(k), a.D, c, b);
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float gt = d[v] + carry[v];
          carry[v] = gv[k][v].a * gt;
          float dl;
          if constexpr (SHUT) {
            if (on && shut_gradients<E, INP>(gv[k][v], x[v], INP ? i[v] : 0.f, lam[v], b[v], gt, carry[v], dx[v], df[v],
                                             di[v], dl)) {
              dlam[v] += dl;
              const_cast<E*>(px.p)[c + v] = (E)dx[v];
              const_cast<E*>(pf.p)[c + v] = (E)df[v];
              if (INP) const_cast<E*>(pi.p)[c + v] = (E)di[v];
            }
            continue;
          }
          gate_gradients<E, G, INP>(gv[k][v], x[v], INP ? i[v] : 0.f, lam[v], b[v], gt, carry[v], dx[v], df[v], di[v], dl,
                                    low);
          if (G == GATE_POWER) dlam[v] += dl;
        }
        if (!SHUT && (PLAIN || on)) {
          store_values<E, V>(px.p, c, dx);
          store_values<E, V>(pf.p, c, df);
          if (INP) store_values<E, V>(pi.p, c, di);
          if (first && a.dh0) store_state<V>(a.dh0, s.batch(k), a.D, c, carry);
        }
      }
      px.back(s, k);
      pf.back(s, k);
      if (INP) pi.back(s, k);
    }
  }
};

template <typename E, int V, int G, bool INP, int R, int W, bool FAR>
__global__ __launch_bounds__(W * WAVE, FAR ? WAVES_FAR : WAVES) void recurrence_tile_bwd_kernel(
    const RecurrenceArgs a, const TileArgs g) {
  const TilePlace place = take_tile(g);
  if (place.turn < 0) return;
  const int turn = place.turn, slice = place.slice, tile = g.tiles - 1 - turn;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), lane = threadIdx.x & (WAVE - 1);
  int c = (slice * WAVE + lane) * V;
  const bool on = c < a.D;
  if (!on) c = 0;
  BackwardStrip<E, V, G, INP, R> strip;
  strip.low = false;
#pragma unroll
  for (int v = 0; v < V; ++v) strip.lam[v] = G == GATE_POWER ? a.lam[c + v] : 0.f;   // (loads return in order)
  const Strip s = strip_of<R>(a, tile * (R * W) + wave * R);
  const bool plain = plain_strip<R>(s) && (slice + 1) * WAVE * V <= a.D;
  const bool even = s.n == R && (g.flat || !(s.first >> 1));
  float A[V], U[V], carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.f;
    U[v] = strip.dlam[v] = 0.f;
  }
  if (plain)
    strip.template first_sweep<true, true>(a, g, s, c, A, U);
  else if (even)
    strip.template first_sweep<false, true>(a, g, s, c, A, U);
  else
    strip.template first_sweep<false, false>(a, g, s, c, A, U);
  // (the tile goes on from the one behind it unless a sequence ends with it; only
  // the last tile of a batch, the first in turn, is not full)
  bool open = false;
  if (wave == W - 1 && turn > 0) open = !(s.last >> (R - 1) & 1);
  enter_strip<V, W, FAR ? LOOK_FAR : LOOK>(g, tile, slice, -1, turn, open, W - 1 - wave, A, U, carry);
  float again[V];
#pragma unroll
  for (int v = 0; v < V; ++v) again[v] = carry[v];
  if (plain)
    strip.template second_sweep<true, true, false>(a, g, s, c, on, carry);
  else if (even)
    strip.template second_sweep<false, true, false>(a, g, s, c, on, carry);
  else
    strip.template second_sweep<false, false, false>(a, g, s, c, on, carry);
  if constexpr (G == GATE_POWER)
    if (strip.shut()) strip.template second_sweep<false, false, true>(a, g, s, c, on, again);
  if constexpr (G == GATE_POWER) {   // the tile's part of dlam, wave after wave
    __shared__ float sm[W][V][WAVE];
#pragma unroll
    for (int v = 0; v < V; ++v) sm[wave][v][lane] = strip.dlam[v];
    __syncthreads();
    if (wave == 0 && on) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) sum += sm[k][v][lane];
        a.part[(long)tile * a.D + c + v] = sum;
      }
    }
  }
}

// (16384 tokens of 256 channels 35 us without looking far, 22 with, backward 66 and
// 38; of 2048 channels 71 without, 88 with; 64 sequences of up to 200 tokens,
// backward, 408 tiles, 19 without, 22 with.  A packed batch goes by the average of its
// sequences, since the host does not read the offsets: one long sequence among many
// short ones looks near.)
template <typename E, int V, int G, bool INP, bool FAR>
hipError_t launch_tiles(const RecurrenceArgs& a, const TileArgs& g, bool bwd, hipStream_t s) {
  const dim3 grid((unsigned)g.tiles * g.slices);
  if (bwd)
    hipLaunchKernelGGL((recurrence_tile_bwd_kernel<E, V, G, INP, REC_BWD_R, REC_BWD_W, FAR>), grid,
                       dim3(REC_BWD_W * WAVE), 0, s, a, g);
  else
    hipLaunchKernelGGL((recurrence_tile_kernel<E, V, G, INP, REC_R, REC_W, FAR>), grid, dim3(REC_W * WAVE), 0, s, a, g);
  return hipGetLastError();
}
template <typename E, int V, int G, bool INP>
hipError_t launch_tiles(const RecurrenceArgs& a, const TileArgs& g, bool bwd, hipStream_t s) {
  const int rows = bwd ? REC_BWD_R * REC_BWD_W : REC_R * REC_W, chain = a.cu ? g.tiles / a.B : a.T / rows;
  return g.words && (long)g.tiles * g.slices <= FAR_TILES && chain >= FAR_CHAIN
             ? launch_tiles<E, V, G, INP, true>(a, g, bwd, s)
             : launch_tiles<E, V, G, INP, false>(a, g, bwd, s);
}
template <typename E, int V, int G>
hipError_t launch_tiles(const RecurrenceArgs& a, const TileArgs& g, bool bwd, hipStream_t s) {
  return a.i ? launch_tiles<E, V, G, true>(a, g, bwd, s) : launch_tiles<E, V, G, false>(a, g, bwd, s);
}
// (a storage type and width in a source file each)
template <typename E, int V>
hipError_t recurrence_tiles(const RecurrenceArgs& a, const TileArgs& g, bool bwd, hipStream_t s);

#define PRISM_RECURRENCE_TILES(E, V)                                                                           \
  template <>                                                                                                  \
  hipError_t recurrence_tiles<E, V>(const RecurrenceArgs& a, const TileArgs& g, bool bwd, hipStream_t s) {     \
    if (a.gate == GATE_LOG) return launch_tiles<E, V, GATE_LOG>(a, g, bwd, s);                                 \
    if (a.gate == GATE_SIGMOID) return launch_tiles<E, V, GATE_SIGMOID>(a, g, bwd, s);                         \
    return launch_tiles<E, V, GATE_POWER>(a, g, bwd, s);                                                       \
  }

}  // namespace prism
