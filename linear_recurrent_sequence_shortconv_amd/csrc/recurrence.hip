// Gated recurrence h_t = a_t h_{t-1} + u_t, channel by channel, and its
// backward pass: with g_t the gradient of h_t from its own row and the tokens
// behind it,
//   g_t = dh_t + a_{t+1} g_{t+1},  d(a_t) = g_t h_{t-1},  d(u_t) = g_t,
// dhT added at the last token, dh0 = a_1 g_1.  h_{t-1} is read from the forward
// pass's output.
//
// Dispatch: whole sequences and the backward pass go through tiles
// (recurrence_tile.h) after a small kernel that readies their words; sequences of
// a few tokens, the single-token step among them, token by token.
#include "recurrence_tile.h"

namespace prism {

namespace {

template <typename E, int V>
__device__ inline void load_v(const void* p, long at, float (&x)[V]) {
  typedef typename VecIo<E, V>::raw raw;
  VecIo<E, V>::unpack(*reinterpret_cast<const raw*>(static_cast<const E*>(p) + at), x);
}
template <typename E, int V>
__device__ inline void store_v(void* p, long at, const float (&x)[V]) {
  typedef typename VecIo<E, V>::raw raw;
  *reinterpret_cast<raw*>(static_cast<E*>(p) + at) = VecIo<E, V>::pack(x);
}

// A lane takes V channels of one dense sequence and walks its tokens.  Memory bound
// where there are many (2048 sequences of 8 tokens of 2048 channels 59 us, 5.1 TB/s),
// else a chain of loads and products (64 sequences of one token of 4096 channels 3 us).
template <typename E, int V, int G, bool INP>
__global__ __launch_bounds__(256) void recurrence_walk_kernel(const RecurrenceArgs a, int cb) {
  const int b = blockIdx.x / cb, c = ((blockIdx.x % cb) * 256 + threadIdx.x) * V;
  if (c >= a.D) return;
  float h[V], lam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = a.h0 ? a.h0[(long)b * a.D + c + v] : 0.f;
    lam[v] = G == GATE_POWER ? a.lam[c + v] : 0.f;
  }
  auto at = [&](const TokenSteps& s, int t) { return b * s.b + t * s.t + c; };
  for (int t = 0; t < a.T; ++t) {
    float x[V], f[V], i[V];
    load_v<E, V>(a.x, at(a.sx, t), x);
    load_v<E, V>(a.f, at(a.sf, t), f);
    if (INP) load_v<E, V>(a.i, at(a.si, t), i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float av, u;
      gate_inputs<E, G, INP>(x[v], f[v], INP ? i[v] : 0.f, lam[v], av, u);
      h[v] = fmaf(av, h[v], u);
    }
    store_v<E, V>(a.h, at(a.sh, t), h);
  }
  if (a.hT) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.hT[(long)b * a.D + c + v] = h[v];
  }
}

// Readies a pass: no word written yet, no tile taken; a copy of the states to
// start from where the last states replace them (a tile whose own decays are 0
// would not wait for the tile that still reads them); the last states of
// sequences without tokens.  (A launch of its own, 3 to 5 us, since no tile may look
// at a word before it is ready.)
__global__ __launch_bounds__(256) void recurrence_ready_kernel(uint4* words, long n, unsigned* counter, float* copy,
                                                               const float* first, long ncopy, const int* cu, int B,
                                                               int T, int rows, int D, float* last) {
  const long at = (long)blockIdx.x * 256 + threadIdx.x, all = (long)gridDim.x * 256;
  if (counter && at == 0) *counter = 0;
  for (long e = at; e < n; e += all) words[e] = make_uint4(NOT_YET, NOT_YET, NOT_YET, NOT_YET);
  for (long e = at; e < ncopy; e += all) copy[e] = first[e];
  if (!last) return;
  __shared__ int sm[4];
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (empty_sequence(cu, T, rows, b, sm))
      for (int c = threadIdx.x; c < D; c += 256) last[(long)b * D + c] = first ? first[(long)b * D + c] : 0.f;
}

template <typename E, int V, int G, bool INP>
hipError_t run_walk(const RecurrenceArgs& a, hipStream_t s) {
  const int cb = (a.D + 256 * V - 1) / (256 * V);
  hipLaunchKernelGGL((recurrence_walk_kernel<E, V, G, INP>), dim3((unsigned)cb * a.B), dim3(256), 0, s, a, cb);
  return hipGetLastError();
}
template <typename E, int V, int G>
hipError_t run_walk(const RecurrenceArgs& a, hipStream_t s) {
  return a.i ? run_walk<E, V, G, true>(a, s) : run_walk<E, V, G, false>(a, s);
}
template <typename E, int V>
hipError_t run_walk(const RecurrenceArgs& a, hipStream_t s) {
  if (a.gate == GATE_LOG) return run_walk<E, V, GATE_LOG>(a, s);
  if (a.gate == GATE_SIGMOID) return run_walk<E, V, GATE_SIGMOID>(a, s);
  return run_walk<E, V, GATE_POWER>(a, s);
}

// Workspace of a pass by tiles.  Words only where a tile goes on from another; the
// counter's place is kept in any case, so that no pass writes anything else there.
struct Plan {
  int tiles;
  bool words;
  size_t first_at, words_at, part_at, bytes;
};
Plan plan_of(int B, int T, int D, int rows, bool packed, bool bwd, bool part) {
  Plan p;
  const int tile = bwd ? REC_BWD_R * REC_BWD_W : REC_R * REC_W;
  p.tiles = (rows + tile - 1) / tile;
  p.words = p.tiles > 1 && (packed || tile % T != 0);
  const size_t wide = ((size_t)D + 127) / 128 * 128;   // (a slice has 64 or 128 channels)
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  p.first_at = p.words || part ? 256 : 0;
  p.words_at = p.first_at + (p.words ? up((size_t)B * D * 4) : 0);
  p.part_at = p.words_at + (p.words ? up(wide * p.tiles * 8) : 0);
  p.bytes = p.part_at + (part ? up((size_t)p.tiles * D * 4) : 0);
  return p;
}

template <typename E, int V>
hipError_t run_tiles(RecurrenceArgs a, bool bwd, char* ws, hipStream_t s) {
  const bool part = bwd && a.gate == GATE_POWER;
  const Plan p = plan_of(a.B, a.T, a.D, a.rows, a.cu != nullptr, bwd, part);
  const int parts = a.B > 0 ? p.tiles : 0;
  float* last = bwd ? a.dh0 : a.hT;
  TileArgs g = {};
  g.tiles = p.tiles;
  g.slices = (a.D + WAVE * V - 1) / (WAVE * V);
  g.first = bwd ? a.dhT : a.h0;
  auto flat = [&](const TokenSteps& t) { return t.b == a.T * t.t; };
  g.flat = a.cu || a.B == 1 ||
           (flat(a.sx) && flat(a.sf) && (!a.i || flat(a.si)) && flat(a.sh) &&
            (!bwd || (flat(a.sdh) && flat(a.sdx) && flat(a.sdf) && (!a.i || flat(a.sdi)))));
  a.part = part ? reinterpret_cast<float*>(ws + p.part_at) : nullptr;
  if (parts > 0 && p.words) {
    g.counter = reinterpret_cast<unsigned*>(ws);
    g.words = reinterpret_cast<unsigned long long*>(ws + p.words_at);
  }
  const bool copy = g.words && last && last == g.first, empty = last && last != g.first && (a.cu || a.T == 0);
  if (a.B > 0 && (g.words || empty)) {
    const long n = g.words ? (long)g.slices * WAVE * V * p.tiles / 2 : 0;
    long blocks = n / 256 + 1;
    if (empty && a.B > blocks) blocks = a.B;
    if (blocks > 1024) blocks = 1024;
    hipLaunchKernelGGL(recurrence_ready_kernel, dim3((unsigned)blocks), dim3(256), 0, s,
                       reinterpret_cast<uint4*>(g.words), n, g.counter,
                       copy ? reinterpret_cast<float*>(ws + p.first_at) : nullptr, g.first, copy ? (long)a.B * a.D : 0L,
                       a.cu, a.B, a.T, a.rows, a.D, empty ? last : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (copy) g.first = reinterpret_cast<float*>(ws + p.first_at);
  }
  if (parts > 0) {
    const hipError_t e = recurrence_tiles<E, V>(a, g, bwd, s);
    if (e != hipSuccess) return e;
  }
  if (part) return launch_column_sums(a.part, parts, a.D, 0, nullptr, a.dlam, s);
  return hipSuccess;
}

// bf16 channels two a lane where every row starts at a multiple of 4 bytes (one
// sequence of 16384 tokens of 2048 channels 68 us with two, 77 with one; backward of
// 8 x 2048 tokens 129 and 144).
bool pairs(const RecurrenceArgs& a, bool bwd) {
  long m = a.D | a.sx.b | a.sx.t | a.sf.b | a.sf.t | a.sh.b | a.sh.t;
  uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.f | (uintptr_t)a.i | (uintptr_t)a.h;
  if (a.i) m |= a.si.b | a.si.t;
  if (bwd) {
    m |= a.sdh.b | a.sdh.t | a.sdx.b | a.sdx.t | a.sdf.b | a.sdf.t;
    p |= (uintptr_t)a.dh | (uintptr_t)a.dx | (uintptr_t)a.df | (uintptr_t)a.di;
    if (a.i) m |= a.sdi.b | a.sdi.t;
  }
  return m % 2 == 0 && p % 4 == 0;
}

// Dense sequences of so few tokens are walked: no words to ready, and no strip
// that sequences divide (2048 sequences of 8 tokens of 2048 channels 59 us in place of
// 70, 4 of 8 tokens of 512 4.4 in place of 9.8; of 16 tokens, 64 sequences take 10 us
// walked and 8.8 by tiles).
constexpr int WALK = 8;
bool walked(const RecurrenceArgs& a, bool bwd) { return !bwd && !a.cu && a.T > 0 && a.T <= WALK && a.B > 0; }

template <typename E, int V>
hipError_t run(const RecurrenceArgs& a, bool bwd, void* ws, hipStream_t s) {
  if (walked(a, bwd)) return run_walk<E, V>(a, s);
  return run_tiles<E, V>(a, bwd, static_cast<char*>(ws), s);
}

}  // namespace

size_t recurrence_bytes(const RecurrenceArgs& a, bool packed, bool bwd) {
  if (a.rows == 0 || a.B == 0 || (!packed && !bwd && a.T <= WALK)) return 0;
  return plan_of(a.B, a.T, a.D, a.rows, packed, bwd, bwd && a.gate == GATE_POWER).bytes;
}

hipError_t launch_recurrence_step(const RecurrenceArgs& a, bool f32, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  if (f32) return run_walk<float, 1>(a, s);
  return pairs(a, false) ? run_walk<bf16, 2>(a, s) : run_walk<bf16, 1>(a, s);
}

hipError_t launch_recurrence(const RecurrenceArgs& a, bool f32, bool bwd, void* ws, hipStream_t s) {
  if (f32) return run<float, 1>(a, bwd, ws, s);
  return pairs(a, bwd) ? run<bf16, 2>(a, bwd, ws, s) : run<bf16, 1>(a, bwd, ws, s);
}

}  // namespace prism
