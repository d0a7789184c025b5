// C ABI of the query / key normalisation and of the linear attention: checks,
// workspace carving and launch sequences.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "api_common.h"
#include "operators.h"

namespace {

using prism::Carve;
using prism::check_buffer;
using prism::fail;
using prism::Strides;

Strides strides(const prism_strides& s) { return Strides{(long)s.batch, (long)s.token, (long)s.head}; }

std::string num(long long x) { return std::to_string(x); }

// ---------------------------------------------------------------- qk_norm
prism_status check_qk_strides(const prism_strides& s, const char* name, int unit) {
  const long long v[3] = {s.batch, s.token, s.head};
  for (long long x : v) {
    if (x % unit != 0)
      return fail(PRISM_ERR_ALIGN, std::string("strides of ") + name + " must be multiples of " + num(unit) + " elements");
    if (x >= (1LL << 40) || x <= -(1LL << 40)) return fail(PRISM_ERR_SHAPE, std::string("strides of ") + name + " out of range");
  }
  return PRISM_OK;
}

prism_status check_qk(const prism_qk_norm_desc* desc, bool bwd) {
  if (!desc) return fail(PRISM_ERR_NULL, "desc is NULL");
  const prism_qk_norm_desc& d = *desc;
  if (d.B < 0 || d.T < 0 || d.Hq < 1 || d.Hk < 0)
    return fail(PRISM_ERR_SHAPE, "B, T and Hk must be >= 0 and Hq >= 1 (got B=" + num(d.B) + " T=" + num(d.T) + " Hq=" +
                                     num(d.Hq) + " Hk=" + num(d.Hk) + ")");
  if (d.Hq > (1 << 20) || d.Hk > (1 << 20)) return fail(PRISM_ERR_SHAPE, "Hq and Hk must be <= 1048576");
  if (d.d < 1 || d.rot < 0 || d.rot > d.d) return fail(PRISM_ERR_SHAPE, "d must be >= 1 and 0 <= rot <= d");
  if (d.dtype != PRISM_F32 && d.dtype != PRISM_BF16)
    return fail(PRISM_ERR_UNSUPPORTED, "dtype must be PRISM_F32 or PRISM_BF16");
  if (d.d % 8 || d.d > 256) return fail(PRISM_ERR_UNSUPPORTED, "d must be a multiple of 8 up to 256 (got " + num(d.d) + ")");
  if (d.rot % 8) return fail(PRISM_ERR_UNSUPPORTED, "rot must be a multiple of 8 (got " + num(d.rot) + ")");
  if (d.norm != PRISM_NORM_L2 && d.norm != PRISM_NORM_RMS)
    return fail(PRISM_ERR_UNSUPPORTED, "norm must be PRISM_NORM_L2 or PRISM_NORM_RMS");
  if (!(d.eps >= 0.f) || !std::isfinite(d.eps)) return fail(PRISM_ERR_SHAPE, "eps must be finite and >= 0");
  const struct {
    const prism_strides& s;
    const char* name;
    bool use;
  } all[] = {{d.q, "q", true},        {d.k, "k", d.Hk > 0},         {d.qo, "qo", true},
             {d.ko, "ko", d.Hk > 0}, {d.dq, "dq", bwd},            {d.dk, "dk", bwd && d.Hk > 0}};
  for (const auto& x : all)
    if (x.use) {
      const prism_status st = check_qk_strides(x.s, x.name, 4);
      if (st != PRISM_OK) return st;
    }
  return PRISM_OK;
}

prism::QkNormArgs qk_args(const prism_qk_norm_desc& d, const void* q, const void* k, const void* wq, const void* wk,
                          const int* positions, const long long* turns) {
  prism::QkNormArgs a = {};
  a.B = d.B;
  a.T = d.T;
  a.Hq = d.Hq;
  a.Hk = d.Hk;
  a.d = d.d;
  a.rot = d.rot;
  a.c = d.norm == PRISM_NORM_RMS ? 1.f / (float)d.d : 1.f;
  a.eps = d.eps;
  a.interleaved = d.interleaved != 0;
  a.xq = q;
  a.xk = d.Hk > 0 ? k : nullptr;
  a.wq = wq;
  a.wk = d.Hk > 0 ? wk : nullptr;
  a.pos = positions;
  a.turns = turns;
  a.sxq = strides(d.q);
  a.sxk = strides(d.k);
  return a;
}

prism_status check_rotation(const prism_qk_norm_desc& d, const int* positions, const long long* turns) {
  if (d.rot == 0) return PRISM_OK;
  if (!positions) return fail(PRISM_ERR_NULL, "positions is NULL");
  if (!turns) return fail(PRISM_ERR_NULL, "turns is NULL");
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return fail(PRISM_ERR_ALIGN, "positions is not 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(turns) & 7u) return fail(PRISM_ERR_ALIGN, "turns is not 8-byte aligned");
  return PRISM_OK;
}

prism_status qk_forward(const prism_qk_norm_desc* desc, const void* q, const void* k, const void* wq, const void* wk,
                        const int* positions, const long long* turns, void* qo, void* ko, hipStream_t stream) {
  prism_status st = check_qk(desc, false);
  if (st != PRISM_OK) return st;
  if ((long long)desc->B * desc->T == 0) return PRISM_OK;
  const bool keys = desc->Hk > 0;
  CHECK_PTR(q, true);
  CHECK_PTR(k, keys);
  CHECK_PTR(wq, false);
  CHECK_PTR(wk, false);
  CHECK_PTR(qo, true);
  CHECK_PTR(ko, keys);
  st = check_rotation(*desc, positions, turns);
  if (st != PRISM_OK) return st;
  prism::QkNormArgs a = qk_args(*desc, q, k, wq, wk, positions, turns);
  a.yq = qo;
  a.yk = ko;
  a.syq = strides(desc->qo);
  a.syk = strides(desc->ko);
  HIP_TRY("qk_norm", stream, desc->dtype == PRISM_BF16 ? prism::launch_qk_norm<prism::bf16>(a, stream)
                                                       : prism::launch_qk_norm<float>(a, stream));
  return PRISM_OK;
}

prism_status qk_backward(const prism_qk_norm_desc* desc, const void* q, const void* k, const void* wq, const void* wk,
                         const int* positions, const long long* turns, const void* dqo, const void* dko, void* dq,
                         void* dk, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  prism_status st = check_qk(desc, true);
  if (st != PRISM_OK) return st;
  const bool some = (long long)desc->B * desc->T > 0, keys = desc->Hk > 0;
  CHECK_PTR(q, some);
  CHECK_PTR(k, some && keys);
  CHECK_PTR(wq, false);
  CHECK_PTR(wk, false);
  CHECK_PTR(dqo, some);
  CHECK_PTR(dko, some && keys);
  CHECK_PTR(dq, some);
  CHECK_PTR(dk, some && keys);
  CHECK_PTR(dwq, wq != nullptr);
  CHECK_PTR(dwk, keys && wk != nullptr);
  if (some) {
    st = check_rotation(*desc, positions, turns);
    if (st != PRISM_OK) return st;
  }
  prism::QkNormArgs a = qk_args(*desc, q, k, wq, wk, positions, turns);
  a.gq = dqo;
  a.gk = dko;
  a.sgq = strides(desc->qo);
  a.sgk = strides(desc->ko);
  a.yq = dq;
  a.yk = dk;
  a.syq = strides(desc->dq);
  a.syk = strides(desc->dk);
  a.dwq = a.wq ? dwq : nullptr;
  a.dwk = a.wk ? dwk : nullptr;
  if (a.dwq || a.dwk) {
    st = check_buffer(workspace, workspace_bytes, prism::qk_norm_part_bytes(desc->d), "workspace");
    if (st != PRISM_OK) return st;
    a.part = static_cast<float*>(workspace);
  }
  HIP_TRY("qk_norm_bwd", stream, desc->dtype == PRISM_BF16 ? prism::launch_qk_norm_bwd<prism::bf16>(a, stream)
                                                           : prism::launch_qk_norm_bwd<float>(a, stream));
  return PRISM_OK;
}

// ------------------------------------------------------- linear attention
struct LaPlan {
  int dim, grp, nseg, seglen;
  bool f32;
  bool one;        // dv in the launch of dq and dk that also gives the row dots
  long rows;       // token rows of the tensors
  size_t bh, DD;
};

prism_status check_la(const prism_linear_attention_desc* desc, bool packed, LaPlan* out) {
  if (!desc) return fail(PRISM_ERR_NULL, "desc is NULL");
  const prism_linear_attention_desc& d = *desc;
  if (d.B < 0 || d.T < 0 || d.H < 1 || d.Hk < 1)
    return fail(PRISM_ERR_SHAPE, "B and T must be >= 0, H and Hk >= 1 (got B=" + num(d.B) + " T=" + num(d.T) + " H=" +
                                     num(d.H) + " Hk=" + num(d.Hk) + ")");
  if (d.H % d.Hk) return fail(PRISM_ERR_SHAPE, "H must be a multiple of Hk (got " + num(d.H) + ", " + num(d.Hk) + ")");
  if (d.dtype != PRISM_F32 && d.dtype != PRISM_BF16)
    return fail(PRISM_ERR_UNSUPPORTED, "dtype must be PRISM_F32 or PRISM_BF16");
  const int dims[2] = {d.dk, d.dv};
  for (int x : dims)
    if (x < 16 || x > 128 || x % 16)
      return fail(PRISM_ERR_UNSUPPORTED, "dk and dv must be multiples of 16 from 16 to 128 (got " + num(d.dk) + ", " +
                                             num(d.dv) + ")");
  if (!std::isfinite(d.scale)) return fail(PRISM_ERR_SHAPE, "scale must be finite");
  // (32-bit token arithmetic with room for a segment; 32-bit offsets in a chunk
  // of the contiguous gradients)
  if (d.T > (1 << 30)) return fail(PRISM_ERR_SHAPE, "T must be <= 1073741824 (got " + num(d.T) + ")");
  if ((long long)d.H * (d.dk > d.dv ? d.dk : d.dv) > (1LL << 22))
    return fail(PRISM_ERR_SHAPE, "H * dk and H * dv must be <= 4194304");
  if (packed && d.packed_tokens < 0) return fail(PRISM_ERR_SHAPE, "packed_tokens must be >= 0 with cu_seqlens");
  const int unit = d.dtype == PRISM_F32 ? 4 : 8;
  const struct {
    const prism_strides& s;
    const char* name;
    int unit;
  } all[] = {{d.q, "q", unit}, {d.k, "k", unit}, {d.v, "v", unit}, {d.o, "o", unit}, {d.g, "g", 1}};
  for (const auto& x : all) {
    const long long v[3] = {x.s.batch, x.s.token, x.s.head};
    for (long long y : v) {
      if (y < 0 || y >= (1LL << 40)) return fail(PRISM_ERR_SHAPE, std::string("strides of ") + x.name + " out of range");
      if (y % x.unit) return fail(PRISM_ERR_ALIGN, std::string("strides of ") + x.name + " must be multiples of 16 bytes");
    }
    if (x.s.token > (1LL << 22))
      return fail(PRISM_ERR_SHAPE, std::string("the token stride of ") + x.name + " must be <= 4194304 elements");
  }
  LaPlan p;
  p.dim = d.dk > d.dv ? d.dk : d.dv;
  p.f32 = d.dtype == PRISM_F32;
  p.grp = d.H / d.Hk;
  p.rows = packed ? d.packed_tokens : (long)d.B * d.T;
  p.bh = (size_t)d.B * d.H;
  p.DD = (size_t)d.dk * d.dv;
  p.nseg = 1;
  p.seglen = 0;
  p.one = false;
  // (a launch has at most 8 workgroups of 256 threads for each head: under 2^32 threads)
  if ((double)p.bh * p.DD * 4 > 1.0e12 || (double)p.rows * d.H * p.dim > 4.0e12 || p.bh >= (size_t(1) << 21))
    return fail(PRISM_ERR_SHAPE, "problem too large");
  *out = p;
  return PRISM_OK;
}

// Up to this many segments a workgroup forms its entering state from the own
// states of the segments before it; more are joined by a kernel of its own.
// 8 x 2048 tokens, 16 heads, forward: by itself 129, 121 and 151 us with 2, 4
// and 6 segments, joined 136, 124 and 144.  The decays' gradient uses each of these
// states in three launches: the same tokens, by itself 358, 446 and 406 us with 2,
// 3 and 4, joined 367, 422 and 392; 2 x 333 tokens, 3 heads in fp32 71, 58 and
// 52, joined 71, 55 and 47 (dv in a launch of its own throughout).
constexpr int LA_SELF_JOIN = 4, LA_SELF_JOIN_DG = 2;

// Segments a sequence is cut into.  A launch runs B H workgroups for each of
// its passes and each segment, 512 of them at once (two a CU); more than one
// segment also needs the states at their starts, from a further pass (backward:
// two) of half the work over all but one segment.  Taken is the count with the
// least cost in the time of one chunk on a full chip (4 us in bf16 at d = 128),
// as measured there: a workgroup costs 2.5 chunks beside its own (4 where it
// forms states alone, with their join: 8 x 512 tokens, 16 heads 44 us in one
// segment, 56 in the four that 2 would give), a round of at most one workgroup a
// CU goes by 0.6 of the time for each chunk, fp32 takes twice and the decays'
// gradient 1.6 times as long.  The join's launch is priced from 5 segments on,
// with the decays' gradient too, whose join of 3 or 4 takes the place of work in
// three launches: priced from 3 on, a backward pass with dg, 16 heads of 128,
// takes 109 in place of 87 us for 3 x 700 tokens, 48 in place of 45 for 1 x 256
// (one segment chosen) and 82 in place of 88 for 2 x 1024 (5 in place of 4).
// 8 x 2048 tokens, 16 heads, forward, with 1, 2, 3, 4, 5 and 8 segments: 146, 130,
// 127, 122, 133 and 151 us (4 taken); one sequence of 16384 tokens with 1, 4, 8,
// 16 and 32: 1089, 441, 228, 131 and 114 (32 taken); a backward pass of 2 x 4096
// tokens, 16 heads on 4, with 1, 2, 4, 5 and 8: 305, 253, 183, 170 and 169 (5
// taken).
constexpr int LA_AT_ONCE = 512;   // workgroups
enum LaWork { LA_FORWARD, LA_BACKWARD, LA_BACKWARD_DG };
void plan_segments(const prism_linear_attention_desc& d, LaWork work, LaPlan* p) {
  const long chunks = ((long)d.T + prism::LA_CHUNK - 1) / prism::LA_CHUNK;
  const long most = chunks / 2 < 64 ? chunks / 2 : 64;
  const double bh = (double)p->bh, unit = p->f32 ? 2.0 : 1.0;
  auto rounds = [&](double groups, double each, double fixed) {
    const double full = std::floor(groups / LA_AT_ONCE), rest = groups - LA_AT_ONCE * full;
    each *= unit;
    return full * (each + fixed) + (rest == 0 ? 0.0 : rest <= 256 ? 0.6 * each + fixed : each + fixed);
  };
  long best = 1;
  double least = 0.0;
  for (long n = 1; n <= (most > 1 ? most : 1); ++n) {
    const double per = chunks > 0 ? (double)((chunks + n - 1) / n) : 1.0;
    double cost = work == LA_FORWARD    ? rounds(bh * n, per, 2.5)
                  : work == LA_BACKWARD ? rounds(bh * 3 * n, per, 2.5)
                  : bh * 3 * n <= LA_AT_ONCE ? rounds(bh * 3 * n, 1.6 * per, 2.5)
                                             : rounds(bh * 2 * n, 1.6 * per, 2.5) + rounds(bh * n, per, 2.5);
    if (n > 1) cost += rounds(bh * (work == LA_FORWARD ? 1 : 2) * (n - 1), 0.5 * per, 4.0);
    if (n > LA_SELF_JOIN) cost += 2.0;
    if (n == 1 || cost < least) {
      best = n;
      least = cost;
    }
  }
  const long per = chunks > 0 ? (chunks + best - 1) / best : 1;
  p->seglen = (int)(per * prism::LA_CHUNK);
  p->nseg = (int)(chunks > 0 ? (chunks + per - 1) / per : 1);
  // (dv takes 1.3 times as long in the kernel with the row dots as in its own, but
  // where all workgroups run at once it costs no launch after the other two:
  // 8 x 128 tokens, 16 heads, 384 workgroups, 32 us in place of 39, 2 x 333 in fp32,
  // 72, 33 in place of 48; 2 x 4096 tokens, 16 heads, 227 in place of 196)
  p->one = p->bh * p->nseg * 3 <= (size_t)LA_AT_ONCE;
}

void plan_forward(const prism_linear_attention_desc& d, LaPlan* p) { plan_segments(d, LA_FORWARD, p); }
void plan_backward(const prism_linear_attention_desc& d, bool dg, LaPlan* p) {
  plan_segments(d, dg ? LA_BACKWARD_DG : LA_BACKWARD, p);
}

struct LaFwdWs {
  float *seg, *dec;
};
LaFwdWs carve_la_fwd(const prism_linear_attention_desc& d, const LaPlan& p, Carve& cv) {
  LaFwdWs w = {};
  if (p.nseg > 1) {
    w.seg = cv.take<float>(p.bh * p.nseg * p.DD * 4);
    w.dec = cv.take<float>(p.bh * p.nseg * 4);
  }
  return w;
}

struct LaBwdWs {
  float *segf, *segr, *decf, *decr;
  float *dkp, *dvp;              // per query head (shared keys and values)
  float *eq, *ek, *ST, *tmp;     // decay gradient
};
LaBwdWs carve_la_bwd(const prism_linear_attention_desc& d, const LaPlan& p, bool dg, Carve& cv) {
  LaBwdWs w = {};
  if (p.nseg > 1) {
    w.segf = cv.take<float>(p.bh * p.nseg * p.DD * 4);
    w.segr = cv.take<float>(p.bh * p.nseg * p.DD * 4);
    w.decf = cv.take<float>(p.bh * p.nseg * 4);
    w.decr = cv.take<float>(p.bh * p.nseg * 4);
  }
  if (p.grp > 1) {
    w.dkp = cv.take<float>((size_t)p.rows * d.H * d.dk * 4);
    w.dvp = cv.take<float>((size_t)p.rows * d.H * d.dv * 4);
  }
  if (dg) {
    w.eq = cv.take<float>((size_t)p.rows * d.H * prism::LA_PARTS * 4);
    w.ek = cv.take<float>((size_t)p.rows * d.H * prism::LA_PARTS * 4);
    w.ST = cv.take<float>(p.bh * p.DD * 4);
    w.tmp = cv.take<float>((size_t)p.rows * d.H * 4);
  }
  return w;
}

prism_status check_offsets(const int* cu) {
  if (reinterpret_cast<uintptr_t>(cu) & 3u) return fail(PRISM_ERR_ALIGN, "cu_seqlens is not 4-byte aligned");
  return PRISM_OK;
}

template <typename E>
prism::LaArgs<E> la_args(const prism_linear_attention_desc& d, const LaPlan& p, const int* cu, const float* g) {
  prism::LaArgs<E> a = {};
  a.B = d.B;
  a.T = d.T;
  a.H = d.H;
  a.nseg = p.nseg;
  a.seglen = p.seglen;
  a.DD = (int)p.DD;
  a.cu = cu;
  a.N = d.packed_tokens;
  a.rows = p.rows;
  a.g = g;
  a.sg = strides(d.g);
  return a;
}

// Operands of one pass: rows a, b of da values, c of dc values; X's place in
// the [dv][dk] states follows from whether da is dk.
template <typename E>
prism::LaRole<E> la_role(const E* a, Strides sa, int ga, const E* b, Strides sb, int gb, const E* c, Strides sc, int gc,
                         int da, int dc, bool keys_first, const prism_linear_attention_desc& d) {
  prism::LaRole<E> r = {};
  r.a = a;
  r.b = b;
  r.c = c;
  r.sa = sa;
  r.sb = sb;
  r.sc = sc;
  r.ga = ga;
  r.gb = gb;
  r.gc = gc;
  r.ge = 1;
  r.da = da;
  r.dc = dc;
  r.xa = keys_first ? 1 : d.dk;
  r.xc = keys_first ? d.dk : 1;
  r.s_in = r.s_row = r.s_upd = 1.f;
  return r;
}

template <typename E>
prism_status la_forward(const prism_linear_attention_desc& d, const LaPlan& p, const E* q, const E* k, const E* v,
                        const float* g, const float* S0, const int* cu, E* o, float* ST, void* ws, hipStream_t s) {
  Carve cv;
  cv.base = static_cast<char*>(ws);
  const LaFwdWs w = carve_la_fwd(d, p, cv);
  prism::LaArgs<E> a = la_args<E>(d, p, cu, g);
  prism::LaRole<E> r =
      la_role<E>(q, strides(d.q), 1, k, strides(d.k), p.grp, v, strides(d.v), p.grp, d.dk, d.dv, true, d);
  r.s_in = r.s_row = d.scale;
  r.out = o;
  r.so = strides(d.o);
  r.X0 = S0;
  r.fin = ST;
  r.seg = w.seg;
  r.segdec = w.dec;
  a.r[0] = r;
  a.nroles = 1;
  if (p.nseg > 1)
    HIP_TRY("la_states", s, prism::launch_la_pass<E>(a, p.dim, ST ? prism::LA_STATES_FP32 : prism::LA_STATES, s));
  // (a state updated in place is written while other segments still start from
  // it, so they then start from the joined copies)
  if (p.nseg > LA_SELF_JOIN || (p.nseg > 1 && ST && ST == S0)) {
    prism::LaJoin j = {};
    j.B = d.B;
    j.T = d.T;
    j.H = d.H;
    j.nseg = p.nseg;
    j.seglen = p.seglen;
    j.DD = (int)p.DD;
    j.cu = cu;
    j.N = d.packed_tokens;
    j.seg[0] = w.seg;
    j.dec[0] = w.dec;
    j.X0[0] = S0;
    HIP_TRY("la_join", s, prism::launch_la_join(j, s));
    a.joined = 1;
  }
  HIP_TRY("la_fwd", s, prism::launch_la_pass<E>(a, p.dim, ST ? prism::LA_OUT_STATE : prism::LA_OUT, s));
  return PRISM_OK;
}

template <typename E>
prism_status la_backward(const prism_linear_attention_desc& d, const LaPlan& p, const E* q, const E* k, const E* v,
                         const float* g, const float* S0, const int* cu, const E* dO, const float* dST, E* dq, E* dk,
                         E* dv, float* dg, float* dS0, void* ws, hipStream_t s) {
  Carve cv;
  cv.base = static_cast<char*>(ws);
  const LaBwdWs w = carve_la_bwd(d, p, dg != nullptr, cv);
  const Strides sq = strides(d.q), sk = strides(d.k), sv = strides(d.v), so = strides(d.o);
  auto flat = [&](int H, int dim) { return Strides{(long)d.T * H * dim, (long)H * dim, (long)dim}; };
  // dq_t = scale sum_{i<=t} (dO_t . v_i) k_i: forward in time, through S
  prism::LaRole<E> rq = la_role<E>(dO, so, 1, v, sv, p.grp, k, sk, p.grp, d.dv, d.dk, false, d);
  rq.s_in = rq.s_row = d.scale;
  rq.out = dq;
  rq.so = flat(d.H, d.dk);
  rq.X0 = S0;
  rq.seg = w.segf;
  rq.segdec = w.decf;
  // dk_i = sum_{t>=i} scale (v_i . dO_t) q_t: backward in time, through dS
  prism::LaRole<E> rk = la_role<E>(v, sv, p.grp, dO, so, 1, q, sq, 1, d.dv, d.dk, false, d);
  rk.rev = 1;
  rk.s_in = rk.s_upd = d.scale;
  rk.out = p.grp > 1 ? nullptr : dk;
  rk.out32 = w.dkp;
  rk.so = flat(d.H, d.dk);
  rk.X0 = dST;
  rk.fin = dS0;
  rk.seg = w.segr;
  rk.segdec = w.decr;
  // dv_i = sum_{t>=i} scale (k_i . q_t) dO_t: the same state, transposed
  prism::LaRole<E> rv = la_role<E>(k, sk, p.grp, q, sq, 1, dO, so, 1, d.dk, d.dv, true, d);
  rv.rev = 1;
  rv.s_in = rv.s_upd = d.scale;
  rv.out = p.grp > 1 ? nullptr : dv;
  rv.out32 = w.dvp;
  rv.so = flat(d.H, d.dv);
  rv.X0 = dST;
  rv.seg = w.segr;
  rv.segdec = w.decr;
  prism::LaArgs<E> a = la_args<E>(d, p, cu, g);
  if (p.nseg > 1 && d.B > 0) {
    prism::LaArgs<E> b = a;
    b.r[0] = rq;
    b.r[1] = rk;
    b.nroles = 2;
    HIP_TRY("la_states", s,
            prism::launch_la_pass<E>(b, p.dim, dg || dS0 ? prism::LA_STATES_FP32 : prism::LA_STATES, s));
  }
  if (p.nseg > (dg ? LA_SELF_JOIN_DG : LA_SELF_JOIN) && d.B > 0) {
    prism::LaJoin j = {};
    j.B = d.B;
    j.T = d.T;
    j.H = d.H;
    j.nseg = p.nseg;
    j.seglen = p.seglen;
    j.DD = (int)p.DD;
    j.cu = cu;
    j.N = d.packed_tokens;
    j.seg[0] = w.segf;
    j.seg[1] = w.segr;
    j.dec[0] = w.decf;
    j.dec[1] = w.decr;
    j.X0[0] = S0;
    j.X0[1] = dST;
    HIP_TRY("la_join", s, prism::launch_la_join(j, s));
    a.joined = 1;
  }
  if (d.B > 0 && dg) {
    rq.e = q;
    rq.se = sq;
    rq.ge = 1;
    rq.edot = w.eq;
    rq.fin = dST ? w.ST : nullptr;
    rk.e = k;
    rk.se = sk;
    rk.ge = p.grp;
    rk.edot = w.ek;
    a.r[0] = rq;
    a.r[1] = rk;
    a.r[2] = rv;
    a.nroles = p.one ? 3 : 2;
    HIP_TRY("la_bwd_qk", s, prism::launch_la_pass<E>(a, p.dim, prism::LA_OUT_DOTS, s));
    if (!p.one) {
      a.r[0] = rv;
      a.nroles = 1;
      HIP_TRY("la_bwd_v", s, prism::launch_la_pass<E>(a, p.dim, prism::LA_OUT, s));
    }
  } else if (d.B > 0) {
    a.r[0] = rq;
    a.r[1] = rk;
    a.r[2] = rv;
    a.nroles = 3;
    HIP_TRY("la_bwd", s, prism::launch_la_pass<E>(a, p.dim, dS0 ? prism::LA_OUT_STATE : prism::LA_OUT, s));
  }
  if (dg) {
    prism::LaDecay x = {};
    x.B = d.B;
    x.T = d.T;
    x.H = d.H;
    x.nseg = p.nseg;
    x.seglen = p.seglen;
    x.DD = (int)p.DD;
    x.cu = cu;
    x.N = d.packed_tokens;
    x.rows = p.rows;
    x.g = g;
    x.sg = strides(d.g);
    x.eq = w.eq;
    x.ek = w.ek;
    x.segf = w.segf;
    x.segr = w.segr;
    x.decf = w.decf;
    x.decr = w.decr;
    x.joined = a.joined;
    x.S0 = S0;
    x.ST = w.ST;
    x.dST = dST;
    x.dg = dg;
    x.per_head = d.g.batch == 0 && d.g.token == 0;
    x.tmp = w.tmp;
    HIP_TRY("la_decay", s, prism::launch_la_decay(x, s));
  }
  if (p.grp > 1)
    HIP_TRY("la_group", s,
            prism::launch_la_group_sum<E>(w.dkp, w.dvp, dk, dv, p.rows, d.Hk, p.grp, d.dk, d.dv, s));
  return PRISM_OK;
}

bool has_tokens(const LaPlan& p) { return p.rows > 0; }

// Workspace of calls with cu_seqlens (packed), or of either layout: as many
// rows as the larger of the two has.
prism_status la_workspace(const prism_linear_attention_desc* desc, bool packed, bool backward, bool dg, size_t* bytes) {
  if (!bytes) return fail(PRISM_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  LaPlan p;
  const prism_status st = check_la(desc, packed, &p);
  if (st != PRISM_OK) return st;
  if (desc->packed_tokens > p.rows) p.rows = desc->packed_tokens;
  Carve cv;
  if (backward) {
    plan_backward(*desc, dg, &p);
    carve_la_bwd(*desc, p, dg, cv);
  } else {
    plan_forward(*desc, &p);
    carve_la_fwd(*desc, p, cv);
  }
  *bytes = cv.off;
  return PRISM_OK;
}

}  // namespace

extern "C" {

prism_status prism_qk_norm(const prism_qk_norm_desc* desc, const void* q, const void* k, const void* wq,
                           const void* wk, const int* positions, const long long* turns, void* qo, void* ko,
                           hipStream_t stream) {
  return prism::guarded([&] { return qk_forward(desc, q, k, wq, wk, positions, turns, qo, ko, stream); });
}

prism_status prism_qk_norm_backward_workspace(const prism_qk_norm_desc* desc, int weights, size_t* bytes) {
  return prism::guarded([&] {
    if (!bytes) return fail(PRISM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    const prism_status st = check_qk(desc, true);
    if (st == PRISM_OK && weights) *bytes = prism::qk_norm_part_bytes(desc->d);
    return st;
  });
}

prism_status prism_qk_norm_backward(const prism_qk_norm_desc* desc, const void* q, const void* k, const void* wq,
                                    const void* wk, const int* positions, const long long* turns, const void* dqo,
                                    const void* dko, void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  return prism::guarded([&] {
    return qk_backward(desc, q, k, wq, wk, positions, turns, dqo, dko, dq, dk, dwq, dwk, workspace, workspace_bytes,
                       stream);
  });
}

prism_status prism_linear_attention_workspace(const prism_linear_attention_desc* desc, int backward, int dg,
                                              size_t* bytes) {
  return prism::guarded([&] { return la_workspace(desc, false, backward != 0, dg != 0, bytes); });
}

prism_status prism_linear_attention_packed_workspace(const prism_linear_attention_desc* desc, int backward, int dg,
                                                     size_t* bytes) {
  return prism::guarded([&] { return la_workspace(desc, true, backward != 0, dg != 0, bytes); });
}

prism_status prism_linear_attention(const prism_linear_attention_desc* desc, const void* q, const void* k,
                                    const void* v, const float* g, const float* S0, const int* cu_seqlens, void* o,
                                    float* ST, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return prism::guarded([&]() -> prism_status {
    LaPlan p;
    prism_status st = check_la(desc, cu_seqlens != nullptr, &p);
    if (st != PRISM_OK) return st;
    if (cu_seqlens && (st = check_offsets(cu_seqlens)) != PRISM_OK) return st;
    if (desc->B == 0) return PRISM_OK;
    const bool some = has_tokens(p);
    CHECK_PTR(q, some);
    CHECK_PTR(k, some);
    CHECK_PTR(v, some);
    if (!g && some) return fail(PRISM_ERR_NULL, "g is NULL");
    if (reinterpret_cast<uintptr_t>(g) & 3u) return fail(PRISM_ERR_ALIGN, "g is not 4-byte aligned");
    CHECK_PTR(S0, false);
    CHECK_PTR(o, some);
    CHECK_PTR(ST, false);
    plan_forward(*desc, &p);
    Carve cv;
    carve_la_fwd(*desc, p, cv);
    if (cv.off > 0 && (st = check_buffer(workspace, workspace_bytes, cv.off, "workspace")) != PRISM_OK) return st;
    if (desc->dtype == PRISM_BF16)
      return la_forward<prism::bf16>(*desc, p, (const prism::bf16*)q, (const prism::bf16*)k, (const prism::bf16*)v, g,
                                     S0, cu_seqlens, (prism::bf16*)o, ST, workspace, stream);
    return la_forward<float>(*desc, p, (const float*)q, (const float*)k, (const float*)v, g, S0, cu_seqlens, (float*)o,
                             ST, workspace, stream);
  });
}

prism_status prism_linear_attention_backward(const prism_linear_attention_desc* desc, const void* q, const void* k,
                                             const void* v, const float* g, const float* S0, const int* cu_seqlens,
                                             const void* dO, const float* dST, void* dq, void* dk, void* dv,
                                             float* dg, float* dS0, void* workspace, size_t workspace_bytes,
                                             hipStream_t stream) {
  return prism::guarded([&]() -> prism_status {
    LaPlan p;
    prism_status st = check_la(desc, cu_seqlens != nullptr, &p);
    if (st != PRISM_OK) return st;
    if (cu_seqlens && (st = check_offsets(cu_seqlens)) != PRISM_OK) return st;
    const bool some = has_tokens(p);
    CHECK_PTR(q, some);
    CHECK_PTR(k, some);
    CHECK_PTR(v, some);
    if (!g && some) return fail(PRISM_ERR_NULL, "g is NULL");
    if (reinterpret_cast<uintptr_t>(g) & 3u) return fail(PRISM_ERR_ALIGN, "g is not 4-byte aligned");
    CHECK_PTR(S0, false);
    CHECK_PTR(dO, some);
    CHECK_PTR(dST, false);
    CHECK_PTR(dq, some);
    CHECK_PTR(dk, some);
    CHECK_PTR(dv, some);
    if (reinterpret_cast<uintptr_t>(dg) & 3u) return fail(PRISM_ERR_ALIGN, "dg is not 4-byte aligned");
    CHECK_PTR(dS0, false);
    if (dg && some) {
      // dg has g's strides: a value of g that serves several tokens or heads
      // would be written by each of them (one a head is summed)
      const prism_strides& x = desc->g;
      const bool head = x.batch == 0 && x.token == 0;
      if ((x.head == 0 && desc->H > 1) || (!head && x.token == 0 && desc->T > 1) ||
          (!head && !cu_seqlens && x.batch == 0 && desc->B > 1) || (!head && cu_seqlens && x.token == 0))
        return fail(PRISM_ERR_UNSUPPORTED, "dg needs a g for each token and head, or one for each head");
    }
    if (dS0 && (dS0 == dST || dS0 == S0))
      return fail(PRISM_ERR_UNSUPPORTED, "dS0 must not be the buffer of dST or S0");
    if (desc->B == 0 && !dg) return PRISM_OK;
    plan_backward(*desc, dg != 0, &p);
    Carve cv;
    carve_la_bwd(*desc, p, dg != nullptr, cv);
    if (cv.off > 0 && (st = check_buffer(workspace, workspace_bytes, cv.off, "workspace")) != PRISM_OK) return st;
    if (desc->dtype == PRISM_BF16)
      return la_backward<prism::bf16>(*desc, p, (const prism::bf16*)q, (const prism::bf16*)k, (const prism::bf16*)v, g,
                                      S0, cu_seqlens, (const prism::bf16*)dO, dST, (prism::bf16*)dq, (prism::bf16*)dk,
                                      (prism::bf16*)dv, dg, dS0, workspace, stream);
    return la_backward<float>(*desc, p, (const float*)q, (const float*)k, (const float*)v, g, S0, cu_seqlens,
                              (const float*)dO, dST, (float*)dq, (float*)dk, (float*)dv, dg, dS0, workspace, stream);
  });
}

prism_status prism_linear_attention_step(const prism_linear_attention_desc* desc, const void* q, const void* k,
                                         const void* v, const float* g, const float* S, float* S_out, void* o,
                                         hipStream_t stream) {
  return prism::guarded([&]() -> prism_status {
    LaPlan p;
    const prism_status st = check_la(desc, false, &p);
    if (st != PRISM_OK) return st;
    if (desc->B == 0) return PRISM_OK;
    const bool some = has_tokens(p);
    CHECK_PTR(q, some);
    CHECK_PTR(k, some);
    CHECK_PTR(v, some);
    if (!g && some) return fail(PRISM_ERR_NULL, "g is NULL");
    if (reinterpret_cast<uintptr_t>(g) & 3u) return fail(PRISM_ERR_ALIGN, "g is not 4-byte aligned");
    CHECK_PTR(S, true);
    CHECK_PTR(S_out, true);
    CHECK_PTR(o, some);
    auto run = [&](auto zero) -> hipError_t {
      typedef decltype(zero) E;
      prism::LaStepArgs<E> a = {};
      a.B = desc->B;
      a.T = desc->T;
      a.H = desc->H;
      a.dk = desc->dk;
      a.dv = desc->dv;
      a.grp = p.grp;
      a.scale = desc->scale;
      a.q = (const E*)q;
      a.k = (const E*)k;
      a.v = (const E*)v;
      a.sq = strides(desc->q);
      a.sk = strides(desc->k);
      a.sv = strides(desc->v);
      a.so = strides(desc->o);
      a.sg = strides(desc->g);
      a.g = g;
      a.S = S;
      a.S_out = S_out;
      a.o = (E*)o;
      return prism::launch_la_step<E>(a, stream);
    };
    HIP_TRY("la_step", stream, desc->dtype == PRISM_BF16 ? run((prism::bf16)0.f) : run(0.f));
    return PRISM_OK;
  });
}

}  // extern "C"
