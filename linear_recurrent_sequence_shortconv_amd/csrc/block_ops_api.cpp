// C ABI of the operators of a recurrent block (layer norm, short convolution,
// gated recurrence): checks, workspace sizes and launch sequences.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <string>

#include "api_common.h"
#include "block_ops.h"

namespace {

using prism::check_buffer;
using prism::fail;
using prism::guarded;
using prism::Strides;
using prism::TokenSteps;

std::string num(long long x) { return std::to_string(x); }

Strides strides(const prism_strides& s) { return Strides{(long)s.batch, (long)s.token, (long)s.head}; }
TokenSteps steps(const prism_strides& s) { return TokenSteps{(long)s.batch, (long)s.token}; }

// Rows of a launch.
constexpr long long MOST_ROWS = 1LL << 30;

prism_status check_elem(const void* p, const char* name, bool required, int size) {
  if (!p) return required ? fail(PRISM_ERR_NULL, std::string(name) + " is NULL") : PRISM_OK;
  if (reinterpret_cast<uintptr_t>(p) & (unsigned)(size - 1))
    return fail(PRISM_ERR_ALIGN, std::string(name) + " is not " + num(size) + "-byte aligned");
  return PRISM_OK;
}
#define CHECK_ELEM(p, req, size)                               \
  do {                                                         \
    prism_status st_ = check_elem((p), #p, (req), (size));     \
    if (st_ != PRISM_OK) return st_;                           \
  } while (0)

// Steps of a tensor of rows of D values whose dimensions (batch, token, head) have n
// entries; of a result, none that would put values of several rows in one place:
// from the smallest to the largest, each step leaves the rows inside it behind.
prism_status check_steps(const prism_strides& s, const char* name, const long long (&n)[3], int D, bool result) {
  const long long v[3] = {s.batch, s.token, s.head};
  constexpr long long MOST = 1LL << 40;
  for (int k = 0; k < 3; ++k)
    if (v[k] >= MOST || v[k] <= -MOST)
      return fail(PRISM_ERR_SHAPE, std::string("strides of ") + name + " out of range");
  if (!result || !n[0] || !n[1] || !n[2]) return PRISM_OK;
  long long reach = D;   // of the rows inside a dimension (no step is beyond MOST)
  bool taken[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
  while (true) {
    int k = -1;
    for (int m = 0; m < 3; ++m)
      if (!taken[m] && (k < 0 || std::llabs(v[m]) < std::llabs(v[k]))) k = m;
    if (k < 0) return PRISM_OK;
    const long long step = std::llabs(v[k]);
    if (step < reach)
      return fail(PRISM_ERR_SHAPE, std::string("strides of ") + name + " put several rows in one place");
    reach = (n[k] - 1) >= MOST / step ? MOST : reach + step * (n[k] - 1);
    taken[k] = true;
  }
}

prism_status check_dtype(prism_dtype t) {
  if (t != PRISM_F32 && t != PRISM_BF16) return fail(PRISM_ERR_UNSUPPORTED, "dtype must be PRISM_F32 or PRISM_BF16");
  return PRISM_OK;
}
int size_of(prism_dtype t) { return t == PRISM_BF16 ? 2 : 4; }

// --------------------------------------------------------------- layer norm
prism_status check_ln(const prism_layer_norm_desc* desc) {
  if (!desc) return fail(PRISM_ERR_NULL, "desc is NULL");
  const prism_layer_norm_desc& d = *desc;
  if (d.B < 0 || d.T < 0 || d.H < 0)
    return fail(PRISM_ERR_SHAPE, "B, T and H must be >= 0 (got B=" + num(d.B) + " T=" + num(d.T) + " H=" + num(d.H) + ")");
  // (two products: three 31-bit sizes leave 64 bits)
  const long long bt = (long long)d.B * d.T;
  if (bt > 0 && d.H > 0 && (bt > MOST_ROWS || bt * d.H > MOST_ROWS))
    return fail(PRISM_ERR_SHAPE, "B * T * H must be <= " + num(MOST_ROWS));
  if (d.D < 1) return fail(PRISM_ERR_SHAPE, "D must be >= 1 (got " + num(d.D) + ")");
  const prism_status st = check_dtype(d.dtype);
  if (st != PRISM_OK) return st;
  if (d.D > prism::LN_MAX_D)
    return fail(PRISM_ERR_UNSUPPORTED, "D must be <= " + num(prism::LN_MAX_D) + " (got " + num(d.D) + ")");
  if (d.norm != PRISM_NORM_RMS && d.norm != PRISM_NORM_LAYER)
    return fail(PRISM_ERR_UNSUPPORTED, "norm must be PRISM_NORM_RMS or PRISM_NORM_LAYER");
  if (!(d.eps >= 0.f) || !std::isfinite(d.eps)) return fail(PRISM_ERR_SHAPE, "eps must be finite and >= 0");
  return PRISM_OK;
}

prism::LayerNormArgs ln_args(const prism_layer_norm_desc& d, const void* x, const void* w) {
  prism::LayerNormArgs a = {};
  a.rows = (long)d.B * d.T * d.H;
  a.T = d.T;
  a.H = d.H;
  a.D = d.D;
  a.center = d.norm == PRISM_NORM_LAYER;
  a.eps = d.eps;
  a.x = x;
  a.w = w;
  a.sx = strides(d.x);
  a.sr = strides(d.r);
  a.sy = strides(d.y);
  a.sh = strides(d.h);
  return a;
}

prism_status ln_forward(const prism_layer_norm_desc* desc, const void* x, const void* residual, const void* w,
                        const void* b, void* y, void* h, hipStream_t stream) {
  prism_status st = check_ln(desc);
  if (st != PRISM_OK) return st;
  const prism_layer_norm_desc& d = *desc;
  const long long n[3] = {d.B, d.T, d.H};
  const int size = size_of(d.dtype);
  if (n[0] * n[1] == 0 || n[2] == 0) return PRISM_OK;
  CHECK_ELEM(x, true, size);
  CHECK_ELEM(residual, false, size);
  CHECK_ELEM(w, false, size);
  CHECK_ELEM(b, false, size);
  CHECK_ELEM(y, true, size);
  CHECK_ELEM(h, false, size);
  if (h && !residual) return fail(PRISM_ERR_NULL, "h without residual");
  if ((st = check_steps(d.x, "x", n, d.D, false)) != PRISM_OK) return st;
  if (residual && (st = check_steps(d.r, "residual", n, d.D, false)) != PRISM_OK) return st;
  if ((st = check_steps(d.y, "y", n, d.D, true)) != PRISM_OK) return st;
  if (h && (st = check_steps(d.h, "h", n, d.D, true)) != PRISM_OK) return st;
  prism::LayerNormArgs a = ln_args(d, x, w);
  a.r = residual;
  a.b = b;
  a.y = y;
  a.h = h;
  HIP_TRY("layer_norm", stream, d.dtype == PRISM_BF16 ? prism::launch_layer_norm<prism::bf16>(a, stream)
                                                      : prism::launch_layer_norm<float>(a, stream));
  return PRISM_OK;
}

prism_status ln_backward(const prism_layer_norm_desc* desc, const void* x, const void* w, const void* dy, const void* dh,
                         void* dx, float* dw, float* db, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  prism_status st = check_ln(desc);
  if (st != PRISM_OK) return st;
  const prism_layer_norm_desc& d = *desc;
  const long long n[3] = {d.B, d.T, d.H};
  const int size = size_of(d.dtype);
  const bool some = n[0] * n[1] > 0 && n[2] > 0;
  CHECK_ELEM(x, some, size);
  CHECK_ELEM(w, false, size);
  CHECK_ELEM(dy, some, size);
  CHECK_ELEM(dh, false, size);
  CHECK_ELEM(dx, some, size);
  CHECK_ELEM(dw, false, 4);
  CHECK_ELEM(db, false, 4);
  if ((st = check_steps(d.x, "x", n, d.D, false)) != PRISM_OK) return st;
  if ((st = check_steps(d.y, "dy", n, d.D, false)) != PRISM_OK) return st;
  if (dh && (st = check_steps(d.r, "dh", n, d.D, false)) != PRISM_OK) return st;
  if ((st = check_steps(d.h, "dx", n, d.D, true)) != PRISM_OK) return st;
  if (!some && !dw && !db) return PRISM_OK;
  prism::LayerNormArgs a = ln_args(d, x, w);
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  if (dw || db) {
    st = check_buffer(workspace, workspace_bytes, prism::layer_norm_part_bytes(d.D), "workspace");
    if (st != PRISM_OK) return st;
    a.part = static_cast<float*>(workspace);
  }
  HIP_TRY("layer_norm_bwd", stream, d.dtype == PRISM_BF16 ? prism::launch_layer_norm_bwd<prism::bf16>(a, stream)
                                                          : prism::launch_layer_norm_bwd<float>(a, stream));
  return PRISM_OK;
}

// ----------------------------------------------- batches of token sequences
// B, T, D, dtype and rows of a dense or packed batch.
prism_status check_batch(int B, int T, int D, prism_dtype dtype, int packed_tokens, bool packed) {
  if (B < 0 || T < 0)
    return fail(PRISM_ERR_SHAPE, "B and T must be >= 0 (got B=" + num(B) + " T=" + num(T) + ")");
  if (D < 1 || D > (1 << 22)) return fail(PRISM_ERR_SHAPE, "D must be from 1 to 4194304 (got " + num(D) + ")");
  if (packed && packed_tokens < 0) return fail(PRISM_ERR_SHAPE, "packed_tokens must be >= 0 with cu_seqlens");
  const long long rows = packed ? packed_tokens : (long long)B * T;
  if (rows > MOST_ROWS) return fail(PRISM_ERR_SHAPE, "a batch has at most " + num(MOST_ROWS) + " tokens");
  // (a launch has under 2^32 threads, 256 for 256 channels of a sequence)
  if ((long long)B * D >= (1LL << 31) || B * ((D + 255LL) / 256) >= (1LL << 23))
    return fail(PRISM_ERR_SHAPE, "problem too large: B * D has to be below 2^31, B * ceil(D / 256) below 2^23");
  return check_dtype(dtype);
}

prism_status check_token_steps(const prism_strides& s, const char* name, int B, int T, int D, int rows, bool packed,
                               bool result) {
  const long long n[3] = {packed ? 1 : B, packed ? rows : T, 1};
  return check_steps(prism_strides{s.batch, s.token, 0}, name, n, D, result);
}

prism_status check_cu(const int* cu) {
  if (reinterpret_cast<uintptr_t>(cu) & 3u) return fail(PRISM_ERR_ALIGN, "cu_seqlens is not 4-byte aligned");
  return PRISM_OK;
}

// -------------------------------------------------------- short convolution
prism_status check_conv(const prism_short_conv_desc* desc, bool packed, prism::ShortConvArgs* a) {
  if (!desc) return fail(PRISM_ERR_NULL, "desc is NULL");
  const prism_short_conv_desc& d = *desc;
  const prism_status st = check_batch(d.B, d.T, d.D, d.dtype, d.packed_tokens, packed);
  if (st != PRISM_OK) return st;
  if (d.K < 2 || d.K > 4) return fail(PRISM_ERR_UNSUPPORTED, "K must be from 2 to 4 (got " + num(d.K) + ")");
  if (d.activation != PRISM_ACT_IDENTITY && d.activation != PRISM_ACT_SILU)
    return fail(PRISM_ERR_UNSUPPORTED, "activation must be PRISM_ACT_IDENTITY or PRISM_ACT_SILU");
  *a = prism::ShortConvArgs{};
  a->B = d.B;
  a->T = d.T;
  a->D = d.D;
  a->K = d.K;
  a->rows = packed ? d.packed_tokens : d.B * d.T;
  a->silu = d.activation == PRISM_ACT_SILU;
  a->sx = steps(d.x);
  a->sy = steps(d.y);
  a->sd = steps(d.dx);
  return PRISM_OK;
}

prism_status conv_forward(const prism_short_conv_desc* desc, const void* x, const void* w, const void* b,
                          const void* hist, const int* cu, void* y, void* hist_out, hipStream_t stream) {
  prism::ShortConvArgs a;
  const bool packed = cu != nullptr;
  prism_status st = check_conv(desc, packed, &a);
  if (st != PRISM_OK) return st;
  const prism_short_conv_desc& d = *desc;
  const int size = size_of(d.dtype);
  const bool some = a.rows > 0 && d.B > 0;
  CHECK_ELEM(x, some, size);
  CHECK_ELEM(w, some, size);
  CHECK_ELEM(b, false, size);
  CHECK_ELEM(hist, false, size);
  CHECK_ELEM(y, some, size);
  CHECK_ELEM(hist_out, false, size);
  if ((st = check_cu(cu)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.x, "x", d.B, d.T, d.D, a.rows, packed, false)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.y, "y", d.B, d.T, d.D, a.rows, packed, true)) != PRISM_OK) return st;
  a.cu = cu;
  a.x = x;
  a.w = w;
  a.b = b;
  a.hist = hist;
  a.y = y;
  a.hist_out = hist_out;
  if (d.B == 0) return PRISM_OK;
  HIP_TRY("short_conv", stream, d.dtype == PRISM_BF16 ? prism::launch_short_conv<prism::bf16>(a, stream)
                                                      : prism::launch_short_conv<float>(a, stream));
  return PRISM_OK;
}

prism_status conv_backward(const prism_short_conv_desc* desc, const void* x, const void* w, const void* b,
                           const void* hist, const int* cu, const void* dy, void* dx, float* dw, float* db, float* dhist,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  prism::ShortConvArgs a;
  const bool packed = cu != nullptr;
  prism_status st = check_conv(desc, packed, &a);
  if (st != PRISM_OK) return st;
  const prism_short_conv_desc& d = *desc;
  const int size = size_of(d.dtype);
  if (d.B == 0) a.rows = 0;
  const bool some = a.rows > 0;
  CHECK_ELEM(x, some, size);
  CHECK_ELEM(w, some, size);
  CHECK_ELEM(b, false, size);
  CHECK_ELEM(hist, false, size);
  CHECK_ELEM(dy, some, size);
  CHECK_ELEM(dx, some, size);
  CHECK_ELEM(dw, true, 4);
  CHECK_ELEM(db, false, 4);
  CHECK_ELEM(dhist, false, 4);
  if ((st = check_cu(cu)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.x, "x", d.B, d.T, d.D, a.rows, packed, false)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.y, "dy", d.B, d.T, d.D, a.rows, packed, false)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.dx, "dx", d.B, d.T, d.D, a.rows, packed, true)) != PRISM_OK) return st;
  const size_t need = prism::short_conv_part_bytes(a.rows, d.D, d.K);
  if (need > 0 && (st = check_buffer(workspace, workspace_bytes, need, "workspace")) != PRISM_OK) return st;
  a.cu = cu;
  a.x = x;
  a.w = w;
  a.b = b;
  a.hist = hist;
  a.dy = dy;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  a.dhist = dhist;
  a.part = static_cast<float*>(workspace);
  HIP_TRY("short_conv_bwd", stream, d.dtype == PRISM_BF16 ? prism::launch_short_conv_bwd<prism::bf16>(a, stream)
                                                          : prism::launch_short_conv_bwd<float>(a, stream));
  return PRISM_OK;
}

// --------------------------------------------------------- gated recurrence
prism_status check_rec(const prism_gated_recurrence_desc* desc, bool packed, prism::RecurrenceArgs* a) {
  if (!desc) return fail(PRISM_ERR_NULL, "desc is NULL");
  const prism_gated_recurrence_desc& d = *desc;
  const prism_status st = check_batch(d.B, d.T, d.D, d.dtype, d.packed_tokens, packed);
  if (st != PRISM_OK) return st;
  if (d.gate != PRISM_GATE_LOG && d.gate != PRISM_GATE_SIGMOID && d.gate != PRISM_GATE_POWER)
    return fail(PRISM_ERR_UNSUPPORTED, "gate must be PRISM_GATE_LOG, PRISM_GATE_SIGMOID or PRISM_GATE_POWER");
  // (a tile of at least 64 rows and 64 channels is 512 threads)
  const long long rows = packed ? d.packed_tokens : (long long)d.B * d.T;
  if ((rows + 63) / 64 * ((d.D + 63) / 64) > (1LL << 22))
    return fail(PRISM_ERR_SHAPE, "problem too large: ceil(tokens / 64) * ceil(D / 64) has to be at most 2^22");
  *a = prism::RecurrenceArgs{};
  a->B = d.B;
  a->T = d.T;
  a->D = d.D;
  a->rows = packed ? d.packed_tokens : d.B * d.T;
  a->gate = d.gate == PRISM_GATE_LOG       ? prism::GATE_LOG
            : d.gate == PRISM_GATE_SIGMOID ? prism::GATE_SIGMOID
                                           : prism::GATE_POWER;
  a->sx = steps(d.x);
  a->sf = steps(d.f);
  a->si = steps(d.i);
  a->sh = steps(d.h);
  a->sdh = steps(d.dh);
  a->sdx = steps(d.dx);
  a->sdf = steps(d.df);
  a->sdi = steps(d.di);
  return PRISM_OK;
}

// What forward, step and backward read.
prism_status check_rec_inputs(const prism_gated_recurrence_desc& d, bool packed, int rows, const void* x, const void* f,
                              const void* i, const float* lam, const float* h0) {
  const int size = size_of(d.dtype);
  const bool some = rows > 0 && d.B > 0;
  CHECK_ELEM(x, some, size);
  CHECK_ELEM(f, some, size);
  CHECK_ELEM(i, false, size);
  CHECK_ELEM(lam, some && d.gate == PRISM_GATE_POWER, 4);
  if (lam && d.gate != PRISM_GATE_POWER) return fail(PRISM_ERR_UNSUPPORTED, "lam goes with PRISM_GATE_POWER alone");
  CHECK_ELEM(h0, false, 4);
  prism_status st;
  if ((st = check_token_steps(d.x, "x", d.B, d.T, d.D, rows, packed, false)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.f, "f", d.B, d.T, d.D, rows, packed, false)) != PRISM_OK) return st;
  if (i && (st = check_token_steps(d.i, "i", d.B, d.T, d.D, rows, packed, false)) != PRISM_OK) return st;
  return PRISM_OK;
}

prism_status rec_forward(const prism_gated_recurrence_desc* desc, const void* x, const void* f, const void* i,
                         const float* lam, const float* h0, const int* cu, void* h, float* hT, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  prism::RecurrenceArgs a;
  const bool packed = cu != nullptr;
  prism_status st = check_rec(desc, packed, &a);
  if (st != PRISM_OK) return st;
  const prism_gated_recurrence_desc& d = *desc;
  if ((st = check_rec_inputs(d, packed, a.rows, x, f, i, lam, h0)) != PRISM_OK) return st;
  CHECK_ELEM(h, a.rows > 0 && d.B > 0, size_of(d.dtype));
  CHECK_ELEM(hT, false, 4);
  if ((st = check_cu(cu)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.h, "h", d.B, d.T, d.D, a.rows, packed, true)) != PRISM_OK) return st;
  a.cu = cu;
  a.x = x;
  a.f = f;
  a.i = i;
  a.lam = lam;
  a.h0 = h0;
  a.h = h;
  a.hT = hT;
  const size_t need = prism::recurrence_bytes(a, packed, false);
  if (need > 0 && (st = check_buffer(workspace, workspace_bytes, need, "workspace")) != PRISM_OK) return st;
  HIP_TRY("recurrence", stream, prism::launch_recurrence(a, d.dtype == PRISM_F32, false, workspace, stream));
  return PRISM_OK;
}

prism_status rec_backward(const prism_gated_recurrence_desc* desc, const void* x, const void* f, const void* i,
                          const float* lam, const float* h0, const int* cu, const void* h, const void* dh,
                          const float* dhT, void* dx, void* df, void* di, float* dlam, float* dh0, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  prism::RecurrenceArgs a;
  const bool packed = cu != nullptr;
  prism_status st = check_rec(desc, packed, &a);
  if (st != PRISM_OK) return st;
  const prism_gated_recurrence_desc& d = *desc;
  if ((st = check_rec_inputs(d, packed, a.rows, x, f, i, lam, h0)) != PRISM_OK) return st;
  const int size = size_of(d.dtype);
  const bool some = a.rows > 0 && d.B > 0;
  CHECK_ELEM(h, some, size);
  CHECK_ELEM(dh, some, size);
  CHECK_ELEM(dhT, false, 4);
  CHECK_ELEM(dx, some, size);
  CHECK_ELEM(df, some, size);
  CHECK_ELEM(di, some && i != nullptr, size);
  CHECK_ELEM(dlam, d.gate == PRISM_GATE_POWER, 4);
  CHECK_ELEM(dh0, false, 4);
  if ((st = check_cu(cu)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.h, "h", d.B, d.T, d.D, a.rows, packed, false)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.dh, "dh", d.B, d.T, d.D, a.rows, packed, false)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.dx, "dx", d.B, d.T, d.D, a.rows, packed, true)) != PRISM_OK) return st;
  if ((st = check_token_steps(d.df, "df", d.B, d.T, d.D, a.rows, packed, true)) != PRISM_OK) return st;
  if (i && (st = check_token_steps(d.di, "di", d.B, d.T, d.D, a.rows, packed, true)) != PRISM_OK) return st;
  if (dh0 && (dh0 == dhT || dh0 == h0)) return fail(PRISM_ERR_UNSUPPORTED, "dh0 is the buffer of dhT or h0");
  const size_t need = prism::recurrence_bytes(a, packed, true);
  if (need > 0 && (st = check_buffer(workspace, workspace_bytes, need, "workspace")) != PRISM_OK) return st;
  a.cu = cu;
  a.x = x;
  a.f = f;
  a.i = i;
  a.lam = lam;
  a.h0 = h0;
  a.h = const_cast<void*>(h);
  a.dh = dh;
  a.dhT = dhT;
  a.dx = dx;
  a.df = df;
  a.di = i ? di : nullptr;
  a.dlam = dlam;
  a.dh0 = dh0;
  HIP_TRY("recurrence_bwd", stream, prism::launch_recurrence(a, d.dtype == PRISM_F32, true, workspace, stream));
  return PRISM_OK;
}

}  // namespace

extern "C" {

prism_status prism_layer_norm(const prism_layer_norm_desc* desc, const void* x, const void* residual, const void* w,
                              const void* b, void* y, void* h, hipStream_t stream) {
  return guarded([&] { return ln_forward(desc, x, residual, w, b, y, h, stream); });
}

prism_status prism_layer_norm_backward_workspace(const prism_layer_norm_desc* desc, int weights, size_t* bytes) {
  return guarded([&]() -> prism_status {
    if (!bytes) return fail(PRISM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    const prism_status st = check_ln(desc);
    if (st != PRISM_OK) return st;
    if (weights) *bytes = prism::layer_norm_part_bytes(desc->D);
    return PRISM_OK;
  });
}

prism_status prism_layer_norm_backward(const prism_layer_norm_desc* desc, const void* x, const void* w, const void* dy,
                                       const void* dh, void* dx, float* dw, float* db, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  return guarded([&] { return ln_backward(desc, x, w, dy, dh, dx, dw, db, workspace, workspace_bytes, stream); });
}

prism_status prism_short_conv(const prism_short_conv_desc* desc, const void* x, const void* w, const void* b,
                              const void* hist, const int* cu_seqlens, void* y, void* hist_out, hipStream_t stream) {
  return guarded([&] { return conv_forward(desc, x, w, b, hist, cu_seqlens, y, hist_out, stream); });
}

prism_status prism_short_conv_backward_workspace(const prism_short_conv_desc* desc, int packed, size_t* bytes) {
  return guarded([&]() -> prism_status {
    if (!bytes) return fail(PRISM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    prism::ShortConvArgs a;
    const prism_status st = check_conv(desc, packed != 0, &a);
    if (st != PRISM_OK) return st;
    *bytes = desc->B ? prism::short_conv_part_bytes(a.rows, desc->D, desc->K) : 0;
    return PRISM_OK;
  });
}

prism_status prism_short_conv_backward(const prism_short_conv_desc* desc, const void* x, const void* w, const void* b,
                                       const void* hist, const int* cu_seqlens, const void* dy, void* dx, float* dw,
                                       float* db, float* dhist, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
  return guarded([&] {
    return conv_backward(desc, x, w, b, hist, cu_seqlens, dy, dx, dw, db, dhist, workspace, workspace_bytes, stream);
  });
}

prism_status prism_gated_recurrence_workspace(const prism_gated_recurrence_desc* desc, int packed, int backward,
                                              size_t* bytes) {
  return guarded([&]() -> prism_status {
    if (!bytes) return fail(PRISM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    prism::RecurrenceArgs a;
    const prism_status st = check_rec(desc, packed != 0, &a);
    if (st != PRISM_OK) return st;
    *bytes = prism::recurrence_bytes(a, packed != 0, backward != 0);
    return PRISM_OK;
  });
}

prism_status prism_gated_recurrence(const prism_gated_recurrence_desc* desc, const void* x, const void* f, const void* i,
                                    const float* lam, const float* h0, const int* cu_seqlens, void* h, float* hT,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return guarded(
      [&] { return rec_forward(desc, x, f, i, lam, h0, cu_seqlens, h, hT, workspace, workspace_bytes, stream); });
}

prism_status prism_gated_recurrence_backward(const prism_gated_recurrence_desc* desc, const void* x, const void* f,
                                             const void* i, const float* lam, const float* h0, const int* cu_seqlens,
                                             const void* h, const void* dh, const float* dhT, void* dx, void* df,
                                             void* di, float* dlam, float* dh0, void* workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
  return guarded([&] {
    return rec_backward(desc, x, f, i, lam, h0, cu_seqlens, h, dh, dhT, dx, df, di, dlam, dh0, workspace,
                        workspace_bytes, stream);
  });
}

prism_status prism_gated_recurrence_step(const prism_gated_recurrence_desc* desc, const void* x, const void* f,
                                         const void* i, const float* lam, const float* state, float* state_out, void* h,
                                         hipStream_t stream) {
  return guarded([&]() -> prism_status {
    prism::RecurrenceArgs a;
    prism_status st = check_rec(desc, false, &a);
    if (st != PRISM_OK) return st;
    const prism_gated_recurrence_desc& d = *desc;
    if ((st = check_rec_inputs(d, false, a.rows, x, f, i, lam, nullptr)) != PRISM_OK) return st;
    CHECK_ELEM(lam, d.B > 0 && d.gate == PRISM_GATE_POWER, 4);   // (read without tokens too)
    CHECK_ELEM(state, d.B > 0, 4);
    CHECK_ELEM(state_out, d.B > 0, 4);
    CHECK_ELEM(h, a.rows > 0, size_of(d.dtype));
    if ((st = check_token_steps(d.h, "h", d.B, d.T, d.D, a.rows, false, true)) != PRISM_OK) return st;
    a.x = x;
    a.f = f;
    a.i = i;
    a.lam = lam;
    a.h0 = state;
    a.h = h;
    a.hT = state_out;
    HIP_TRY("recurrence_step", stream, prism::launch_recurrence_step(a, d.dtype == PRISM_F32, stream));
    return PRISM_OK;
  });
}

}  // extern "C"
