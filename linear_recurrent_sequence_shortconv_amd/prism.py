"""Thin ctypes binding of libprism.so (the C ABI in include/prism.h).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI.  PyTorch provides device memory (outputs, workspace) and
the current stream.  There is no fallback: if the library is missing or a
call fails, a RuntimeError is raised.
"""
import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libprism.so")

PRISM_F32 = 0
PRISM_BF16 = 1
STATUS = {0: "PRISM_OK", 1: "PRISM_ERR_NULL", 2: "PRISM_ERR_SHAPE", 3: "PRISM_ERR_UNSUPPORTED",
          4: "PRISM_ERR_ALIGN", 5: "PRISM_ERR_WORKSPACE", 6: "PRISM_ERR_HIP"}

EXPORTS = ("prism_forward_workspace", "prism_backward_workspace",
           "prism_forward_train_workspace", "prism_backward_train_workspace", "prism_forward",
           "prism_backward", "prism_saved_bytes", "prism_forward_train", "prism_backward_train",
           "prism_step_workspace", "prism_step", "prism_step_noalloc", "prism_status_string", "prism_last_error", "prism_timing_begin",
           "prism_timing_end",
           "prism_qk_norm", "prism_qk_norm_backward_workspace", "prism_qk_norm_backward",
           "prism_linear_attention_workspace", "prism_linear_attention_packed_workspace",
           "prism_linear_attention",
           "prism_linear_attention_backward", "prism_linear_attention_step",
           "prism_layer_norm", "prism_layer_norm_backward_workspace", "prism_layer_norm_backward",
           "prism_short_conv", "prism_short_conv_backward_workspace", "prism_short_conv_backward",
           "prism_gated_recurrence_workspace", "prism_gated_recurrence",
           "prism_gated_recurrence_backward", "prism_gated_recurrence_step")


class Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("L", ctypes.c_int),
                ("chunk", ctypes.c_int), ("conv_width", ctypes.c_int), ("dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("conv_offset", ctypes.c_int),
                ("packed_tokens", ctypes.c_int)]


class Strides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_longlong), ("token", ctypes.c_longlong),
                ("head", ctypes.c_longlong)]


class QkNormDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hk", ctypes.c_int), ("d", ctypes.c_int), ("rot", ctypes.c_int),
                ("dtype", ctypes.c_int), ("norm", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("eps", ctypes.c_float), ("q", Strides), ("k", Strides), ("qo", Strides),
                ("ko", Strides), ("dq", Strides), ("dk", Strides)]


class LinearAttentionDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("Hk", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("packed_tokens", ctypes.c_int), ("q", Strides), ("k", Strides), ("v", Strides),
                ("o", Strides), ("g", Strides)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("norm", ctypes.c_int), ("eps", ctypes.c_float),
                ("x", Strides), ("r", Strides), ("y", Strides), ("h", Strides)]


class ShortConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int), ("K", ctypes.c_int),
                ("dtype", ctypes.c_int), ("activation", ctypes.c_int),
                ("packed_tokens", ctypes.c_int), ("x", Strides), ("y", Strides), ("dx", Strides)]


class GatedRecurrenceDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("gate", ctypes.c_int), ("packed_tokens", ctypes.c_int),
                ("x", Strides), ("f", Strides), ("i", Strides), ("h", Strides), ("dh", Strides),
                ("dx", Strides), ("df", Strides), ("di", Strides)]


_lib = None
_P = ctypes.c_void_p


def lib():
    """Load libprism.so once.  torch is imported first so that its HIP runtime
    (same SONAME as the system one) is the single runtime in the process."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "`python -m linear_recurrent_sequence_shortconv_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.prism_forward_workspace.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(ctypes.c_size_t)]
        L.prism_backward_workspace.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(ctypes.c_size_t)]
        L.prism_forward_train_workspace.argtypes = [ctypes.POINTER(Desc),
                                                    ctypes.POINTER(ctypes.c_size_t)]
        L.prism_backward_train_workspace.argtypes = [ctypes.POINTER(Desc),
                                                     ctypes.POINTER(ctypes.c_size_t)]
        # inputs q..conv, S0, conv_hist, cu_seqlens (12); forward outputs o, ST,
        # conv_hist_out (3); backward: dO, dST, then 11 gradients (dq..dconv, dS0, dconv_hist)
        L.prism_forward.argtypes = [ctypes.POINTER(Desc)] + [_P] * 15 + [_P, ctypes.c_size_t, _P]
        L.prism_backward.argtypes = [ctypes.POINTER(Desc)] + [_P] * 25 + [_P, ctypes.c_size_t, _P]
        L.prism_saved_bytes.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(ctypes.c_size_t)]
        L.prism_forward_train.argtypes = ([ctypes.POINTER(Desc)] + [_P] * 15
                                          + [_P, ctypes.c_size_t, _P, ctypes.c_size_t, _P])
        L.prism_backward_train.argtypes = ([ctypes.POINTER(Desc)] + [_P] * 12 + [_P, ctypes.c_size_t]
                                           + [_P] * 13 + [_P, ctypes.c_size_t, _P])
        L.prism_step_workspace.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(ctypes.c_size_t)]
        L.prism_step.argtypes = [ctypes.POINTER(Desc)] + [_P] * 12 + [_P, ctypes.c_size_t, _P]
        L.prism_step_noalloc.argtypes = [ctypes.POINTER(Desc)] + [_P] * 12 + [_P]
        for f in ("prism_forward_workspace", "prism_backward_workspace",
                  "prism_forward_train_workspace", "prism_backward_train_workspace", "prism_forward",
                  "prism_backward", "prism_saved_bytes", "prism_forward_train",
                  "prism_backward_train", "prism_step_workspace", "prism_step",
                  "prism_step_noalloc"):
            getattr(L, f).restype = ctypes.c_int
        # (descriptors as bytes or structures)
        qd = ld = _P
        size = ctypes.c_size_t
        L.prism_qk_norm.argtypes = [qd] + [_P] * 9
        L.prism_qk_norm_backward_workspace.argtypes = [qd, ctypes.c_int, ctypes.POINTER(size)]
        L.prism_qk_norm_backward.argtypes = [qd] + [_P] * 13 + [size, _P]
        for query in (L.prism_linear_attention_workspace,
                      L.prism_linear_attention_packed_workspace):
            query.argtypes = [ld, ctypes.c_int, ctypes.c_int, ctypes.POINTER(size)]
        L.prism_linear_attention.argtypes = [ld] + [_P] * 9 + [size, _P]
        L.prism_linear_attention_backward.argtypes = [ld] + [_P] * 14 + [size, _P]
        L.prism_linear_attention_step.argtypes = [ld] + [_P] * 8
        out_size = ctypes.POINTER(size)
        L.prism_layer_norm.argtypes = [_P] * 8
        L.prism_layer_norm_backward_workspace.argtypes = [_P, ctypes.c_int, out_size]
        L.prism_layer_norm_backward.argtypes = [_P] * 9 + [size, _P]
        L.prism_short_conv.argtypes = [_P] * 9
        L.prism_short_conv_backward_workspace.argtypes = [_P, ctypes.c_int, out_size]
        L.prism_short_conv_backward.argtypes = [_P] * 12 + [size, _P]
        L.prism_gated_recurrence_workspace.argtypes = [_P, ctypes.c_int, ctypes.c_int, out_size]
        L.prism_gated_recurrence.argtypes = [_P] * 10 + [size, _P]
        L.prism_gated_recurrence_backward.argtypes = [_P] * 16 + [size, _P]
        L.prism_gated_recurrence_step.argtypes = [_P] * 9
        for f in EXPORTS[EXPORTS.index("prism_qk_norm"):]:
            getattr(L, f).restype = ctypes.c_int
        L.prism_status_string.argtypes = [ctypes.c_int]
        L.prism_status_string.restype = ctypes.c_char_p
        L.prism_last_error.restype = ctypes.c_char_p
        L.prism_timing_end.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_int), ctypes.c_int]
        L.prism_timing_end.restype = ctypes.c_int
        _lib = L
    return _lib


ACTIVATIONS = {"gelu": 0, "identity": 1}


def make_desc(B, T, H, dk, dv, L, chunk, dtype, conv_width=4, activation="gelu", conv_offset=0,
              packed_tokens=0):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    return Desc(B, T, H, dk, dv, L, chunk, conv_width, dtype, ACTIVATIONS[activation],
                int(conv_offset), int(packed_tokens))


def _check(status):
    if status != 0:
        msg = lib().prism_last_error().decode()
        raise RuntimeError(f"{STATUS.get(status, status)}: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return PRISM_BF16
    if t.dtype == torch.float32:
        return PRISM_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _req(t, name, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _desc_from(q, v, Wk, chunk, activation="gelu", conv_offset=0, cu_seqlens=None,
               max_seqlen=None):
    """Descriptor of a dense batch (q [B,T,H,dk]) or, with cu_seqlens, of a
    packed one (q [N,H,dk], B = len(cu_seqlens) - 1, T = max_seqlen, N rows)."""
    N = 0
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError(f"q: expected [B, T, H, dk], got shape {tuple(q.shape)}")
        B, T, H, dk = q.shape
    else:
        if max_seqlen is None:
            raise ValueError("max_seqlen is required with cu_seqlens")
        N, H, dk = q.shape
        B, T = cu_seqlens.numel() - 1, int(max_seqlen)
    dv = v.shape[-1]
    L = 0 if Wk is None else Wk.shape[1]
    return make_desc(B, T, H, dk, dv, L, chunk, _dtype_code(q), activation=activation,
                     conv_offset=conv_offset, packed_tokens=N)


def _shape(t, name, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_shapes(desc, packed, k, v, alpha, beta, Wk, Wp, wbeta, conv, S0, extra=(),
                  state_name="S0"):
    """Every tensor's shape against the descriptor, on the host, before the
    library sees a pointer: the C ABI cannot see shapes, and a wrong one
    would make the kernels read or write outside the tensor."""
    B, T, H, d, L = desc.B, desc.T, desc.H, desc.dk, desc.L
    tok = (desc.packed_tokens, H) if packed else (B, T, H)
    _shape(k, "k", tok + (d,))
    _shape(v, "v", tok + (d,))
    _shape(alpha, "alpha", tok)
    _shape(beta, "beta", tok)
    if L > 0:
        _shape(Wk, "Wk", (H, L, d, d))
        _shape(Wp, "Wp", (H, L, d, d))
        _shape(wbeta, "wbeta", (H, L, d))
        _shape(conv, "conv", (H, d, 4))
    _shape(S0, state_name, (B, H, d, d))
    for name, t, kind in extra:
        _shape(t, name, tok + (d,) if kind == "tok" else (B, H, d, d))


def _on_gpu(q):
    if q.device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {q.device}")


def _req_cu(cu, q):
    if cu is None:
        return
    if cu.dtype != torch.int32 or cu.device != q.device or not cu.is_contiguous() or cu.dim() != 1:
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor on q's device")
    if q.dim() != 3:
        raise ValueError("with cu_seqlens, q, k, v are packed [N, H, d]")


def _workspace(nbytes, device):
    ws = torch.empty(max(int(nbytes), 256) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws, ws[off:]


def _given(t, name, like):
    """A buffer of the caller's, which the kernels write by its address and size:
    on the tensors' device and without gaps or repeats."""
    if t.device != like.device:
        raise ValueError(f"{name}: expected device {like.device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def forward_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(lib().prism_forward_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def backward_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(lib().prism_backward_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def forward_train_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(lib().prism_forward_train_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def backward_train_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(lib().prism_backward_train_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def saved_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(lib().prism_saved_bytes(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def _validate_inputs(q, k, v, alpha, beta, Wk, Wp, wbeta, conv, S0):
    dev, dt = q.device, q.dtype
    for name, t in (("q", q), ("k", k), ("v", v)):
        _req(t, name, dt, dev)
    for name, t in (("alpha", alpha), ("beta", beta)):
        _req(t, name, torch.float32, dev)
    if Wk is not None:
        for name, t in (("Wk", Wk), ("Wp", Wp), ("wbeta", wbeta), ("conv", conv)):
            if t is None:
                raise ValueError(f"{name} is required when Wk is given")
            _req(t, name, dt, dev)
    if S0 is not None:
        _req(S0, "S0", torch.float32, dev)


def _req_hist(h, name, q, v, B=None):
    B = v.shape[0] if B is None else B
    H = v.shape[-2]
    _req(h, name, q.dtype, q.device)
    if tuple(h.shape) != (B, 4, H, v.shape[-1]):
        raise ValueError(f"{name}: expected shape {(B, 4, H, v.shape[-1])}, got {tuple(h.shape)}")


def forward(q, k, v, alpha, beta, Wk=None, Wp=None, wbeta=None, conv=None, S0=None, chunk=64,
            workspace=None, saved=None, activation="gelu", conv_offset=0, conv_hist=None,
            conv_hist_out=None, cu_seqlens=None, max_seqlen=None):
    """PRISM layer forward.  Returns (o, S_T).

    q, k [B,T,H,dk], v [B,T,H,dv] (bf16 or fp32); alpha, beta [B,T,H] fp32;
    Wk [H,L,dk,dv], Wp [H,L,dv,dv], wbeta [H,L,dv], conv [H,dv,4] in q's
    dtype (all None for L = 0); S0 [B,H,dv,dk] fp32 or None.
    activation: "gelu" (delta = GELU(p r)) or "identity" (delta = p r);
    conv_offset: 0 (tap j on v_{t-j}) or 1 (tap j on v_{t-1-j}).
    conv_hist [B,4,H,dv] (v's dtype): the four values of v before the
    sequence (None: zeros); conv_hist_out (same shape, may be conv_hist)
    receives them for the next call.  cu_seqlens (int32 [B+1] on the device)
    with max_seqlen packs B sequences of different lengths: q, k, v are then
    [N, H, d], alpha, beta [N, H].
    With `saved` (a buffer from saved_buffer()) this is the training forward
    (prism_forward_train): the buffer then holds what backward(saved=...)
    needs.
    """
    _validate_inputs(q, k, v, alpha, beta, Wk, Wp, wbeta, conv, S0)
    _req_cu(cu_seqlens, q)
    desc = _desc_from(q, v, Wk, chunk, activation, conv_offset, cu_seqlens, max_seqlen)
    _check_shapes(desc, cu_seqlens is not None, k, v, alpha, beta, Wk, Wp, wbeta, conv, S0)
    B, H, dk, dv = desc.B, desc.H, desc.dk, desc.dv
    for name, h in (("conv_hist", conv_hist), ("conv_hist_out", conv_hist_out)):
        if h is not None:
            _req_hist(h, name, q, v, B)
    _on_gpu(q)
    o = torch.empty_like(v)
    ST = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
    need = forward_workspace_bytes(desc) if saved is None else forward_train_workspace_bytes(desc)
    if saved is not None:
        _given(saved, "saved", q)
    if workspace is None:
        _, ws = _workspace(need, q.device)
    else:
        _given(workspace, "workspace", q)
        ws = workspace
    stream = torch.cuda.current_stream(q.device).cuda_stream
    if saved is None:
        _check(lib().prism_forward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                   _ptr(beta), _ptr(Wk), _ptr(Wp), _ptr(wbeta), _ptr(conv),
                                   _ptr(S0), _ptr(conv_hist), _ptr(cu_seqlens), _ptr(o), _ptr(ST),
                                   _ptr(conv_hist_out), _ptr(ws), ctypes.c_size_t(ws.numel()),
                                   ctypes.c_void_p(stream)))
    else:
        _check(lib().prism_forward_train(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                         _ptr(beta), _ptr(Wk), _ptr(Wp), _ptr(wbeta), _ptr(conv),
                                         _ptr(S0), _ptr(conv_hist), _ptr(cu_seqlens), _ptr(o),
                                         _ptr(ST), _ptr(conv_hist_out), _ptr(saved),
                                         ctypes.c_size_t(saved.numel()), _ptr(ws),
                                         ctypes.c_size_t(ws.numel()), ctypes.c_void_p(stream)))
    return o, ST


def saved_buffer(q, v, Wk=None, chunk=64, cu_seqlens=None, max_seqlen=None):
    """A 256-byte aligned device buffer for the training pair (uint8 view);
    its size does not depend on the activation or the tap offset."""
    desc = _desc_from(q, v, Wk, chunk, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
    return _workspace(saved_bytes(desc), q.device)[1]


def backward(q, k, v, alpha, beta, Wk=None, Wp=None, wbeta=None, conv=None, S0=None, dO=None,
             dST=None, chunk=64, need_dS0=False, workspace=None, saved=None, activation="gelu",
             conv_offset=0, conv_hist=None, need_dconv_hist=False, cu_seqlens=None,
             max_seqlen=None):
    """Gradients of <dO, o> + <dST, S_T> with respect to every input.

    Returns a dict: dq, dk, dv (input dtype), dalpha, dbeta (fp32), and for
    L > 0 dWk, dWp, dwbeta, dconv (fp32); dS0 (fp32) when need_dS0.
    With `saved` (filled by forward(..., saved=...) on the same inputs) this is
    prism_backward_train, which skips the forward recompute.  activation,
    conv_offset and conv_hist as in forward() (and equal to the forward's
    with `saved`); need_dconv_hist adds dconv_hist [B,4,H,dv] fp32.
    cu_seqlens and max_seqlen as in forward().
    """
    _validate_inputs(q, k, v, alpha, beta, Wk, Wp, wbeta, conv, S0)
    if dO is None:
        raise ValueError("dO is required")
    _req(dO, "dO", q.dtype, q.device)
    _req_cu(cu_seqlens, q)
    desc = _desc_from(q, v, Wk, chunk, activation, conv_offset, cu_seqlens, max_seqlen)
    if dST is not None:
        _req(dST, "dST", torch.float32, q.device)
    _check_shapes(desc, cu_seqlens is not None, k, v, alpha, beta, Wk, Wp, wbeta, conv, S0,
                  extra=(("dO", dO, "tok"), ("dST", dST, "state")))
    B, H, dk, dv_ = desc.B, desc.H, desc.dk, desc.dv
    if conv_hist is not None:
        _req_hist(conv_hist, "conv_hist", q, v, B)
    _on_gpu(q)
    dev = q.device
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dalpha": torch.empty_like(alpha), "dbeta": torch.empty_like(beta)}
    if Wk is not None:
        g["dWk"] = torch.empty(Wk.shape, dtype=torch.float32, device=dev)
        g["dWp"] = torch.empty(Wp.shape, dtype=torch.float32, device=dev)
        g["dwbeta"] = torch.empty(wbeta.shape, dtype=torch.float32, device=dev)
        g["dconv"] = torch.empty(conv.shape, dtype=torch.float32, device=dev)
    if need_dS0:
        g["dS0"] = torch.empty((B, H, dv_, dk), dtype=torch.float32, device=dev)
    if need_dconv_hist:
        g["dconv_hist"] = torch.empty((B, 4, H, dv_), dtype=torch.float32, device=dev)
    need = backward_workspace_bytes(desc) if saved is None else backward_train_workspace_bytes(desc)
    if saved is not None:
        _given(saved, "saved", q)
    if workspace is None:
        _, ws = _workspace(need, dev)
    else:
        _given(workspace, "workspace", q)
        ws = workspace
    stream = torch.cuda.current_stream(dev).cuda_stream
    grads = (_ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dalpha"]), _ptr(g["dbeta"]),
             _ptr(g.get("dWk")), _ptr(g.get("dWp")), _ptr(g.get("dwbeta")), _ptr(g.get("dconv")),
             _ptr(g.get("dS0")), _ptr(g.get("dconv_hist")))
    inputs = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(Wk), _ptr(Wp),
              _ptr(wbeta), _ptr(conv), _ptr(S0), _ptr(conv_hist), _ptr(cu_seqlens))
    if saved is None:
        _check(lib().prism_backward(ctypes.byref(desc), *inputs, _ptr(dO), _ptr(dST), *grads,
                                    _ptr(ws), ctypes.c_size_t(ws.numel()), ctypes.c_void_p(stream)))
    else:
        _check(lib().prism_backward_train(ctypes.byref(desc), *inputs, _ptr(saved),
                                          ctypes.c_size_t(saved.numel()), _ptr(dO), _ptr(dST),
                                          *grads, _ptr(ws), ctypes.c_size_t(ws.numel()),
                                          ctypes.c_void_p(stream)))
    return g


def step_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(lib().prism_step_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def step(q, k, v, alpha, beta, Wk=None, Wp=None, wbeta=None, conv=None, S=None, conv_state=None,
         activation="gelu", conv_offset=0, workspace=None, noalloc=False):
    """Recurrent form (prism_step): the T tokens of each sequence in order,
    token by token.  S [B,H,dv,dk] fp32 is required and updated in place
    (S_0 in, S_T out); conv_state [B,4,H,dv] (v's dtype) likewise, or None
    for a zero history that is not kept.  Returns o [B,T,H,dv].  With T = 1
    this is one decode step.  noalloc=True calls prism_step_noalloc (the
    pairs go to the library's fixed device array; no workspace, nothing
    allocated but the output)."""
    _validate_inputs(q, k, v, alpha, beta, Wk, Wp, wbeta, conv, S)
    if S is None:
        raise ValueError("S is required")
    desc = _desc_from(q, v, Wk, 16, activation, conv_offset)
    _check_shapes(desc, False, k, v, alpha, beta, Wk, Wp, wbeta, conv, S, state_name="S")
    if conv_state is not None:
        _req_hist(conv_state, "conv_state", q, v)
    _on_gpu(q)
    o = torch.empty_like(v)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    if noalloc:
        _check(lib().prism_step_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                        _ptr(beta), _ptr(Wk), _ptr(Wp), _ptr(wbeta), _ptr(conv),
                                        _ptr(S), _ptr(conv_state), _ptr(o), ctypes.c_void_p(stream)))
        return o
    if workspace is None:
        _, workspace = _workspace(step_workspace_bytes(desc), q.device)
    else:
        _given(workspace, "workspace", q)
    _check(lib().prism_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                            _ptr(beta), _ptr(Wk), _ptr(Wp), _ptr(wbeta), _ptr(conv), _ptr(S),
                            _ptr(conv_state), _ptr(o), _ptr(workspace),
                            ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(stream)))
    return o


# --------------------------------------------------------------------------
# query / key normalisation with rotary positions
# --------------------------------------------------------------------------
NORMS = {"l2": 0, "rms": 1}


def rope_turns(rot, base=10000.0, inv_freq=None, device="cuda"):
    """Frequencies of a rotation of `rot` values as qk_norm takes them: an int64
    tensor [rot/2] of turns per position in units of 2^-64.  inv_freq (radians
    per position, a sequence or tensor of rot/2 numbers) replaces
    base^(-2i/rot)."""
    if inv_freq is None:
        inv_freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    freq = [float(f) for f in inv_freq]
    if len(freq) != rot // 2:
        raise ValueError(f"inv_freq: expected {rot // 2} numbers, got {len(freq)}")
    turns = [round(f / (2.0 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]
    return torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64,
                        device=device)


def _steps(t, name):
    """(batch, token, head) steps of a token tensor [B,T,H,d] or [N,H,d] whose
    last dimension is contiguous; 0 for a dimension of one entry."""
    s, n = t.stride(), t.shape
    if s[-1] != 1 and n[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if len(n) == 4:
        return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)
    return (0, s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0)


def _like(t, name, dtype, device, shape):
    """Type, device (a number, -1: host) and shape of a tensor."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected device {device}, got {t.get_device()}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _addr(t):
    return None if t is None else t.data_ptr()


# the descriptors' bytes (QkNormDesc, LinearAttentionDesc): one pack costs a
# fraction of filling the structures field by field, which shows in the calls
# for single tokens
_QK_DESC = struct.Struct("=9if18q")
_LA_DESC = struct.Struct("=7ifi4x15q")
assert _QK_DESC.size == ctypes.sizeof(QkNormDesc)
assert _LA_DESC.size == ctypes.sizeof(LinearAttentionDesc)
_NO_STEPS = (0, 0, 0)


def _qk_desc(q, k, wq, wk, positions, turns, norm, eps, interleaved):
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}, got {norm!r}")
    if q.dim() not in (3, 4):
        raise ValueError(f"q: expected [B, T, H, d] or [N, H, d], got shape {tuple(q.shape)}")
    code, dev, lead, d = _dtype_code(q), q.get_device(), q.shape[:-2], q.shape[-1]
    B, T = lead if len(lead) == 2 else (1, lead[0])
    Hk = 0
    if k is not None:
        if k.dim() != q.dim():
            raise ValueError(f"k: expected {q.dim()} dimensions, got shape {tuple(k.shape)}")
        Hk = k.shape[-2]
        _like(k, "k", q.dtype, dev, lead + (Hk, d))
    elif wk is not None:
        raise ValueError("wk without k")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            _like(w, name, q.dtype, dev, (d,))
            if not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    rot = 0
    if (positions is None) != (turns is None):
        raise ValueError("positions and turns go together")
    if positions is not None:
        _like(positions, "positions", torch.int32, dev, lead)
        if turns.dtype != torch.int64 or turns.get_device() != dev or turns.dim() != 1:
            raise ValueError("turns must be a 1-D int64 tensor on q's device")
        if not (positions.is_contiguous() and turns.is_contiguous()):
            raise ValueError("positions and turns must be contiguous")
        rot = 2 * turns.shape[0]
    return (B, T, q.shape[-2], Hk, d, rot, code, NORMS[norm], int(interleaved), eps,
            *_steps(q, "q"), *(_NO_STEPS if k is None else _steps(k, "k")))


def _out(t, out, name):
    if out is None:
        return t.new_empty(t.shape)
    _like(out, name, t.dtype, t.get_device(), t.shape)
    return out


# the current stream's handle without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def qk_norm(q, k=None, wq=None, wk=None, positions=None, turns=None, norm="l2", eps=1e-6,
            interleaved=False, q_out=None, k_out=None):
    """Queries and keys normalised for each head, weighted and rotated by
    position (prism_qk_norm).  Returns (q_out, k_out).

    q [B,T,Hq,d] (or [N,Hq,d]) and k [B,T,Hk,d] in bf16 or fp32, views of a
    fused projection allowed (contiguous last dimension); k may be None.
    norm: "l2" (x / |x|) or "rms" (x / root mean square); wq, wk [d] or None.
    positions (int32, [B,T] or [N]) with turns (rope_turns) rotates the first
    2 * len(turns) values of each head, in pairs (i, i + rot/2), or (2i, 2i+1)
    when interleaved.  q_out, k_out: where the results go (new contiguous
    tensors by default; q and k themselves: in place)."""
    desc = _qk_desc(q, k, wq, wk, positions, turns, norm, eps, interleaved)
    _on_gpu(q)
    q_out = _out(q, q_out, "q_out")
    ko = _NO_STEPS
    if k is not None:
        k_out = _out(k, k_out, "k_out")
        ko = _steps(k_out, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _check(lib().prism_qk_norm(
        _QK_DESC.pack(*desc, *_steps(q_out, "q_out"), *ko, 0, 0, 0, 0, 0, 0), _addr(q), _addr(k),
        _addr(wq), _addr(wk), _addr(positions), _addr(turns), _addr(q_out), _addr(k_out),
        _stream(q.device)))
    return q_out, k_out


# workspace bytes of the backward pass by descriptor
_qk_bytes = {}


def qk_norm_backward(q, k, dq_out, dk_out, wq=None, wk=None, positions=None, turns=None,
                     norm="l2", eps=1e-6, interleaved=False, dq=None, dk=None, workspace=None):
    """Gradients of <dq_out, q_out> + <dk_out, k_out> of qk_norm on the same
    inputs.  Returns a dict: dq, dk (input type; into dq, dk when given), and
    dwq, dwk (fp32 [d]) for the weights given."""
    desc = _qk_desc(q, k, wq, wk, positions, turns, norm, eps, interleaved)
    _like(dq_out, "dq_out", q.dtype, q.get_device(), q.shape)
    if k is not None:
        if dk_out is None:
            raise ValueError("dk_out is required with k")
        _like(dk_out, "dk_out", k.dtype, k.get_device(), k.shape)
    elif dk_out is not None or dk is not None:
        raise ValueError("dk_out or dk without k")
    steps = (*_steps(dq_out, "dq_out"), *(_NO_STEPS if k is None else _steps(dk_out, "dk_out")))
    _on_gpu(q)
    out = {"dq": _out(q, dq, "dq")}
    steps += _steps(out["dq"], "dq")
    if k is not None:
        out["dk"] = _out(k, dk, "dk")
        steps += _steps(out["dk"], "dk")
    else:
        steps += _NO_STEPS
    for name, w in (("dwq", wq), ("dwk", wk)):
        if w is not None:
            out[name] = w.new_empty(w.shape, dtype=torch.float32)
    packed = _QK_DESC.pack(*desc, *steps)
    if workspace is None and (wq is not None or wk is not None):
        size = _qk_bytes.get(packed)
        if size is None:
            n = ctypes.c_size_t(0)
            _check(lib().prism_qk_norm_backward_workspace(packed, 1, ctypes.byref(n)))
            if len(_qk_bytes) >= 4096:
                _qk_bytes.clear()
            size = _qk_bytes[packed] = n.value
        workspace = _workspace(size, q.device)[1]
    elif workspace is not None:
        _given(workspace, "workspace", q)
    _check(lib().prism_qk_norm_backward(
        packed, _addr(q), _addr(k), _addr(wq), _addr(wk), _addr(positions), _addr(turns),
        _addr(dq_out), _addr(dk_out), _addr(out["dq"]), _addr(out.get("dk")),
        _addr(out.get("dwq")), _addr(out.get("dwk")), _addr(workspace),
        0 if workspace is None else workspace.numel(), _stream(q.device)))
    return out


# --------------------------------------------------------------------------
# linear attention with a decay for each head
# --------------------------------------------------------------------------
def _la_desc(q, k, v, g, states, scale, cu_seqlens, max_seqlen):
    """Every operand's type, device and shape checked; the descriptor's fields
    up to the steps of v, the steps of g, and the shapes of a state and of o.
    q is [B,T,H,dk] or, packed, [N,H,dk]."""
    qs = q.shape
    code, dev, lead = _dtype_code(q), q.get_device(), qs[:-2]
    N = 0
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError(f"q: expected [B, T, H, dk], got shape {tuple(q.shape)}")
        B, T = lead
    else:
        if max_seqlen is None:
            raise ValueError("max_seqlen is required with cu_seqlens")
        _req_cu(cu_seqlens, q)
        B, T, N = cu_seqlens.numel() - 1, int(max_seqlen), lead[0]
    if k.dim() != q.dim() or v.dim() != q.dim():
        raise ValueError(f"k and v: expected {q.dim()} dimensions, got shapes {tuple(k.shape)}, "
                         f"{tuple(v.shape)}")
    H, dk, Hk, dv = qs[-2], qs[-1], k.shape[-2], v.shape[-1]
    _like(k, "k", q.dtype, dev, lead + (Hk, dk))
    _like(v, "v", q.dtype, dev, lead + (Hk, dv))
    if g.dim() == 1:
        _like(g, "g", torch.float32, dev, (H,))
        steps = (0, 0, 1)
    else:
        _like(g, "g", torch.float32, dev, lead + (H,))
        steps = (T * H if cu_seqlens is None else 0, H, 1)
    if not g.is_contiguous():
        raise ValueError("g must be contiguous")
    for name, S in states:
        if S is not None:
            _like(S, name, torch.float32, dev, (B, H, dv, dk))
            if not S.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    return ((B, T, H, Hk, dk, dv, code, scale, N, *_steps(q, "q"), *_steps(k, "k"), *_steps(v, "v")),
            steps, (B, H, dv, dk), lead + (H, dv))


# workspace bytes by descriptor, layout, pass and wish
_la_bytes = {}


def _la_workspace(desc, packed, backward, dg, device):
    key = (desc, packed, backward, dg)
    size = _la_bytes.get(key)
    if size is None:
        n = ctypes.c_size_t(0)
        query = (lib().prism_linear_attention_packed_workspace if packed
                 else lib().prism_linear_attention_workspace)
        _check(query(desc, backward, dg, ctypes.byref(n)))
        if len(_la_bytes) >= 4096:
            _la_bytes.clear()
        size = _la_bytes[key] = n.value
    return _workspace(size, device)[1] if size else None


def linear_attention(q, k, v, g, S0=None, scale=1.0, cu_seqlens=None, max_seqlen=None, o=None,
                     ST=None, workspace=None, need_state=True):
    """Linear attention with a decay for each head (prism_linear_attention):
    S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.  Returns (o, S_T),
    or (o, None) with need_state false: the last state is then neither kept to
    fp32 accuracy nor written.

    q [B,T,H,dk], k [B,T,Hk,dk], v [B,T,Hk,dv] in bf16 or fp32 (views of a
    fused projection allowed), H a multiple of Hk; dk, dv multiples of 16 up to
    128.  g fp32: [H], or [B,T,H] for a decay of each token.  S0 [B,H,dv,dk]
    fp32 or None.  cu_seqlens (int32 [B+1]) with max_seqlen packs sequences:
    token tensors [N,..], g [N,H] or [H].  o, ST: where the results go (new
    tensors by default; ST may be S0)."""
    if ST is not None and not need_state:
        raise ValueError("ST given, but need_state is false")
    desc, gs, state, shape = _la_desc(q, k, v, g, (("S0", S0), ("ST", ST)), scale, cu_seqlens,
                                      max_seqlen)
    _on_gpu(q)
    if o is None:
        o = q.new_empty(shape)
    else:
        _like(o, "o", q.dtype, q.get_device(), shape)
    if ST is None and need_state:
        ST = g.new_empty(state)
    packed = _LA_DESC.pack(*desc, *_steps(o, "o"), *gs)
    if workspace is None:
        workspace = _la_workspace(packed, cu_seqlens is not None, 0, 0, q.device)
    else:
        _given(workspace, "workspace", q)
    _check(lib().prism_linear_attention(
        packed, _addr(q), _addr(k), _addr(v), _addr(g), _addr(S0), _addr(cu_seqlens), _addr(o),
        _addr(ST), _addr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(q.device)))
    return o, ST


def linear_attention_backward(q, k, v, g, dO, S0=None, dST=None, scale=1.0, need_dS0=False,
                              need_dg=False, cu_seqlens=None, max_seqlen=None, workspace=None):
    """Gradients of <dO, o> + <dST, S_T> of linear_attention on the same
    inputs.  Returns a dict: dq, dk, dv (input type), dg (fp32, g's shape) when
    need_dg, dS0 (fp32) when need_dS0."""
    desc, gs, state, shape = _la_desc(q, k, v, g, (("S0", S0), ("dST", dST)), scale, cu_seqlens,
                                      max_seqlen)
    _like(dO, "dO", q.dtype, q.get_device(), shape)
    packed = _LA_DESC.pack(*desc, *_steps(dO, "dO"), *gs)
    _on_gpu(q)
    out = {n: t.new_empty(t.shape)
           for n, t in (("dq", q), ("dk", k), ("dv", v))}
    if need_dg:
        out["dg"] = g.new_empty(g.shape)
    if need_dS0:
        out["dS0"] = g.new_empty(state)
    if workspace is None:
        workspace = _la_workspace(packed, cu_seqlens is not None, 1, int(need_dg), q.device)
    else:
        _given(workspace, "workspace", q)
    _check(lib().prism_linear_attention_backward(
        packed, _addr(q), _addr(k), _addr(v), _addr(g), _addr(S0), _addr(cu_seqlens), _addr(dO),
        _addr(dST), _addr(out["dq"]), _addr(out["dk"]), _addr(out["dv"]), _addr(out.get("dg")),
        _addr(out.get("dS0")), _addr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(q.device)))
    return out


def linear_attention_step(q, k, v, g, S, S_out=None, scale=1.0, o=None):
    """The recurrence of linear_attention token by token over the T tokens of
    each sequence (prism_linear_attention_step); T = 1 is a decode step.  The
    state S [B,H,dv,dk] fp32 is read; S_T goes to S_out, or into S itself when
    S_out is None.  Returns o [B,T,H,dv]."""
    desc, gs, _, shape = _la_desc(q, k, v, g, (("S", S), ("S_out", S_out)), scale, None, None)
    _on_gpu(q)
    if o is None:
        o = q.new_empty(shape)
    else:
        _like(o, "o", q.dtype, q.get_device(), shape)
    _check(lib().prism_linear_attention_step(
        _LA_DESC.pack(*desc, *_steps(o, "o"), *gs), _addr(q), _addr(k), _addr(v), _addr(g),
        _addr(S), _addr(S if S_out is None else S_out), _addr(o), _stream(q.device)))
    return o


# --------------------------------------------------------------------------
# layer norm, short convolution, gated recurrence
# --------------------------------------------------------------------------
LAYER_NORMS = {"rms": 1, "layer": 2}
CONV_ACTIVATIONS = {"identity": 1, "silu": 2}
GATES = {"log": 0, "sigmoid": 1, "power": 2}

_LN_DESC = struct.Struct("=6if4x12q")
_SC_DESC = struct.Struct("=7i4x9q")
_GR_DESC = struct.Struct("=6i24q")
assert _LN_DESC.size == ctypes.sizeof(LayerNormDesc)
assert _SC_DESC.size == ctypes.sizeof(ShortConvDesc)
assert _GR_DESC.size == ctypes.sizeof(GatedRecurrenceDesc)
# workspace bytes of the backward passes and of the recurrence by descriptor
_block_bytes = {}


def _block_workspace(query, desc, args, like):
    key = (query, desc, args)
    size = _block_bytes.get(key)
    if size is None:
        n = ctypes.c_size_t(0)
        _check(getattr(lib(), query)(desc, *args, ctypes.byref(n)))
        if len(_block_bytes) >= 4096:
            _block_bytes.clear()
        size = _block_bytes[key] = n.value
    if size == 0:
        return None
    workspace = like.new_empty(size, dtype=torch.uint8)
    # (the allocator's blocks start at multiples of 512 bytes)
    return workspace if workspace.data_ptr() % 256 == 0 else _workspace(size, like.device)[1]


# (by device number, without the device object)
def _stream_of(device):
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(entry, device, *args):
    """Calls a C entry with the device's stream, the tensors' device current (a
    default stream is the current device's)."""
    if device == _current_device():
        return _check(entry(*args, _stream_of(device)))
    with torch.cuda.device(device):
        return _check(entry(*args, _stream_of(device)))


def _size(workspace):
    return 0 if workspace is None else workspace.numel()


def _reach(t):
    """A tensor's first address and the one behind its last."""
    lo, size = t.data_ptr(), t.element_size()
    if t.is_contiguous():
        return lo, lo + size * t.numel()
    return lo, lo + size * (1 + sum([(n - 1) * s for n, s in zip(t.shape, t.stride())]))


class _Layout:
    """A tensor's addresses as numpy looks at them (which reads none of them)."""

    def __init__(self, t):
        size = t.element_size()
        self.__array_interface__ = {"version": 3, "shape": tuple(t.shape), "typestr": f"|V{size}",
                                    "strides": tuple([s * size for s in t.stride()]),
                                    "data": (t.data_ptr(), False)}


def _overlap(a, b):
    """Whether two tensors have an address in common (columns of one fused row, or
    parts of a longer sequence, have none though they lie between one another)."""
    (a0, a1), (b0, b1) = _reach(a), _reach(b)
    if a1 <= b0 or b1 <= a0:
        return False
    import numpy
    try:
        return numpy.shares_memory(numpy.asarray(_Layout(a)), numpy.asarray(_Layout(b)), max_work=1 << 20)
    except RuntimeError:       # (too many strides to tell)
        return True


def _apart(out, name, *others):
    """A result has no address in common with the others."""
    lo, hi = _reach(out)
    for t in others:
        if t is not None and lo < hi and t.data_ptr() < hi and _overlap(out, t):
            raise ValueError(f"{name} must not share a buffer with another operand")


def _in_place(out, name, *others):
    """A result is in the very place of an operand, row by row, or apart from it."""
    for t in others:
        if t is None or t is out:
            continue
        if t.data_ptr() == out.data_ptr() and t.shape == out.shape and (
                t.stride() == out.stride()
                or all([n == 1 or a == b for n, a, b in zip(t.shape, t.stride(), out.stride())])):
            continue
        _apart(out, name, t)


def _vector(t, name, dtype, device, shape):
    """A small operand: type, device, shape, and contiguous."""
    _like(t, name, dtype, device, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _row_steps(t, name, flat):
    """Steps of rows [D], [N,D], [B,T,D] or [B,T,H,D] as (batch, token, head),
    dimensions of one entry 0; flat: those of a contiguous tensor."""
    if t.is_contiguous():
        return flat
    n, s = t.shape, t.stride()
    if s[-1] != 1 and n[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    steps = tuple([a if m > 1 else 0 for a, m in zip(s[:-1], n)])
    return (0, 0, 0)[len(steps):] + steps


def _norm_desc(x, norm, eps):
    """The descriptor's fields up to the steps of x, and the steps of a
    contiguous tensor of x's shape."""
    code = LAYER_NORMS.get(norm)
    if code is None:
        raise ValueError(f"norm must be one of {sorted(LAYER_NORMS)}, got {norm!r}")
    n = x.dim()
    if n == 3:
        T, H, D = x.shape
        B = 1
    elif 1 <= n <= 4:
        B, T, H, D = (1, 1, 1, 1)[n:] + tuple(x.shape)
    else:
        raise ValueError(f"x: expected 1 to 4 dimensions, got shape {tuple(x.shape)}")
    flat = (T * H * D, H * D, D)
    return (B, T, H, D, _dtype_code(x), code, eps, *_row_steps(x, "x", flat)), flat


def _weights(w, b, dt, dev, D):
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _vector(t, name, dt, dev, (D,))


def layer_norm(x, w=None, b=None, residual=None, norm="layer", eps=1e-5, y=None, h=None):
    """Rows normalised over the last dimension, with the residual sum in front
    (prism_layer_norm): s = x + residual, y = (s - mean) / deviation * w + b
    (norm "rms": by the root mean square alone).  Returns (y, h), h the sum, or
    None without a residual.

    x, residual [.., D] of one to four dimensions in bf16 or fp32 (contiguous
    last dimension, views allowed), w, b [D] or None.  y, h: where the results go
    (new contiguous tensors by default; each may be x or residual: in place)."""
    desc, flat = _norm_desc(x, norm, eps)
    dt, dev = x.dtype, x.get_device()
    _weights(w, b, dt, dev, desc[3])
    if y is not None:
        _in_place(y, "y", x, residual)
        _apart(y, "y", h, w, b)
    if h is not None:
        _in_place(h, "h", x, residual)
        _apart(h, "h", w, b)
    if dev < 0:
        _on_gpu(x)
    rs = hs = _NO_STEPS
    if residual is not None:
        _like(residual, "residual", dt, dev, x.shape)
        rs = _row_steps(residual, "residual", flat)
        if h is None:
            h, hs = x.new_empty(x.shape), flat
        else:
            hs = _row_steps(_out(x, h, "h"), "h", flat)
    elif h is not None:
        raise ValueError("h without residual")
    if y is None:
        y, ys = x.new_empty(x.shape), flat
    else:
        ys = _row_steps(_out(x, y, "y"), "y", flat)
    _launch((_lib or lib()).prism_layer_norm, dev,
        _LN_DESC.pack(*desc, *rs, *ys, *hs), x.data_ptr(), _addr(residual), _addr(w), _addr(b),
        y.data_ptr(), _addr(h))
    return y, h


def layer_norm_backward(x, dy, w=None, dh=None, norm="layer", eps=1e-5, need_db=False, dx=None,
                        workspace=None):
    """Gradients of <dy, y> + <dh, h> of layer_norm, from x, the rows that were
    normalised (the h that layer_norm returned where there was a residual).
    Returns a dict: dx (the gradient of x and of the residual alike; into dx when
    given, which may be dy, dh or x), dw (fp32 [D]) with w, db (fp32 [D]) when
    need_db."""
    desc, flat = _norm_desc(x, norm, eps)
    dt, dev = x.dtype, x.get_device()
    _like(dy, "dy", dt, dev, x.shape)
    hs = _NO_STEPS
    if dh is not None:
        _like(dh, "dh", dt, dev, x.shape)
        hs = _row_steps(dh, "dh", flat)
    _weights(w, None, dt, dev, desc[3])
    if dx is not None:
        _in_place(dx, "dx", x, dy, dh)
        _apart(dx, "dx", w)
    if workspace is not None:
        _given(workspace, "workspace", x)
    if dev < 0:
        _on_gpu(x)
    if dx is None:
        dx, xs = x.new_empty(x.shape), flat
    else:
        xs = _row_steps(_out(x, dx, "dx"), "dx", flat)
    out, dw, db = {"dx": dx}, None, None
    if w is not None:
        dw = out["dw"] = x.new_empty(x.shape[-1:], dtype=torch.float32)
    if need_db:
        db = out["db"] = x.new_empty(x.shape[-1:], dtype=torch.float32)
    packed = _LN_DESC.pack(*desc, *hs, *_row_steps(dy, "dy", flat), *xs)
    if workspace is None and len(out) > 1:
        workspace = _block_workspace("prism_layer_norm_backward_workspace", packed, (1,), x)
    _launch((_lib or lib()).prism_layer_norm_backward, dev,
        packed, x.data_ptr(), _addr(w), dy.data_ptr(), _addr(dh), dx.data_ptr(), _addr(dw),
        _addr(db), _addr(workspace), _size(workspace))
    return out


def _token_steps(t, name, flat):
    """Steps of [B,T,D] or, packed, [N,D] as (batch, token, 0); flat: those of a
    contiguous tensor."""
    if t.is_contiguous():
        return flat
    _, b, s = _row_steps(t, name, flat)
    return b, s, 0


def _batch(x, cu_seqlens):
    """B, T, D, rows of a packed batch, of x [B,T,D] or [N,D] with cu_seqlens, and
    the steps of a contiguous tensor of x's shape."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"x: expected [B, T, D], got shape {tuple(x.shape)}")
        B, T, D = x.shape
        return B, T, D, 0, (T * D, D, 0)
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device or cu_seqlens.dim() != 1
            or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor of B + 1 entries on x's device")
    if x.dim() != 2:
        raise ValueError(f"x: expected [N, D] with cu_seqlens, got shape {tuple(x.shape)}")
    return cu_seqlens.numel() - 1, 0, x.shape[1], x.shape[0], (0, x.shape[1], 0)


def _conv_desc(x, w, b, hist, activation, cu_seqlens):
    """The descriptor's fields up to the steps of x, and the steps of a
    contiguous tensor of x's shape."""
    code = CONV_ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(CONV_ACTIVATIONS)}, got {activation!r}")
    B, T, D, N, flat = _batch(x, cu_seqlens)
    dt, dev = x.dtype, x.get_device()
    if w.dim() != 2:
        raise ValueError(f"w: expected [D, K], got shape {tuple(w.shape)}")
    K = w.shape[1]
    _vector(w, "w", dt, dev, (D, K))
    if b is not None:
        _vector(b, "b", dt, dev, (D,))
    if hist is not None:
        _vector(hist, "hist", dt, dev, (B, K - 1, D))
    return (B, T, D, K, _dtype_code(x), code, N, *_token_steps(x, "x", flat)), flat


def short_conv(x, w, b=None, hist=None, activation="identity", cu_seqlens=None, y=None,
               hist_out=None):
    """Depthwise causal convolution over the last K tokens (prism_short_conv):
    z_t = b + sum_j w[:, j] x_{t-j}, y = z, or z sigmoid(z) with "silu".  Returns
    y.

    x [B,T,D] in bf16 or fp32 (views of a fused projection allowed), w [D,K], K
    from 2 to 4, b [D] or None; hist [B,K-1,D], the tokens before the sequence,
    oldest first (None: zeros); hist_out (same shape, may be hist) receives the
    last ones for the next call.  cu_seqlens (int32 [B+1]) packs sequences: x is
    [N,D].  y: where the result goes (a new tensor by default)."""
    desc, flat = _conv_desc(x, w, b, hist, activation, cu_seqlens)
    dev, at, old, last = x.get_device(), x.data_ptr(), None, None
    if hist is not None:
        old = hist.data_ptr()
    if hist_out is not None:
        B, T, D, K, code, _, N, sb, st, _ = desc
        _vector(hist_out, "hist_out", x.dtype, dev, (B, K - 1, D))
        value, last = 2 if code == PRISM_BF16 else 4, hist_out.data_ptr()
        end = last + value * B * (K - 1) * D
        # (by the addresses that either reaches at most: what a call for single tokens
        # has time for)
        if old is not None and old != last and 2 * last - end < old < end:
            _apart(hist_out, "hist_out", hist)
        if at < end and last < at + value * ((B - 1) * sb + ((N or T) - 1) * st + D):
            _apart(hist_out, "hist_out", x)
    if y is not None:
        _apart(y, "y", x, w, b, hist, hist_out, cu_seqlens)
    if dev < 0:
        _on_gpu(x)
    if y is None:
        y, ys = x.new_empty(x.shape), flat
    else:
        ys = _token_steps(_out(x, y, "y"), "y", flat)
    _launch((_lib or lib()).prism_short_conv, dev,
        _SC_DESC.pack(*desc, *ys, 0, 0, 0), at, w.data_ptr(), _addr(b), old,
        _addr(cu_seqlens), y.data_ptr(), last)
    return y


def short_conv_backward(x, w, dy, b=None, hist=None, activation="identity", cu_seqlens=None,
                        need_dhist=False, dx=None, workspace=None):
    """Gradients of <dy, y> of short_conv on the same inputs.  Returns a dict: dx
    (into dx when given), dw (fp32 [D,K]), db (fp32 [D]) with b, dhist (fp32
    [B,K-1,D]) when need_dhist."""
    desc, flat = _conv_desc(x, w, b, hist, activation, cu_seqlens)
    dev = x.get_device()
    _like(dy, "dy", x.dtype, dev, x.shape)
    if dx is not None:
        _apart(dx, "dx", x, dy, w, b, hist, cu_seqlens)
    if workspace is not None:
        _given(workspace, "workspace", x)
    if dev < 0:
        _on_gpu(x)
    B, K, D = desc[0], desc[3], desc[2]
    f32 = torch.float32
    if dx is None:
        dx, xs = x.new_empty(x.shape), flat
    else:
        xs = _token_steps(_out(x, dx, "dx"), "dx", flat)
    dw, db, dhist = x.new_empty((D, K), dtype=f32), None, None
    out = {"dx": dx, "dw": dw}
    if b is not None:
        db = out["db"] = x.new_empty((D,), dtype=f32)
    if need_dhist:
        dhist = out["dhist"] = x.new_empty((B, K - 1, D), dtype=f32)
    packed = _SC_DESC.pack(*desc, *_token_steps(dy, "dy", flat), *xs)
    if workspace is None:
        workspace = _block_workspace("prism_short_conv_backward_workspace", packed,
                                     (int(cu_seqlens is not None),), x)
    _launch((_lib or lib()).prism_short_conv_backward, dev,
        packed, x.data_ptr(), w.data_ptr(), _addr(b), _addr(hist), _addr(cu_seqlens),
        dy.data_ptr(), dx.data_ptr(), dw.data_ptr(), _addr(db), _addr(dhist), _addr(workspace),
        _size(workspace))
    return out


def _rec_desc(x, f, i, lam, gate, states, cu_seqlens):
    """The descriptor's fields up to the steps of i, the shape of a state, and the
    steps of a contiguous tensor of x's shape."""
    code = GATES.get(gate)
    if code is None:
        raise ValueError(f"gate must be one of {sorted(GATES)}, got {gate!r}")
    B, T, D, N, flat = _batch(x, cu_seqlens)
    dt, dev = x.dtype, x.get_device()
    _like(f, "f", dt, dev, x.shape)
    si = _NO_STEPS
    if i is not None:
        _like(i, "i", dt, dev, x.shape)
        si = _token_steps(i, "i", flat)
    if (lam is not None) != (gate == "power"):
        raise ValueError('lam goes with the gate "power", and with it alone')
    if lam is not None:
        _vector(lam, "lam", torch.float32, dev, (D,))
    for name, t in states:
        if t is not None:
            _vector(t, name, torch.float32, dev, (B, D))
    return (B, T, D, _dtype_code(x), code, N, *_token_steps(x, "x", flat),
            *_token_steps(f, "f", flat), *si), (B, D), flat


_NO_GRADS = (0,) * 12


def gated_recurrence(x, f, i=None, lam=None, h0=None, gate="sigmoid", cu_seqlens=None, h=None,
                     hT=None, need_state=True, workspace=None):
    """h_t = a_t h_{t-1} + u_t channel by channel, with its gates
    (prism_gated_recurrence).  Returns (h, h_T), or (h, None) with need_state
    false.  With s = sigmoid(i), or 1 without i:

        "log"      a = exp(f),                u = s x
        "sigmoid"  a = sigmoid(f),            u = (1 - a) s x
        "power"    a = exp(-lam sigmoid(f)),  u = sqrt(1 - a^2) s x

    x, f, i [B,T,D] in bf16 or fp32 (views of a fused projection allowed), lam
    fp32 [D] >= 0; h0 fp32 [B,D] or None.  cu_seqlens (int32 [B+1]) packs
    sequences: token tensors [N,D].  h, hT: where the results go (new tensors by
    default; hT may be h0)."""
    if hT is not None and not need_state:
        raise ValueError("hT given, but need_state is false")
    desc, state, flat = _rec_desc(x, f, i, lam, gate, (("h0", h0), ("hT", hT)), cu_seqlens)
    dev = x.get_device()
    if h is not None:
        _apart(h, "h", x, f, i, lam, h0, hT, cu_seqlens)
    if hT is not None:
        _in_place(hT, "hT", h0)
        _apart(hT, "hT", x, f, i, lam, cu_seqlens)
    if workspace is not None:
        _given(workspace, "workspace", x)
    if dev < 0:
        _on_gpu(x)
    if h is None:
        h, hs = x.new_empty(x.shape), flat
    else:
        hs = _token_steps(_out(x, h, "h"), "h", flat)
    if hT is None and need_state:
        hT = x.new_empty(state, dtype=torch.float32)
    packed = _GR_DESC.pack(*desc, *hs, *_NO_GRADS)
    if workspace is None:
        workspace = _block_workspace("prism_gated_recurrence_workspace", packed,
                                     (int(cu_seqlens is not None), 0), x)
    _launch((_lib or lib()).prism_gated_recurrence, dev,
        packed, x.data_ptr(), f.data_ptr(), _addr(i), _addr(lam), _addr(h0), _addr(cu_seqlens),
        h.data_ptr(), _addr(hT), _addr(workspace), _size(workspace))
    return h, hT


def gated_recurrence_backward(x, f, h, dh, i=None, lam=None, h0=None, dhT=None, gate="sigmoid",
                              need_dh0=False, cu_seqlens=None, dx=None, df=None, di=None,
                              workspace=None):
    """Gradients of <dh, h> + <dhT, h_T> of gated_recurrence from its inputs and
    its output h.  Returns a dict: dx, df (input type; into dx, df when given), di
    with i, dlam (fp32 [D]) with lam, dh0 (fp32 [B,D]) when need_dh0."""
    desc, state, flat = _rec_desc(x, f, i, lam, gate, (("h0", h0), ("dhT", dhT)), cu_seqlens)
    dt, dev = x.dtype, x.get_device()
    _like(h, "h", dt, dev, x.shape)
    _like(dh, "dh", dt, dev, x.shape)
    if di is not None and i is None:
        raise ValueError("di without i")
    for name, t, others in (("dx", dx, (df, di)), ("df", df, (di,)), ("di", di, ())):
        if t is not None:
            _apart(t, name, x, f, i, h, dh, lam, h0, dhT, cu_seqlens, *others)
    if workspace is not None:
        _given(workspace, "workspace", x)
    if dev < 0:
        _on_gpu(x)
    def result(t, name):
        if t is None:
            return x.new_empty(x.shape), flat
        return t, _token_steps(_out(x, t, name), name, flat)

    dx, xs = result(dx, "dx")
    df, fs = result(df, "df")
    out, dis, dlam, dh0 = {"dx": dx, "df": df}, _NO_STEPS, None, None
    if i is not None:
        di, dis = result(di, "di")
        out["di"] = di
    if lam is not None:
        dlam = out["dlam"] = torch.empty_like(lam)
    if need_dh0:
        dh0 = out["dh0"] = x.new_empty(state, dtype=torch.float32)
    packed = _GR_DESC.pack(*desc, *_token_steps(h, "h", flat), *_token_steps(dh, "dh", flat), *xs,
                           *fs, *dis)
    if workspace is None:
        workspace = _block_workspace("prism_gated_recurrence_workspace", packed,
                                     (int(cu_seqlens is not None), 1), x)
    _launch((_lib or lib()).prism_gated_recurrence_backward, dev,
        packed, x.data_ptr(), f.data_ptr(), _addr(i), _addr(lam), _addr(h0), _addr(cu_seqlens),
        h.data_ptr(), dh.data_ptr(), _addr(dhT), dx.data_ptr(), df.data_ptr(), _addr(di),
        _addr(dlam), _addr(dh0), _addr(workspace), _size(workspace))
    return out


def gated_recurrence_step(x, f, state, i=None, lam=None, gate="sigmoid", state_out=None, h=None):
    """The T tokens of each sequence, x [B,T,D], one after another from `state`
    fp32 [B,D] (prism_gated_recurrence_step; T = 1: a decode step).  The state
    after them goes to state_out, or into state itself when that is None.
    Returns h."""
    desc, (B, D), flat = _rec_desc(x, f, i, lam, gate, (("state", state), ("state_out", state_out)), None)
    dev = x.get_device()
    if h is not None:
        _like(h, "h", x.dtype, dev, x.shape)
        _apart(h, "h", x, f, i, lam)
        # (one fp32 token's h is the state after it)
        _in_place(h[:, 0] if h.shape[1] == 1 else h, "h", state, state_out)
    at = to = state.data_ptr()
    if state_out is not None:
        to = state_out.data_ptr()
        if at != to and at - 4 * B * D < to < at + 4 * B * D:
            _apart(state_out, "state_out", state)
    if desc[3] != PRISM_BF16:          # (a state in the place of bf16 tokens is none)
        for t, k in ((x, 6), (f, 9), (i, 12)):
            if (t is not None and t.data_ptr() < to + 4 * B * D
                    and to < t.data_ptr() + 4 * ((B - 1) * desc[k] + (desc[1] - 1) * desc[k + 1] + D)):
                _apart(state if state_out is None else state_out, "the state", t)
    if dev < 0:
        _on_gpu(x)
    if h is None:
        h, hs = x.new_empty(x.shape), flat
    else:
        hs = _token_steps(_out(x, h, "h"), "h", flat)
    _launch((_lib or lib()).prism_gated_recurrence_step, dev,
        _GR_DESC.pack(*desc, *hs, *_NO_GRADS), x.data_ptr(), f.data_ptr(), _addr(i), _addr(lam),
        at, to, h.data_ptr())
    return h


class KernelTimer:
    """Context manager: event-measured duration of every library kernel
    launched inside the block (prism_timing_begin / prism_timing_end)."""

    def __enter__(self):
        lib().prism_timing_begin()
        self.result = {}
        return self

    def __exit__(self, *exc):
        cap = 64
        names = (ctypes.c_char_p * cap)()
        ms = (ctypes.c_double * cap)()
        cnt = (ctypes.c_int * cap)()
        n = lib().prism_timing_end(names, ms, cnt, cap)
        self.result = {names[i].decode(): (ms[i], cnt[i]) for i in range(min(n, cap))}
        return False
