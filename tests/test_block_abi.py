"""Refusals of layer_norm, short_conv and gated_recurrence, on the host: the C
entries check every argument before any HIP call, and the binding every shape,
type and device before a pointer leaves Python.  No kernel is launched."""
import ctypes

import pytest
import torch

from linear_recurrent_sequence_shortconv_amd import prism as P

OK, E_NULL, E_SHAPE, E_UNSUP, E_ALIGN, E_WS = 0, 1, 2, 3, 4, 5
FAKE = ctypes.c_void_p(0x10000)
NAN, INF = float("nan"), float("inf")

# the C entries get fake device pointers here, which only a host without a GPU
# may be trusted with
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run on hosts without a GPU")


def _err():
    return P.lib().prism_last_error().decode()


def _st(b, t, h=0):
    return P.Strides(b, t, h)


def _desc(cls, fields, strides, kw):
    D = cls(*{**fields, **{k: v for k, v in kw.items() if k in fields}}.values())
    for n, s in strides.items():
        setattr(D, n, kw.get("s" + n, s))
    return D


# ------------------------------------------------------------- layer norm
def ln(**kw):
    return _desc(P.LayerNormDesc, dict(B=2, T=3, H=4, D=64, dtype=P.PRISM_BF16, norm=2, eps=1e-5),
                 dict.fromkeys(("x", "r", "y", "h"), _st(768, 256, 64)), kw)


def _ln(D, **kw):
    names = ("x", "residual", "w", "b", "y", "h")
    return P.lib().prism_layer_norm(ctypes.byref(D), *[kw.get(n, FAKE) for n in names], None)


def _ln_bwd(D, ws=FAKE, nbytes=1 << 30, **kw):
    names = ("x", "w", "dy", "dh", "dx", "dw", "db")
    return P.lib().prism_layer_norm_backward(ctypes.byref(D), *[kw.get(n, FAKE) for n in names], ws, nbytes, None)


@no_gpu
@pytest.mark.parametrize("field,value,code", [
    ("B", -1, E_SHAPE), ("T", -1, E_SHAPE), ("H", -1, E_SHAPE), ("D", 0, E_SHAPE), ("D", -4, E_SHAPE),
    ("D", 16385, E_UNSUP), ("B", 1 << 30, E_SHAPE), ("dtype", 2, E_UNSUP), ("norm", 0, E_UNSUP), ("norm", 3, E_UNSUP),
    ("eps", -1.0, E_SHAPE), ("eps", NAN, E_SHAPE), ("eps", INF, E_SHAPE)])
def test_layer_norm_descriptor(field, value, code):
    D = ln(**{field: value})
    assert _ln(D) == code and _ln_bwd(D) == code and _err()
    n = ctypes.c_size_t(5)
    assert P.lib().prism_layer_norm_backward_workspace(ctypes.byref(D), 1, ctypes.byref(n)) == code and n.value == 0


@no_gpu
def test_layer_norm_pointers_strides_workspace():
    L = P.lib()
    assert L.prism_layer_norm(None, *([None] * 6), None) == E_NULL
    for n in ("x", "y", "residual"):
        assert _ln(ln(), **{n: None}) == E_NULL and n in _err()
    for n in ("x", "residual", "w", "b", "y", "h"):
        assert _ln(ln(), **{n: ctypes.c_void_p(0x10001)}) == E_ALIGN and n in _err()
        assert _ln(ln(dtype=P.PRISM_F32), **{n: ctypes.c_void_p(0x10002)}) == E_ALIGN
    for s, n in (("sx", "x"), ("sr", "residual"), ("sy", "y"), ("sh", "h")):
        assert _ln(ln(**{s: _st(1 << 40, 256, 64)})) == E_SHAPE and n in _err()
    assert _ln(ln(sy=_st(0, 256, 64))) == E_SHAPE and "y" in _err()
    assert _ln(ln(sh=_st(768, 0, 64))) == E_SHAPE and "h" in _err()
    for n in ("x", "dy", "dx"):
        assert _ln_bwd(ln(), **{n: None}) == E_NULL and n in _err()
    assert _ln_bwd(ln(), dw=ctypes.c_void_p(0x10002)) == E_ALIGN
    assert _ln_bwd(ln(sh=_st(768, 256, 0))) == E_SHAPE and "dx" in _err()
    need = ctypes.c_size_t(0)
    assert L.prism_layer_norm_backward_workspace(ctypes.byref(ln()), 1, ctypes.byref(need)) == OK and need.value > 0
    assert _ln_bwd(ln(), nbytes=need.value - 1) == E_WS and str(need.value) in _err()
    assert _ln_bwd(ln(), ws=None) == E_WS
    assert _ln_bwd(ln(), ws=ctypes.c_void_p(0x10010)) == E_ALIGN
    assert L.prism_layer_norm_backward_workspace(ctypes.byref(ln()), 0, ctypes.byref(need)) == OK and need.value == 0
    assert L.prism_layer_norm_backward_workspace(ctypes.byref(ln()), 1, None) == E_NULL
    # no rows: nothing is read, so nothing is required
    assert _ln(ln(B=0), x=None, y=None) == OK
    assert _ln_bwd(ln(H=0), x=None, dy=None, dx=None, dw=None, db=None, ws=None) == OK


# ------------------------------------------------------ short convolution
def sc(**kw):
    return _desc(P.ShortConvDesc, dict(B=2, T=5, D=64, K=4, dtype=P.PRISM_BF16, activation=2, packed_tokens=9),
                 dict.fromkeys(("x", "y", "dx"), _st(320, 64)), kw)


def _sc(D, **kw):
    names = ("x", "w", "b", "hist", "cu_seqlens", "y", "hist_out")
    p = [kw.get(n, None if n == "cu_seqlens" else FAKE) for n in names]
    return P.lib().prism_short_conv(ctypes.byref(D), *p, None)


def _sc_bwd(D, ws=FAKE, nbytes=1 << 30, **kw):
    names = ("x", "w", "b", "hist", "cu_seqlens", "dy", "dx", "dw", "db", "dhist")
    p = [kw.get(n, None if n == "cu_seqlens" else FAKE) for n in names]
    return P.lib().prism_short_conv_backward(ctypes.byref(D), *p, ws, nbytes, None)


BATCH = [("B", -1, E_SHAPE), ("T", -1, E_SHAPE), ("D", 0, E_SHAPE), ("D", (1 << 22) + 1, E_SHAPE), ("B", 1 << 28, E_SHAPE),
         ("T", 1 << 30, E_SHAPE), ("B", 1 << 23, E_SHAPE), ("dtype", 7, E_UNSUP)]


@no_gpu
@pytest.mark.parametrize("field,value,code", BATCH + [
    ("K", 1, E_UNSUP), ("K", 5, E_UNSUP), ("activation", 0, E_UNSUP), ("activation", 3, E_UNSUP)])
def test_short_conv_descriptor(field, value, code):
    D = sc(**{field: value})
    assert _sc(D) == code and _sc_bwd(D) == code and _err()
    n = ctypes.c_size_t(5)
    assert P.lib().prism_short_conv_backward_workspace(ctypes.byref(D), 0, ctypes.byref(n)) == code and n.value == 0


@no_gpu
def test_short_conv_pointers_strides_workspace():
    L = P.lib()
    assert L.prism_short_conv(None, *([None] * 7), None) == E_NULL
    for n in ("x", "w", "y"):
        assert _sc(sc(), **{n: None}) == E_NULL and n in _err()
    for n in ("x", "w", "b", "hist", "y", "hist_out"):
        assert _sc(sc(), **{n: ctypes.c_void_p(0x10001)}) == E_ALIGN and n in _err()
    assert _sc(sc(), cu_seqlens=ctypes.c_void_p(0x10002)) == E_ALIGN and "cu_seqlens" in _err()
    assert _sc(sc(packed_tokens=-1), cu_seqlens=FAKE) == E_SHAPE
    assert _sc(sc(sy=_st(320, 0))) == E_SHAPE and "y" in _err()
    assert _sc(sc(sy=_st(0, 64))) == E_SHAPE
    assert _sc(sc(sx=_st(320, -(1 << 40)))) == E_SHAPE and "x" in _err()
    for n in ("x", "w", "dy", "dx", "dw"):
        assert _sc_bwd(sc(), **{n: None}) == E_NULL and n in _err()
    assert _sc_bwd(sc(), db=ctypes.c_void_p(0x10002)) == E_ALIGN
    assert _sc_bwd(sc(sdx=_st(320, 0))) == E_SHAPE and "dx" in _err()
    for packed, cu in ((0, None), (1, FAKE)):
        need = ctypes.c_size_t(0)
        assert L.prism_short_conv_backward_workspace(ctypes.byref(sc()), packed, ctypes.byref(need)) == OK
        assert need.value > 0
        assert _sc_bwd(sc(), nbytes=need.value - 1, cu_seqlens=cu) == E_WS and str(need.value) in _err()
        assert _sc_bwd(sc(), ws=None, cu_seqlens=cu) == E_WS
        assert _sc_bwd(sc(), ws=ctypes.c_void_p(0x10010), cu_seqlens=cu) == E_ALIGN
    assert L.prism_short_conv_backward_workspace(ctypes.byref(sc()), 0, None) == E_NULL


# ------------------------------------------------------- gated recurrence
def gr(**kw):
    return _desc(P.GatedRecurrenceDesc, dict(B=2, T=500, D=64, dtype=P.PRISM_BF16, gate=2, packed_tokens=900),
                 dict.fromkeys(("x", "f", "i", "h", "dh", "dx", "df", "di"), _st(32000, 64)), kw)


def _gr(D, ws=FAKE, nbytes=1 << 30, **kw):
    names = ("x", "f", "i", "lam", "h0", "cu_seqlens", "h", "hT")
    p = [kw.get(n, None if n == "cu_seqlens" else FAKE) for n in names]
    return P.lib().prism_gated_recurrence(ctypes.byref(D), *p, ws, nbytes, None)


def _gr_bwd(D, ws=FAKE, nbytes=1 << 30, **kw):
    names = ("x", "f", "i", "lam", "h0", "cu_seqlens", "h", "dh", "dhT", "dx", "df", "di", "dlam", "dh0")
    own = {"cu_seqlens": None, "dh0": ctypes.c_void_p(0x30000)}
    p = [kw.get(n, own.get(n, FAKE)) for n in names]
    return P.lib().prism_gated_recurrence_backward(ctypes.byref(D), *p, ws, nbytes, None)


def _gr_step(D, **kw):
    names = ("x", "f", "i", "lam", "state", "state_out", "h")
    return P.lib().prism_gated_recurrence_step(ctypes.byref(D), *[kw.get(n, FAKE) for n in names], None)


@no_gpu
@pytest.mark.parametrize("field,value,code", BATCH + [("gate", 3, E_UNSUP), ("gate", -1, E_UNSUP)])
def test_gated_recurrence_descriptor(field, value, code):
    D = gr(**{field: value})
    assert _gr(D) == code and _gr_bwd(D) == code and _gr_step(D) == code and _err()
    for back in (0, 1):
        n = ctypes.c_size_t(5)
        assert P.lib().prism_gated_recurrence_workspace(ctypes.byref(D), 0, back, ctypes.byref(n)) == code
        assert n.value == 0


@no_gpu
def test_gated_recurrence_pointers_strides_workspace():
    L = P.lib()
    assert L.prism_gated_recurrence(None, *([None] * 8), None, 0, None) == E_NULL
    for n in ("x", "f", "lam", "h"):
        assert _gr(gr(), **{n: None}) == E_NULL and n in _err()
    for n in ("x", "f", "i", "h"):
        assert _gr(gr(), **{n: ctypes.c_void_p(0x10001)}) == E_ALIGN and n in _err()
    for n in ("lam", "h0", "hT", "cu_seqlens"):
        assert _gr(gr(), **{n: ctypes.c_void_p(0x10002)}) == E_ALIGN and n in _err()
    assert _gr(gr(gate=1)) == E_UNSUP and "lam" in _err()
    for n in ("x", "f", "i"):
        assert _gr(gr(**{"s" + n: _st(1 << 40, 64)})) == E_SHAPE and n in _err()
    assert _gr(gr(sh=_st(32000, 0))) == E_SHAPE and "h" in _err()
    for n in ("x", "f", "lam", "h", "dh", "dx", "df", "di", "dlam"):
        assert _gr_bwd(gr(), **{n: None}) == E_NULL and n in _err()
    for n in ("dx", "df", "di"):
        assert _gr_bwd(gr(**{"s" + n: _st(0, 64)})) == E_SHAPE and n in _err()
    for n in ("dhT", "dlam", "dh0"):
        assert _gr_bwd(gr(), **{n: ctypes.c_void_p(0x10002)}) == E_ALIGN and n in _err()
    for n in ("dhT", "h0"):
        assert _gr_bwd(gr(), **{n: FAKE, "dh0": FAKE}) == E_UNSUP and "dh0" in _err()
    for n in ("x", "f", "lam", "state", "state_out", "h"):
        assert _gr_step(gr(), **{n: None}) == E_NULL and n in _err()
    assert _gr_step(gr(sh=_st(0, 64))) == E_SHAPE
    for packed, cu in ((0, None), (1, FAKE)):
        for back, call in ((0, _gr), (1, _gr_bwd)):
            need = ctypes.c_size_t(0)
            assert L.prism_gated_recurrence_workspace(ctypes.byref(gr()), packed, back, ctypes.byref(need)) == OK
            if need.value:
                assert call(gr(), nbytes=need.value - 1, cu_seqlens=cu) == E_WS and str(need.value) in _err()
                assert call(gr(), ws=None, cu_seqlens=cu) == E_WS
                assert call(gr(), ws=ctypes.c_void_p(0x10010), cu_seqlens=cu) == E_ALIGN
    assert L.prism_gated_recurrence_workspace(ctypes.byref(gr()), 0, 0, None) == E_NULL


# ---------------------------------------------------------------- binding
def _refused(error, match, call, *args, **kw):
    with pytest.raises(error, match=match):
        call(*args, **kw)


def test_binding_layer_norm():
    x, w = torch.zeros(2, 3, 64), torch.ones(64)
    _refused(ValueError, "GPU", P.layer_norm, x, w)
    _refused(ValueError, "norm", P.layer_norm, x, norm="l2")
    _refused(ValueError, "dimensions", P.layer_norm, torch.zeros(1, 1, 1, 1, 8))
    _refused(TypeError, "dtype", P.layer_norm, x.half())
    _refused(ValueError, "last dimension", P.layer_norm, x.transpose(1, 2))
    _refused(ValueError, "w: expected shape", P.layer_norm, x, torch.ones(63))
    _refused(TypeError, "b: expected", P.layer_norm, x, w, w.bfloat16())
    _refused(ValueError, "w must be contiguous", P.layer_norm, x, torch.ones(128)[::2])
    _refused(ValueError, "dy: expected shape", P.layer_norm_backward, x, x[:1])
    _refused(TypeError, "dh: expected", P.layer_norm_backward, x, x, dh=x.bfloat16())


def test_binding_short_conv():
    x, w = torch.zeros(2, 5, 64), torch.zeros(64, 4)
    _refused(ValueError, "GPU", P.short_conv, x, w)
    _refused(ValueError, "activation", P.short_conv, x, w, activation="gelu")
    _refused(ValueError, "B, T, D", P.short_conv, x[0], w)
    _refused(ValueError, "w: expected", P.short_conv, x, w[:63])
    _refused(ValueError, "w: expected", P.short_conv, x, w[0])
    _refused(ValueError, "w must be contiguous", P.short_conv, x, torch.zeros(4, 64).t())
    _refused(ValueError, "hist: expected shape", P.short_conv, x, w, hist=torch.zeros(2, 4, 64))
    _refused(ValueError, "hist_out: expected shape", P.short_conv, x, w, hist_out=torch.zeros(1, 3, 64))
    _refused(TypeError, "b: expected", P.short_conv, x, w, b=torch.zeros(64, dtype=torch.bfloat16))
    cu = torch.zeros(3, dtype=torch.int32)
    _refused(ValueError, "N, D", P.short_conv, x, w, cu_seqlens=cu)
    _refused(ValueError, "cu_seqlens", P.short_conv, x[0], w, cu_seqlens=cu.long())
    _refused(ValueError, "cu_seqlens", P.short_conv, x[0], w, cu_seqlens=cu[:0])
    _refused(ValueError, "dy: expected shape", P.short_conv_backward, x, w, x[:1])


def test_binding_gated_recurrence():
    x, lam, h0 = torch.zeros(2, 5, 64), torch.ones(64), torch.zeros(2, 64)
    _refused(ValueError, "GPU", P.gated_recurrence, x, x)
    _refused(ValueError, "gate", P.gated_recurrence, x, x, gate="gelu")
    _refused(ValueError, "lam goes", P.gated_recurrence, x, x, gate="power")
    _refused(ValueError, "lam goes", P.gated_recurrence, x, x, lam=lam, gate="log")
    _refused(ValueError, "lam: expected shape", P.gated_recurrence, x, x, lam=lam[:3], gate="power")
    _refused(TypeError, "lam: expected", P.gated_recurrence, x, x, lam=lam.bfloat16(), gate="power")
    _refused(ValueError, "f: expected shape", P.gated_recurrence, x, x[:1])
    _refused(TypeError, "i: expected", P.gated_recurrence, x, x, i=x.bfloat16())
    _refused(ValueError, "h0: expected shape", P.gated_recurrence, x, x, h0=h0[:1])
    _refused(TypeError, "h0: expected", P.gated_recurrence, x, x, h0=h0.bfloat16())
    _refused(ValueError, "hT given", P.gated_recurrence, x, x, hT=h0, need_state=False)
    _refused(ValueError, "h: expected shape", P.gated_recurrence_backward, x, x, x[:1], x)
    _refused(ValueError, "dh: expected shape", P.gated_recurrence_backward, x, x, x, x[:1])
    _refused(ValueError, "di without i", P.gated_recurrence_backward, x, x, x, x, di=x)
    _refused(ValueError, "dhT: expected shape", P.gated_recurrence_backward, x, x, x, x, dhT=h0[:1])
    _refused(ValueError, "state: expected shape", P.gated_recurrence_step, x, x, h0[:1])
    _refused(ValueError, "state_out: expected shape", P.gated_recurrence_step, x, x, h0, state_out=h0[:1])


def test_binding_results_apart():
    """A result in the place of an operand that is still read is refused by name."""
    t = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)
    x, f, i, dh, h = (t(2, 3, 8) for _ in range(5))
    w, hist = t(8, 4), t(2, 3, 8)

    def refused(name, call, *a, **kw):
        with pytest.raises(ValueError, match=f"{name} must not share"):
            call(*a, **kw)

    out = t(2, 3, 8)
    refused("y", P.layer_norm, x, residual=f, y=out, h=out)
    refused("y", P.short_conv, x, w, y=x)
    refused("y", P.short_conv, x, w, hist=hist, y=hist)
    for other in (x, f):
        refused("dx", P.short_conv_backward, x, w, f, dx=other)
        refused("h", P.gated_recurrence, x, f, h=other)
    refused("h", P.gated_recurrence, x, f, i=i, h=i)
    refused("h", P.gated_recurrence_step, x, f, torch.zeros(2, 8), h=x)
    for other in (x, f, i, h, dh):
        for name in ("dx", "df", "di"):
            refused(name, P.gated_recurrence_backward, x, f, h, dh, i=i, **{name: other})
    refused("dx", P.gated_recurrence_backward, x, f, h, dh, i=i, dx=out, df=out)
    refused("df", P.gated_recurrence_backward, x, f, h, dh, i=i, df=out, di=out)
