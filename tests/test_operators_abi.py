"""Refusals of the added operators, on the host: the C entries check every
argument before any HIP call, and the binding every shape, type and device
before a pointer leaves Python.  No kernel is launched."""
import ctypes

import pytest
import torch

from linear_recurrent_sequence_shortconv_amd import prism as P

OK, E_NULL, E_SHAPE, E_UNSUP, E_ALIGN, E_WS = 0, 1, 2, 3, 4, 5
FAKE = ctypes.c_void_p(0x10000)

# the C entries get fake device pointers here, which only a host without a GPU
# may be trusted with
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run on hosts without a GPU")


def _err():
    return P.lib().prism_last_error().decode()


def _st(b, t, h):
    return P.Strides(b, t, h)


def qk(**kw):
    d = dict(B=2, T=3, Hq=4, Hk=2, d=64, rot=64, dtype=P.PRISM_BF16, norm=0, interleaved=0, eps=1e-6)
    d.update({k: v for k, v in kw.items() if k in d})
    D = P.QkNormDesc(*d.values())
    for n in ("q", "k", "qo", "ko", "dq", "dk"):
        setattr(D, n, kw.get("s" + n, _st(768, 256, 64)))
    return D


def _fwd(D, **kw):
    names = ("q", "k", "wq", "wk", "positions", "turns", "qo", "ko")
    return P.lib().prism_qk_norm(ctypes.byref(D), *[kw.get(n, FAKE) for n in names], None)


def _bwd(D, ws=FAKE, nbytes=1 << 30, **kw):
    names = ("q", "k", "wq", "wk", "positions", "turns", "dqo", "dko", "dq", "dk", "dwq", "dwk")
    return P.lib().prism_qk_norm_backward(ctypes.byref(D), *[kw.get(n, FAKE) for n in names], ws, nbytes, None)


@no_gpu
@pytest.mark.parametrize("field,value,code", [
    ("B", -1, E_SHAPE), ("T", -1, E_SHAPE), ("Hq", 0, E_SHAPE), ("Hk", -1, E_SHAPE), ("d", 0, E_SHAPE),
    ("rot", 72, E_SHAPE), ("rot", -8, E_SHAPE), ("d", 68, E_UNSUP), ("d", 264, E_UNSUP), ("rot", 12, E_UNSUP),
    ("dtype", 5, E_UNSUP), ("norm", 2, E_UNSUP), ("eps", -1.0, E_SHAPE), ("eps", float("nan"), E_SHAPE),
    ("eps", float("inf"), E_SHAPE), ("Hq", (1 << 20) + 1, E_SHAPE)])
def test_qk_norm_descriptor(field, value, code):
    D = qk(**{field: value})
    assert _fwd(D) == code and _bwd(D) == code and _err()
    n = ctypes.c_size_t(5)
    assert P.lib().prism_qk_norm_backward_workspace(ctypes.byref(D), 1, ctypes.byref(n)) == code and n.value == 0


@no_gpu
def test_qk_norm_pointers_strides_workspace():
    L = P.lib()
    assert L.prism_qk_norm(None, *([None] * 8), None) == E_NULL
    for n in ("q", "k", "positions", "turns", "qo", "ko"):
        assert _fwd(qk(), **{n: None}) == E_NULL and n in _err(), n
    for n in ("q", "k", "wq", "qo"):
        assert _fwd(qk(), **{n: ctypes.c_void_p(0x10008)}) == E_ALIGN and n in _err()
    assert _fwd(qk(), turns=ctypes.c_void_p(0x10004)) == E_ALIGN
    assert _fwd(qk(), positions=ctypes.c_void_p(0x10002)) == E_ALIGN
    assert _fwd(qk(sq=_st(768, 254, 64))) == E_ALIGN and "q" in _err()
    assert _fwd(qk(sko=_st(1 << 41, 256, 64))) == E_SHAPE and "ko" in _err()
    for n in ("dqo", "dko", "dq", "dk", "dwq", "dwk"):
        assert _bwd(qk(), **{n: None}) == E_NULL and n in _err(), n
    need = ctypes.c_size_t(0)
    assert L.prism_qk_norm_backward_workspace(ctypes.byref(qk()), 1, ctypes.byref(need)) == OK and need.value > 0
    assert _bwd(qk(), nbytes=need.value - 1) == E_WS and str(need.value) in _err()
    assert _bwd(qk(), ws=None) == E_WS
    assert _bwd(qk(), ws=ctypes.c_void_p(0x10010)) == E_ALIGN
    none = ctypes.c_size_t(9)
    assert L.prism_qk_norm_backward_workspace(ctypes.byref(qk()), 0, ctypes.byref(none)) == OK and none.value == 0
    assert L.prism_qk_norm_backward_workspace(ctypes.byref(qk()), 1, None) == E_NULL
    # no tokens: nothing is read, so nothing is required
    assert _fwd(qk(B=0), q=None, k=None, qo=None, ko=None, positions=None, turns=None) == OK


def la(**kw):
    d = dict(B=2, T=100, H=4, Hk=2, dk=64, dv=32, dtype=P.PRISM_BF16, scale=1.0, packed_tokens=0)
    d.update({k: v for k, v in kw.items() if k in d})
    D = P.LinearAttentionDesc(*d.values())
    for n in ("q", "k", "v", "o", "g"):
        setattr(D, n, kw.get("s" + n, _st(25600, 256, 64)))
    return D


def _la(D, ws=FAKE, nbytes=1 << 40, **kw):
    names = ("q", "k", "v", "g", "S0", "cu_seqlens", "o", "ST")
    p = [kw.get(n, None if n == "cu_seqlens" else FAKE) for n in names]
    return P.lib().prism_linear_attention(ctypes.byref(D), *p, ws, nbytes, None)


def _la_bwd(D, ws=FAKE, nbytes=1 << 40, **kw):
    names = ("q", "k", "v", "g", "S0", "cu_seqlens", "dO", "dST", "dq", "dk", "dv", "dg", "dS0")
    own = {"cu_seqlens": None, "dS0": ctypes.c_void_p(0x30000)}
    p = [kw.get(n, own.get(n, FAKE)) for n in names]
    return P.lib().prism_linear_attention_backward(ctypes.byref(D), *p, ws, nbytes, None)


def _la_step(D, **kw):
    names = ("q", "k", "v", "g", "S", "S_out", "o")
    return P.lib().prism_linear_attention_step(ctypes.byref(D), *[kw.get(n, FAKE) for n in names], None)


@no_gpu
@pytest.mark.parametrize("field,value,code", [
    ("B", -1, E_SHAPE), ("T", -1, E_SHAPE), ("H", 0, E_SHAPE), ("Hk", 0, E_SHAPE), ("Hk", 3, E_SHAPE),
    ("T", (1 << 30) + 1, E_SHAPE), ("H", 1 << 17, E_SHAPE), ("dk", 8, E_UNSUP), ("dk", 144, E_UNSUP), ("dv", 40, E_UNSUP), ("dtype", 3, E_UNSUP),
    ("scale", float("inf"), E_SHAPE), ("scale", float("nan"), E_SHAPE), ("B", 1 << 23, E_SHAPE),
    ("sq", _st(25600, 252, 64), E_ALIGN), ("sv", _st(-8, 256, 64), E_SHAPE), ("so", _st(25600, 256, 12), E_ALIGN),
    ("sk", _st(0, (1 << 22) + 8, 0), E_SHAPE), ("sg", _st(-1, 4, 1), E_SHAPE)])
def test_linear_attention_descriptor(field, value, code):
    D = la(**{field: value})
    assert _la(D) == code and _la_bwd(D) == code and _la_step(D) == code and _err()
    n = ctypes.c_size_t(5)
    assert P.lib().prism_linear_attention_workspace(ctypes.byref(D), 1, 1, ctypes.byref(n)) == code and n.value == 0


@no_gpu
def test_linear_attention_pointers_and_workspace():
    L = P.lib()
    assert L.prism_linear_attention(None, *([None] * 8), None, 0, None) == E_NULL
    for n in ("q", "k", "v", "g", "o"):
        assert _la(la(), **{n: None}) == E_NULL and n in _err(), n
    for n in ("q", "k", "v", "g", "dO", "dq", "dk", "dv"):
        assert _la_bwd(la(), **{n: None}) == E_NULL and n in _err(), n
    for n in ("q", "S", "S_out", "o"):
        assert _la_step(la(), **{n: None}) == E_NULL and n in _err(), n
    for n in ("q", "S0", "o", "ST"):
        assert _la(la(), **{n: ctypes.c_void_p(0x10008)}) == E_ALIGN and n in _err()
    assert _la(la(), g=ctypes.c_void_p(0x10002)) == E_ALIGN
    other = ctypes.c_void_p(0x20000)   # (dS0 may not share a buffer with dST or S0)
    for n in ("dST", "S0"):
        assert _la_bwd(la(), **{"dST": other, "S0": other, "dS0": FAKE, n: FAKE}) == E_UNSUP and "dS0" in _err()
    assert _la_bwd(la(), dg=ctypes.c_void_p(0x10002)) == E_ALIGN
    assert _la(la(), cu_seqlens=ctypes.c_void_p(0x10002)) == E_ALIGN
    assert _la(la(packed_tokens=-1), cu_seqlens=FAKE) == E_SHAPE and "packed_tokens" in _err()
    n = ctypes.c_size_t(0)
    long = lambda: la(B=1, T=5000)   # (few heads, many tokens: cut into segments, whose states need room)
    for bwd, dg, call in ((0, 0, _la), (1, 1, _la_bwd)):
        assert L.prism_linear_attention_workspace(ctypes.byref(long()), bwd, dg, ctypes.byref(n)) == OK and n.value > 0
        assert call(long(), nbytes=n.value - 1) == E_WS and str(n.value) in _err()
        assert call(long(), ws=None) == E_WS and call(long(), ws=ctypes.c_void_p(0x10010)) == E_ALIGN
    assert L.prism_linear_attention_workspace(ctypes.byref(la()), 0, 0, None) == E_NULL
    # an empty batch asks for nothing
    assert _la(la(B=0), q=None, k=None, v=None, g=None, o=None, ST=None, S0=None, ws=None, nbytes=0) == OK


def test_workspace_covers_packed_and_dense_rows():
    """One query serves both layouts: more rows or more wishes, no less room."""
    def size(D, backward=True, dg=False):
        n = ctypes.c_size_t(0)
        assert P.lib().prism_linear_attention_workspace(ctypes.byref(D), int(backward), int(dg), ctypes.byref(n)) == OK
        return n.value

    assert size(la(packed_tokens=1000)) > size(la()) == size(la(packed_tokens=150))
    assert size(la(), True, True) > size(la(), True) > size(la(), False)


def _t(*s, dt=torch.bfloat16):
    return torch.zeros(*s, dtype=dt)


def test_binding_qk_norm():
    q, k = _t(2, 3, 4, 64), _t(2, 3, 2, 64)
    pos, turns = _t(2, 3, dt=torch.int32), P.rope_turns(64, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        P.qk_norm(q, k, positions=pos, turns=turns)
    for kw, what in (({"positions": pos}, "together"), ({"positions": pos[0], "turns": turns}, "positions"),
                     ({"positions": pos, "turns": turns.int()}, "turns"), ({"norm": "max"}, "norm"),
                     ({"wq": _t(32)}, "wq"), ({"positions": pos.t().contiguous().t(), "turns": turns}, "contiguous")):
        with pytest.raises(ValueError, match=what):
            P.qk_norm(q, k, **kw)
    with pytest.raises(ValueError, match="wk without k"):
        P.qk_norm(q, wk=_t(64))
    with pytest.raises(ValueError, match="k:"):
        P.qk_norm(q, _t(2, 4, 2, 64))
    with pytest.raises(TypeError):
        P.qk_norm(q, k.float())
    with pytest.raises(TypeError):
        P.qk_norm(q.half())
    with pytest.raises(ValueError, match="last dimension"):
        P.qk_norm(q.transpose(2, 3).contiguous().transpose(2, 3), k)
    with pytest.raises(ValueError, match="dq_out"):
        P.qk_norm_backward(q, k, q[:, :2], k)


def test_binding_linear_attention():
    q, k, v, g = _t(2, 5, 4, 64), _t(2, 5, 2, 64), _t(2, 5, 2, 32), _t(4, dt=torch.float32)
    with pytest.raises(ValueError, match="GPU"):
        P.linear_attention(q, k, v, g)
    S = _t(2, 4, 32, 64, dt=torch.float32)
    for args, kw, what in (((q, k, v, g[:3]), {}, "g"), ((q, k[:1], v, g), {}, "k"), ((q, k, v[:, :4], g), {}, "v"),
                           ((q[0], k[0], v[0], g), {}, "q"), ((q, k, v, g), {"S0": S[:1]}, "S0"),
                           ((q, k, v, g), {"S0": S.transpose(1, 2).contiguous().transpose(1, 2)}, "contiguous"),
                           ((q, k, v, _t(2, 5, 3, dt=torch.float32)), {}, "g"),
                           ((q[0], k[0], v[0], g), {"cu_seqlens": _t(3, dt=torch.int32)}, "max_seqlen"),
                           ((q, k, v, g), {"cu_seqlens": _t(3, dt=torch.int32), "max_seqlen": 5}, "packed")):
        with pytest.raises(ValueError, match=what):
            P.linear_attention(*args, **kw)
    with pytest.raises(TypeError):
        P.linear_attention(q, k, v.float(), g)
    with pytest.raises(TypeError):
        P.linear_attention(q, k, v, g.double())
    with pytest.raises(ValueError, match="dO"):
        P.linear_attention_backward(q, k, v, g, _t(2, 5, 4, 64))
    with pytest.raises(ValueError, match="S_out"):
        P.linear_attention_step(q, k, v, g, S=S, S_out=S[:1])


def test_turns():
    t = P.rope_turns(4, inv_freq=[2 * 3.141592653589793 * 0.75, 2 * 3.141592653589793 / 4], device="cpu")
    assert t.tolist() == [-(1 << 62), 1 << 62]     # three quarters of a turn: minus one quarter
    with pytest.raises(ValueError):
        P.rope_turns(8, inv_freq=[1.0], device="cpu")


@no_gpu
def test_decay_gradient_of_a_repeated_decay():
    # a value of g that serves several tokens, heads or sequences has no place of its own in dg
    for sg in (_st(0, 4, 1), _st(400, 0, 1), _st(400, 4, 0), _st(0, 0, 0)):
        assert _la_bwd(la(sg=sg)) == E_UNSUP and "dg" in _err(), sg
        # without dg the call is fine so far: it stops at the workspace
        assert _la_bwd(la(sg=sg), dg=None, ws=None) != E_UNSUP, sg
    # one sequence, one token, one head repeat nothing
    for kw in (dict(B=1, sg=_st(0, 4, 1)), dict(T=1, sg=_st(4, 0, 1))):
        assert _la_bwd(la(**kw), ws=None) != E_UNSUP, kw


@no_gpu
def test_heads_in_flight():
    # 2^21 heads of all sequences would pass a launch's threads
    D = la(B=1 << 19, H=4, Hk=4, dk=16, dv=16, T=1)
    assert _la_step(D) == E_SHAPE and _la(D) == E_SHAPE


@no_gpu
def test_packed_workspace_follows_the_rows():
    """The query for packed batches asks for what their rows need, whatever the
    longest length is, and what the call then requires."""
    def size(D, backward=True, dg=True):
        n = ctypes.c_size_t(0)
        assert P.lib().prism_linear_attention_packed_workspace(ctypes.byref(D), int(backward), int(dg),
                                                               ctypes.byref(n)) == OK, _err()
        return n.value

    B, H, N, d = 64, 16, 41984, 128
    D = la(B=B, T=16384, H=H, Hk=4, dk=d, dv=d, packed_tokens=N)
    # fp32 dk and dv of each query head; row dots and dg, nine floats; the last state
    need = N * H * (2 * d * 4 + 9 * 4) + B * H * d * d * 4
    assert need <= size(D) < need + 8 * 256
    assert size(D, True, False) < size(D)
    n = size(D)
    assert _la_bwd(D, nbytes=n - 1, cu_seqlens=FAKE) == E_WS and str(n) in _err()
    # a batch whose padded form would be too large
    D = la(B=4096, T=1 << 20, H=16, Hk=16, packed_tokens=1 << 20)
    assert P.lib().prism_linear_attention_workspace(ctypes.byref(D), 1, 0, ctypes.byref(ctypes.c_size_t(0))) == E_SHAPE
    assert size(D) > 0
    assert P.lib().prism_linear_attention_packed_workspace(ctypes.byref(la()), 1, 1, None) == E_NULL
    assert P.lib().prism_linear_attention_packed_workspace(ctypes.byref(la(packed_tokens=-1)), 1, 1,
                                                           ctypes.byref(ctypes.c_size_t(0))) == E_SHAPE


def test_binding_refuses_a_state_that_is_not_needed():
    q, k, v, g = _t(2, 5, 4, 64), _t(2, 5, 2, 64), _t(2, 5, 2, 32), _t(4, dt=torch.float32)
    with pytest.raises(ValueError, match="need_state"):
        P.linear_attention(q, k, v, g, ST=_t(2, 4, 32, 64, dt=torch.float32), need_state=False)
    with pytest.raises(ValueError, match="GPU"):
        P.linear_attention(q, k, v, g, need_state=False)


def test_binding_wants_key_gradients_with_keys():
    q, k = _t(2, 3, 4, 64), _t(2, 3, 2, 64)
    with pytest.raises(ValueError, match="dk_out is required with k"):
        P.qk_norm_backward(q, k, q, None)
    for kw in ({"dk_out": k}, {"dk_out": None, "dk": k}):
        with pytest.raises(ValueError, match="without k"):
            P.qk_norm_backward(q, None, q, **kw)
