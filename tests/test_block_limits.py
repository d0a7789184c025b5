"""Sizes at the limits that the C entries of short_conv and gated_recurrence state:
just inside accepted, just outside refused.  On the host, by the workspace queries
and by calls that are refused."""
import ctypes

import pytest

from tests.test_block_abi import E_SHAPE, OK, P, _err, _gr_step, _sc, gr, no_gpu, sc


def _conv(packed=0, **kw):
    n = ctypes.c_size_t(0)
    return P.lib().prism_short_conv_backward_workspace(ctypes.byref(sc(**kw)), packed, ctypes.byref(n)), n.value


def _rec(packed=0, back=1, **kw):
    n = ctypes.c_size_t(0)
    return P.lib().prism_gated_recurrence_workspace(ctypes.byref(gr(**kw)), packed, back, ctypes.byref(n)), n.value


@pytest.mark.parametrize("B,T,D,ok", [
    (1 << 20, 1 << 10, 1, True), (1, 1 << 30, 4, True), (1, (1 << 30) + 1, 4, False), (2, (1 << 29) + 1, 1, False),
    (1 << 11, 1 << 10, 16384, True), (1 << 16, 1 << 14, 256, True), (1, 1, 1 << 22, True), (511, 4, 1 << 22, True),
    (512, 4, 1 << 22, False), ((1 << 23) - 1, 4, 1, True), (1 << 23, 4, 1, False), (1 << 22, 4, 257, False),
    ((1 << 22) - 1, 4, 257, True)])
def test_convolution(B, T, D, ok):
    assert _conv(B=B, T=T, D=D)[0] == (OK if ok else E_SHAPE)
    assert ok or _err()
    if not ok:
        assert _sc(sc(B=B, T=T, D=D)) == E_SHAPE
    if ok and B == 1:      # a packed batch of as many rows
        assert _conv(1, B=2, T=0, D=D, packed_tokens=T)[0] == OK


def test_convolution_partials_stay_small_beside_the_tokens():
    """Of wide and of narrow channels: at most 5 of every 64 values (K = 4)."""
    for B, T, D in ((1 << 11, 1 << 10, 16384), (1, 1 << 30, 256), (1, 1 << 20, 1 << 18)):
        status, bytes_ = _conv(B=B, T=T, D=D)
        assert status == OK and 0 < bytes_ <= 4 * 5 * B * T * D // 64


@pytest.mark.parametrize("B,T,D,ok", [
    (1, 1 << 28, 64, True), (1, (1 << 28) + 1, 64, False), (1, 1 << 28, 65, False), (1 << 10, 1 << 10, 16384, True),
    (1 << 10, (1 << 10) + 1, 16384, False), (1, 1 << 27, 128, True), (1, 64, 1 << 22, True), (64, 1, 1 << 22, True),
    (1, 64 * 64, 1 << 22, True), (1, 64 * 64 + 1, 1 << 22, False)])
def test_recurrence(B, T, D, ok):
    for back in (0, 1):
        assert _rec(0, back, B=B, T=T, D=D)[0] == (OK if ok else E_SHAPE)
        assert _rec(1, back, B=1, T=0, D=D, packed_tokens=B * T)[0] == (OK if ok else E_SHAPE)
    if not ok:
        assert "64" in _err()


@no_gpu
def test_step_beyond_the_limit():
    assert _gr_step(gr(B=1, T=(1 << 28) + 1, D=64)) == E_SHAPE
