"""Results whose own rows would overlap are refused by the C entries of layer_norm,
short_conv and gated_recurrence.  On the host; no kernel is launched (a call that is
accepted there fails at the launch)."""
import pytest

from tests.test_block_abi import E_SHAPE, FAKE, _err, _gr, _gr_bwd, _gr_step, _ln, _ln_bwd, _sc, _sc_bwd, _st, gr, ln, no_gpu, sc

HIP = 6


@no_gpu
@pytest.mark.parametrize("steps,ok", [
    ((768, 256, 64), True), ((64, 512, 128), True), ((128, 1024, 256), True), ((64, 128, 384), True),
    ((-768, 256, -64), True), ((1 << 39, 1 << 37, 64), True), ((1 << 39, 1 << 38, 64), False),
    ((768, 256, 63), False), ((768, 255, 64), False), ((767, 256, 64), False), ((768, 256, 1), False),
    ((768, 64, 64), False), ((256, 256, 64), False), ((-1, 256, 64), False), ((64, 256, 64), False)])
def test_layer_norm(steps, ok):
    for call, field in ((_ln, "sy"), (_ln, "sh"), (_ln_bwd, "sh")):
        status = call(ln(**{field: _st(*steps)}))
        assert status == (HIP if ok else E_SHAPE)
        assert ok or "several rows in one place" in _err()
    # operands may repeat rows; a dimension of one entry may have any step
    for field in ("sx", "sr"):
        assert _ln(ln(**{field: _st(*steps)})) == HIP
    assert _ln(ln(B=1, T=1, sy=_st(0, 1, 64))) == HIP
    assert _ln(ln(H=1, sy=_st(64, 128, 0))) == HIP


@no_gpu
@pytest.mark.parametrize("steps,ok", [((320, 64), True), ((64, 128), True), ((128, 256), True),
                                      ((320, 63), False), ((319, 64), False), ((64, 64), False), ((1, 64), False)])
def test_tokens(steps, ok):
    want = HIP if ok else E_SHAPE
    assert _sc(sc(sy=_st(*steps))) == want and _sc_bwd(sc(sdx=_st(*steps))) == want
    rec = lambda **k: gr(T=5, **k)
    assert _gr(rec(sh=_st(*steps))) == want and _gr_step(rec(sh=_st(*steps))) == want
    for n in ("dx", "df", "di"):
        assert _gr_bwd(rec(**{"s" + n: _st(*steps)})) == want
    # packed: the batch's step is not used
    assert _sc(sc(sy=_st(1, 64)), cu_seqlens=FAKE) == HIP
    assert _sc(sc(sy=_st(1, 63)), cu_seqlens=FAKE) == E_SHAPE
