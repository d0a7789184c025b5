"""prism_gated_recurrence_step with no tokens still passes its state on: what its
kernel reads is required then too.  On the host; no kernel is launched."""
import ctypes

from tests.test_block_abi import E_ALIGN, E_NULL, _err, _gr_step, gr, no_gpu


@no_gpu
def test_lam_is_required_without_tokens():
    for n in ("lam", "state", "state_out"):
        assert _gr_step(gr(T=0), **{n: None}) == E_NULL and n in _err()
    assert _gr_step(gr(T=0), lam=ctypes.c_void_p(0x10002)) == E_ALIGN and "lam" in _err()
    # no sequences: nothing is read
    none = {n: None for n in ("x", "f", "i", "lam", "state", "state_out", "h")}
    assert _gr_step(gr(B=0), **none) == 0
