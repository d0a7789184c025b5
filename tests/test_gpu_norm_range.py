"""layer_norm and its backward pass at both ends of their range without eps: rows of
deviations of 2^62 / sqrt(D) and of 2^-62, less 2^3 of room for the largest and the
smallest of normal values' rows.  Tolerances as in test_gpu_layer_norm.py."""
import pytest
import torch

from tests import block_oracle as O
from tests.test_gpu_layer_norm import BF, F, P, TOL, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("D", [16, 333, 2048, 16384])
@pytest.mark.parametrize("dt", [BF, F])
def test_both_ends_of_the_range(dt, D, norm):
    gen = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy, w = r(40, D), r(40, D).to(dt), (1 + 0.2 * r(D)).to(dt)
    print(f"\n[layer_norm range {dt} {D} {norm}]", flush=True)
    for scale in (2.0 ** 59 / D ** 0.5, 2.0 ** -59):
        s = (scale * x).to(dt)
        y, _ = P().layer_norm(s, w, norm=norm, eps=0.0)
        g = P().layer_norm_backward(s, dy, w, norm=norm, eps=0.0, need_db=True)
        assert O.rel2(_np(y), O.layer_norm(_np(s), _np(w), norm=norm, eps=0.0)[0]) < TOL[dt], scale
        want = O.layer_norm_backward(_np(s), _np(dy), _np(w), norm=norm, eps=0.0)
        assert O.rel2(_np(g["dx"]), want["dx"]) < TOL[dt], scale
        assert O.rel2(_np(g["dw"]), want["dw"]) < TOL[F] and O.rel2(_np(g["db"]), want["db"]) < TOL[F], scale
