"""layer_norm and short_conv on rows narrower than a vector, many of them, and
short_conv on as many tokens as it takes.

Tolerances as in test_gpu_layer_norm.py and test_gpu_short_conv.py: 1e-5 of fp32
results and of weight gradients, 2^-8 beside it of bf16 results.  Of one to three
values dx's own part may cancel to nothing; with dh of the size of 1 beside it, what
is left of a cancellation, r U of g, is 1e-6 of the whole over normal rows (r is at
most eps^-1/2 = 316, and 1 / r is spread like |x|).  A single value less its own mean
has r = 316 in every row: dy w less the mean of dy w, which is dy w rounded by U of
itself at most, leaves up to 316 U |dy w| there, beside the above."""
import numpy as np
import pytest
import torch

from tests import block_oracle as O
from tests.test_gpu_short_conv import BF, F, P, TOL, _compare, _draw, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("dt,D", [(BF, 1), (BF, 2), (BF, 3), (BF, 7), (F, 1), (F, 2), (F, 3)])
def test_norm_of_narrow_rows(dt, D, norm):
    gen = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)
    x, res, dy, dh = (r(5, 1013, D) for _ in range(4))
    w, b = r(D), r(D)
    print(f"\n[layer_norm narrow {dt} {D} {norm}]", flush=True)
    y, h = P().layer_norm(x, w, b, residual=res, norm=norm)
    g = P().layer_norm_backward(h, dy, w, dh=dh, norm=norm, need_db=True)
    assert torch.equal(h, (x.float() + res.float()).to(dt))
    # y is formed from the sum before it is rounded
    want = O.layer_norm(_np(x), _np(w), _np(b), _np(res), norm)[0]
    assert O.rel2(_np(y), want) < TOL[dt]
    gw = O.layer_norm_backward(_np(h), _np(dy), _np(w), _np(dh), norm)
    single = 0.0
    if D == 1 and norm == "layer":
        single = 1e-5 ** -0.5 * 2.0 ** -24 * np.linalg.norm(_np(dy) * _np(w)) / np.linalg.norm(gw["dx"])
    assert O.rel2(_np(g["dx"]), gw["dx"]) < TOL[dt] + single and O.rel2(_np(g["db"]), gw["db"]) < TOL[F]
    if D > 1 or norm == "rms":
        assert O.rel2(_np(g["dw"]), gw["dw"]) < TOL[F]
    else:                        # (a value less its own mean)
        assert not bool(g["dw"].any())


@pytest.mark.parametrize("act", ["identity", "silu"])
@pytest.mark.parametrize("dt,D,K", [(BF, 1, 4), (BF, 2, 3), (BF, 3, 4), (F, 1, 2), (F, 2, 4), (F, 3, 3)])
def test_convolution_of_few_channels(dt, D, K, act):
    B, T = 3, 777
    x = _draw(dt, (B, T), D, K, B, D, True, True)
    print(f"\n[short_conv narrow {dt} {D} {K} {act}]", flush=True)
    kw = dict(b=x["b"], hist=x["hist"], activation=act)
    out = torch.empty_like(x["hist"])
    y = P().short_conv(x["x"], x["w"], hist_out=out, **kw)
    g = P().short_conv_backward(x["x"], x["w"], x["dy"], need_dhist=True, **kw)
    _compare(x, list(range(B)), act, y, g, out, dt)
    lens = [400, 0, 1, 1500, 2, 3, 0, 425]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    p = _draw(dt, (cu[-1],), D, K, len(lens), D + 9, True, True)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kw = dict(b=p["b"], hist=p["hist"], activation=act, cu_seqlens=off)
    out = torch.empty_like(p["hist"])
    y = P().short_conv(p["x"], p["w"], hist_out=out, **kw)
    g = P().short_conv_backward(p["x"], p["w"], p["dy"], need_dhist=True, **kw)
    _compare(p, [slice(a, b) for a, b in zip(cu[:-1], cu[1:])], act, y, g, out, dt)


def test_convolution_of_the_most_tokens():
    """2^30 tokens of one channel: parts of the result bitwise what the same tokens
    give by themselves, and the sums over all of them."""
    B, T = 1 << 20, 1 << 10
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(B, T, 1, device="cuda", dtype=BF).normal_(generator=gen)
    w = torch.randn(1, 4, generator=gen, device="cuda").to(BF)
    print("\n[short_conv 2^30 tokens]", flush=True)
    y = P().short_conv(x, w, activation="silu")
    g = P().short_conv_backward(x, w, x, activation="silu")
    torch.cuda.synchronize()
    for at in (slice(0, 64), slice(B // 2 - 3, B // 2 + 61), slice(B - 64, B)):
        part = x[at].contiguous()
        assert torch.equal(y[at], P().short_conv(part, w, activation="silu"))
        assert torch.equal(g["dx"][at], P().short_conv_backward(part, w, part, activation="silu")["dx"])
    # dw of halves adds up (sums of 2^30 terms of x^2's size and of either sign; a term
    # enters 2^-24 of its wave's sum of some 10^2 terms, and partials 2^-24 of theirs)
    half = [P().short_conv_backward(x[k * B // 2:(k + 1) * B // 2], w, x[k * B // 2:(k + 1) * B // 2],
                                    activation="silu")["dw"].double() for k in range(2)]
    assert float((g["dw"].double() - half[0] - half[1]).norm() / g["dw"].double().norm()) < 1e-4
