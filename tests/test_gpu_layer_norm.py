"""layer_norm and its backward pass on the GPU against the float64 oracle.

Tolerances (2-norm of the error over 2-norm of the result).  U = 2^-24 is half a
step of fp32.
* fp32 results: a row's sums are chains of at most 16 values a lane, 6 steps over
  the lanes and 16 over the waves, each rounding at U of the sum so far, and a
  dozen roundings follow: below 64 U = 3.8e-6 of sums that do not cancel; 1e-5
  leaves room for means near zero.  Rows with a mean of m deviations: the mean is
  off by up to 40 U of itself, which is 40 m U of a deviation.
* weight gradients: sums of n terms of either sign, whose roundings are as random:
  sqrt(n) U of the sum's size, n <= 17000: 8e-6; 1e-5 with the terms' own.
* bf16 results: one rounding, at most 2^-8 of a value, beside the above.
"""
import numpy as np
import pytest
import torch

from tests import block_oracle as O

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8 + 1e-5, F: 1e-5}


def P():
    from linear_recurrent_sequence_shortconv_amd import prism
    return prism


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# dtype, leading shape, D, norm, w, b, residual
CASES = [
    (BF, (8, 5), 2048, "layer", True, True, True),
    (BF, (1,), 1, "layer", True, True, False),              # one value: y = b
    (BF, (3, 7), 8, "layer", True, True, True),
    (BF, (2, 9, 5), 48, "layer", True, True, False),        # rows of heads, six lanes a row
    (BF, (2, 3, 4), 128, "rms", True, False, True),
    (BF, (333,), 512, "layer", False, False, False),
    (BF, (70,), 520, "layer", True, True, True),            # a lane's second vector is off for most
    (BF, (5, 13), 333, "layer", True, True, True),          # odd width: single values
    (BF, (9,), 1000, "rms", True, True, True),
    (BF, (3,), 4096, "layer", True, True, True),            # several waves a row
    (BF, (2, 2), 16384, "layer", True, True, True),
    (BF, (2,), 16383, "layer", True, True, False),
    (BF, (4100,), 64, "layer", True, True, True),
    (F, (3, 333, 5), 48, "layer", True, True, True),
    (F, (17,), 2048, "rms", True, False, False),
    (F, (3, 2), 5, "layer", False, True, True),
    (F, (2, 3), 1023, "layer", True, True, True),
    (F, (3,), 8192, "layer", True, True, True),
    (F, (2,), 16384, "rms", True, True, True),
    (F, (16999,), 20, "layer", True, True, False),          # more rows than workgroups
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_forward_and_backward(case):
    dt, lead, D, norm, uw, ub, ur = case
    gen = _gen(D + len(lead))
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, res, dy, dh = ((2 * r(*lead, D) + 0.5).to(dt) for _ in range(4))
    w = (1 + 0.2 * r(D)).to(dt) if uw else None
    b = r(D).to(dt) if ub else None
    res = res if ur else None
    dh = dh if ur else None
    print(f"\n[layer_norm {case}]", flush=True)
    y, h = P().layer_norm(x, w, b, residual=res, norm=norm)
    src = h if ur else x
    g = P().layer_norm_backward(src, dy, w, dh=dh, norm=norm, need_db=ub)
    torch.cuda.synchronize()
    want, s = O.layer_norm(_np(x), _np(w), _np(b), _np(res), norm)
    assert y.dtype == dt and y.shape == x.shape and O.rel2(_np(y), want) < TOL[dt]
    if ur:
        assert torch.equal(h, (x.float() + res.float()).to(dt))
    else:
        assert h is None
    gw = O.layer_norm_backward(_np(src), _np(dy), _np(w), _np(dh), norm)
    # (one value a row: the norm's own gradient is 0, of sums that cancel exactly)
    assert O.rel2(_np(g["dx"]), gw["dx"]) < TOL[dt] or (D == 1 and not np.any(_np(g["dx"]) - gw["dx"]))
    assert ("dw" in g) == uw and ("db" in g) == ub
    if uw:
        assert g["dw"].dtype == F and O.rel2(_np(g["dw"]), gw["dw"]) < TOL[F]
    if ub:
        assert O.rel2(_np(g["db"]), gw["db"]) < TOL[F]


def test_views_and_in_place():
    """Views of fused rows, heads-first tensors and results in place give bitwise
    what contiguous tensors give; what lies between the views stays."""
    gen = _gen(3)
    B, T, H, D = 2, 6, 3, 64
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)
    row, res, w = r(B, T, H + 1, D), r(B, T, H, D), r(D)
    keep = row.clone()
    x = row[:, :, :H]
    y, h = P().layer_norm(x, w, residual=res)
    yc, hc = P().layer_norm(x.contiguous(), w, residual=res)
    assert torch.equal(y, yc) and torch.equal(h, hc)
    hf = x.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(P().layer_norm(hf, w, residual=res)[0], y)
    odd = torch.empty(B, T, H, D + 1, device="cuda", dtype=BF)[..., 1:]      # rows at odd elements
    odd.copy_(x)
    yo = P().layer_norm(odd, w, residual=res)[0]
    assert O.rel2(_np(yo), _np(y)) < 2.0 ** -8                # (sums in another order)
    res2 = res.clone()
    y2, h2 = P().layer_norm(x, w, residual=res2, y=x, h=res2)
    assert y2.data_ptr() == x.data_ptr() and torch.equal(x, y) and torch.equal(res2, h)
    assert torch.equal(row[:, :, H], keep[:, :, H])
    dy, dh = r(B, T, H, D), r(B, T, H, D)
    g = P().layer_norm_backward(h, dy, w, dh=dh)
    into = torch.zeros(B, T, H + 1, D, device="cuda", dtype=BF)
    P().layer_norm_backward(h, dy, w, dh=dh, dx=into[:, :, :H])
    assert torch.equal(into[:, :, :H], g["dx"]) and not bool(into[:, :, H].any())
    P().layer_norm_backward(h, dy, w, dh=dh, dx=dy)
    assert torch.equal(dy, g["dx"])
    # one row for every token, broadcast: read as it is
    one = r(1, 1, H, D).expand(B, T, H, D)
    assert torch.equal(P().layer_norm(one, w)[0], P().layer_norm(one.contiguous(), w)[0])


@pytest.mark.parametrize("D", [64, 1000, 4096])
def test_rows_far_from_zero(D):
    gen = _gen(9)
    m = 1000.0
    x = torch.randn(40, D, generator=gen, device="cuda") + m
    dy = torch.randn(40, D, generator=gen, device="cuda")
    y, _ = P().layer_norm(x)
    g = P().layer_norm_backward(x, dy)
    assert O.rel2(_np(y), O.layer_norm(_np(x))[0]) < 1e-5 + 40 * m * 2.0 ** -24
    assert O.rel2(_np(g["dx"]), O.layer_norm_backward(_np(x), _np(dy))["dx"]) < 1e-5 + 40 * m * 2.0 ** -24


def test_values_out_of_the_ordinary():
    """Constant rows, tiny and large ones, and a row that is not finite, which
    stays by itself."""
    x = torch.zeros(6, 256, device="cuda")
    x[1] = 3.0
    x[2] = torch.arange(256.0, device="cuda") * 1e-20
    x[3] = torch.arange(256.0, device="cuda") * 1e15
    x[4, 7] = float("nan")
    x[5] = torch.arange(256.0, device="cuda")
    y, _ = P().layer_norm(x)
    g = P().layer_norm_backward(x, torch.ones_like(x), need_db=True)
    want = O.layer_norm(_np(x))[0]
    for k in (0, 1):
        assert not bool(y[k].any())
    for k in (2, 3, 5):
        assert O.rel2(_np(y[k]), want[k]) < 1e-5
        assert bool(torch.isfinite(g["dx"][k]).all())
    assert bool(torch.isnan(y[4]).all()) and bool(torch.isfinite(y[5]).all())
    assert torch.equal(g["db"], torch.full((256,), 6.0, device="cuda"))


def test_no_rows():
    x = torch.empty(0, 5, 64, device="cuda", dtype=BF)
    w = torch.ones(64, device="cuda", dtype=BF)
    y, h = P().layer_norm(x, w, residual=x)
    assert y.shape == x.shape and h.shape == x.shape
    g = P().layer_norm_backward(x, x, w, need_db=True)
    assert not bool(g["dw"].any()) and not bool(g["db"].any())
