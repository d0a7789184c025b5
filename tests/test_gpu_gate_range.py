"""gated_recurrence_backward with gates by power that are nearly shut: 1 - a^2, about
2 lam sigmoid(f), from its ordinary size down to where the product leaves fp32's
normal range (below 2^-126) and to 0.

Tolerances as in test_gpu_gated_recurrence.py, with a = 1 for the longest memory.
What nearly shut gates add to them: e^-f is off by its exponent's rounding, |f| U of
itself for |f| <= 100, 1e-5 of dlam's and df's terms, which both limits leave room
for (at T = 150 they are 2e-4 of bf16 and 7e-5 of fp32 inputs).  sigmoid(f) below
2^-126 (f < -87.3) may be taken as 0: of the norm over f from -100 to -40 that is
e^-23 at most."""
import pytest
import torch

from tests import block_oracle as O
from tests.test_gpu_gated_recurrence import BF, F, P, _np, draw, limits

pytestmark = pytest.mark.gpu
RATES = [0.0, 1e-39, 1e-38, 1e-30, 1e-4, 1e-3, 0.1]      # (the first two positive ones are subnormal)
EACH = 24                                                  # channels of each


def _case(dt, inp, low, high, seed, B=2, T=150):
    D = EACH * len(RATES)
    x = draw(dt, (B, T), D, B, "power", inp, True, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x["f"] = (low + (high - low) * torch.rand(B, T, D, generator=gen, device="cuda")).to(dt)
    x["lam"] = torch.tensor(RATES).repeat_interleave(EACH).cuda()
    assert float(x["lam"][EACH]) > 0
    return x


def _backward(x, h, **kw):
    return P().gated_recurrence_backward(x["x"], x["f"], h, x["dh"], i=x["i"], lam=x["lam"], h0=x["h0"],
                                         dhT=x["dhT"], gate="power", need_dh0=True, **kw)


@pytest.mark.parametrize("low,high", [(-100.0, -40.0), (-90.0, -80.0), (-100.0, 5.0)])
@pytest.mark.parametrize("inp", [True, False])
@pytest.mark.parametrize("dt", [BF, F])
def test_gradients_of_nearly_shut_gates(dt, inp, low, high):
    x = _case(dt, inp, low, high, 3)
    h, _ = P().gated_recurrence(x["x"], x["f"], i=x["i"], lam=x["lam"], h0=x["h0"], gate="power")
    g = _backward(x, h)
    for n, t in g.items():
        assert bool(torch.isfinite(t).all()), n
    B, T, D = x["x"].shape
    f32, own, diff = limits(x, "power", T, dt)
    w = [O.recur_backward(*(_np(x[n][b]) for n in ("x", "f", "dh")), _np(h[b]),
                          None if x["i"] is None else _np(x["i"][b]), _np(x["lam"]), _np(x["h0"][b]), _np(x["dhT"][b]),
                          "power") for b in range(B)]
    # sigmoid(f) of fp32's normal range; what lies below may be left out
    kept = _np(x["f"]) > -87.0
    for k, lam in enumerate(RATES):
        at = slice(k * EACH, (k + 1) * EACH)
        for b in range(B):
            for n, lim in (("dx", own), ("df", diff), ("di", own)):
                if n in g:
                    got, want = _np(g[n][b])[:, at] * kept[b][:, at], w[b][n][:, at] * kept[b][:, at]
                    assert O.rel2(got, want) < lim or not want.any() and not got.any(), (n, lam)
            assert O.rel2(_np(g["dh0"][b, at]), w[b]["dh0"][at]) < f32, lam
        if low < -88 and high < -70:      # (a sum of which parts may be left out)
            continue
        want = sum(v["dlam"][at] for v in w)
        assert O.rel2(_np(g["dlam"][at]), want) < 2 * f32 + 1e-5, lam


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dt", [BF, F])
def test_other_channels_stay_as_they_were(dt, packed):
    """Channels with ordinary gates are bitwise what they are without nearly shut ones
    beside them."""
    x = _case(dt, True, -100.0, -40.0, 5)
    ordinary = slice(4 * EACH, None)
    x["f"][..., ordinary] = torch.randn_like(x["f"][..., ordinary]) + 2
    y = {n: v.clone() for n, v in x.items()}
    y["f"][..., :4 * EACH] = 1.0
    y["lam"][:4 * EACH] = 0.05
    kw = {}
    if packed:
        kw["cu_seqlens"] = torch.tensor([0, 133, 300], dtype=torch.int32, device="cuda")
        for t in (x, y):
            t.update({n: t[n].flatten(0, 1) for n in ("x", "f", "i", "dh")})
    h = P().gated_recurrence(y["x"], y["f"], i=y["i"], lam=y["lam"], h0=y["h0"], gate="power", **kw)[0]
    a, b = _backward(x, h, **kw), _backward(y, h, **kw)
    for n in a:
        assert torch.equal(a[n][..., ordinary], b[n][..., ordinary]), n


@pytest.mark.parametrize("dt", [BF, F])
def test_views_and_odd_widths(dt):
    """Batch entries that do not follow one another, results into columns of one row,
    and a width of single channels: as contiguous tensors within a rounding each (strips
    take other paths), and what lies beside the results stays."""
    x = _case(dt, True, -100.0, -40.0, 7)
    B, T, D = x["x"].shape
    h = P().gated_recurrence(x["x"], x["f"], i=x["i"], lam=x["lam"], h0=x["h0"], gate="power")[0]
    want = _backward(x, h)
    tol = 2.0 ** -8 if dt == BF else 1e-6      # (fp32: 150 roundings of 2^-24 of a carried gradient at most)
    tol += 150 * 2.0 ** -24
    far = {n: torch.zeros(B, T + 3, D, device="cuda", dtype=dt) for n in ("x", "f", "i", "dh")}
    for n, t in far.items():
        t[:, :T] = x[n]
    into = torch.full((B, T + 3, 4, D), 7.0, device="cuda", dtype=dt)
    part = [into[:, :T, k] for k in range(3)]
    g = _backward({**x, **{n: t[:, :T] for n, t in far.items()}}, h, dx=part[0], df=part[1], di=part[2])
    assert bool((into[:, :, 3] == 7).all()) and bool((into[:, T:] == 7).all())
    odd = {n: None if t is None else t[..., :D - 1].contiguous() for n, t in x.items()}
    o = _backward(odd, h[..., :D - 1].contiguous())
    for n, t in want.items():
        for k in range(len(RATES)):
            at = slice(k * EACH, (k + 1) * EACH - 1)
            assert O.rel2(_np(g[n][..., at]), _np(t[..., at])) < tol or not bool(t[..., at].any()), (n, k)
            assert O.rel2(_np(o[n][..., at]), _np(t[..., at])) < tol or not bool(t[..., at].any()), (n, k)
