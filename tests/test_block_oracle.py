"""Pins of the float64 oracle of layer norm, short convolution and gated
recurrence: known cases, numpy's own convolution, and central differences of
every gradient."""
import numpy as np
import pytest

from tests import block_oracle as O

H = 1e-6


def _numeric(f, x):
    """Central differences of the scalar f at x."""
    g = np.zeros(x.shape)
    for k in np.ndindex(x.shape):
        y = x.copy()
        y[k] += H
        up = f(y)
        y[k] -= 2 * H
        g[k] = (up - f(y)) / (2 * H)
    return g


def _near(a, b):
    assert np.max(np.abs(a - b)) < 1e-7 * max(1.0, np.max(np.abs(b)))


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_layer_norm(norm):
    rng = np.random.default_rng(1)
    x, r, dy, dh = (rng.normal(size=(3, 7)) for _ in range(4))
    w, b = 1 + 0.2 * rng.normal(size=7), rng.normal(size=7)
    y, s = O.layer_norm(x, norm=norm, eps=0.0)
    if norm == "layer":
        _near(y.mean(-1), np.zeros(3))
    _near((y * y).mean(-1), np.ones(3))
    assert np.array_equal(s, x)
    loss = lambda x_, w_, b_: sum(np.sum(p * q) for p, q in zip(
        (dy, dh), O.layer_norm(x_, w_, b_, residual=r, norm=norm)))
    g = O.layer_norm_backward(x + r, dy, w, dh, norm=norm)
    _near(g["dx"], _numeric(lambda v: loss(v, w, b), x))
    _near(g["dw"], _numeric(lambda v: loss(x, v, b), w))
    _near(g["db"], _numeric(lambda v: loss(x, w, v), b))


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("activation", ["identity", "silu"])
def test_short_conv(K, activation):
    rng = np.random.default_rng(K)
    T, D = 6, 3
    x, dy = rng.normal(size=(T, D)), rng.normal(size=(T, D))
    w, b, hist = rng.normal(size=(D, K)), rng.normal(size=D), rng.normal(size=(K - 1, D))
    y, last = O.short_conv(x, w, b, hist)
    full = np.concatenate([hist, x])
    for c in range(D):
        _near(y[:, c], np.convolve(full[:, c], w[c])[K - 1:K - 1 + T] + b[c])
    _near(O.short_conv(x, w, b, hist, "silu")[0], y / (1 + np.exp(-y)))
    # a cut sequence, its second part continued
    for cut in range(T + 1):
        p, h = O.short_conv(x[:cut], w, b, hist, activation)
        q, h = O.short_conv(x[cut:], w, b, h, activation)
        assert np.array_equal(np.concatenate([p, q]), O.short_conv(x, w, b, hist, activation)[0])
        assert np.array_equal(h, last)
    loss = lambda x_, w_, b_, h_: np.sum(dy * O.short_conv(x_, w_, b_, h_, activation)[0])
    g = O.short_conv_backward(x, w, dy, b, hist, activation)
    _near(g["dx"], _numeric(lambda v: loss(v, w, b, hist), x))
    _near(g["dw"], _numeric(lambda v: loss(x, v, b, hist), w))
    _near(g["db"], _numeric(lambda v: loss(x, w, v, hist), b))
    _near(g["dhist"], _numeric(lambda v: loss(x, w, b, v), hist))


@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
@pytest.mark.parametrize("inp", [False, True])
def test_gated_recurrence(gate, inp):
    rng = np.random.default_rng(7)
    T, D = 5, 3
    x, f, dh = rng.normal(size=(T, D)), rng.normal(size=(T, D)), rng.normal(size=(T, D))
    i = rng.normal(size=(T, D)) if inp else None
    lam = rng.uniform(0.1, 1.0, size=D) if gate == "power" else None
    h0, dhT = rng.normal(size=D), rng.normal(size=D)
    h, hT = O.recur(x, f, i, lam, h0, gate)
    # the sum over all earlier tokens
    a, c = O.gates(f, lam, gate)
    u = c * x * (1 if i is None else 1 / (1 + np.exp(-i)))
    want = [np.prod(a[:t + 1], 0) * h0 + sum(np.prod(a[k + 1:t + 1], 0) * u[k] for k in range(t + 1))
            for t in range(T)]
    _near(h, np.array(want))
    assert np.array_equal(hT, h[-1])
    if gate == "sigmoid":
        _near(a + c, np.ones_like(a))
    if gate == "power":
        _near(a * a + c * c, np.ones_like(a))

    def loss(x_, f_, i_, lam_, h_):
        o, last = O.recur(x_, f_, i_, lam_, h_, gate)
        return np.sum(dh * o) + np.sum(dhT * last)

    g = O.recur_backward(x, f, dh, None, i, lam, h0, dhT, gate)
    _near(g["dx"], _numeric(lambda v: loss(v, f, i, lam, h0), x))
    _near(g["df"], _numeric(lambda v: loss(x, v, i, lam, h0), f))
    _near(g["dh0"], _numeric(lambda v: loss(x, f, i, lam, v), h0))
    if inp:
        _near(g["di"], _numeric(lambda v: loss(x, f, v, lam, h0), i))
    if gate == "power":
        _near(g["dlam"], _numeric(lambda v: loss(x, f, i, v, h0), lam))


def test_open_and_shut_gates():
    x = np.ones((2, 1))
    f = np.array([[-np.inf], [0.0]])
    h, _ = O.recur(x, f, h0=np.array([5.0]), gate="log")
    assert h[0, 0] == 1.0 and h[1, 0] == 2.0            # exp(-inf) forgets, exp(0) keeps
    with np.errstate(over="ignore"):
        a, c = O.gates(np.array([-800.0, 800.0]), None, "sigmoid")
    assert a[0] == 0 and c[0] == 1 and a[1] == 1 and c[1] == 0
    g = O.recur_backward(x, x, x, lam=np.zeros(1), gate="power")
    assert np.all(np.isfinite(g["df"])) and np.all(np.isfinite(g["dlam"]))
