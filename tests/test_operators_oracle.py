"""Pins of the float64 oracle of the added operators: closed forms, and every
gradient against central differences."""
import numpy as np
import pytest

from tests import operators_oracle as O


def _numeric(f, x, h=1e-6):
    """Central differences of the scalar f() with respect to array x (in place)."""
    out = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        down = f()
        x[i] = keep
        out[i] = (up - down) / (2 * h)
    return out


def _turns(half, base=100.0):
    return [round(base ** (-i / half) / (2 * np.pi) * 2.0 ** 64) for i in range(half)]


@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients(norm, interleaved):
    rng = np.random.default_rng(3)
    x, w, dz = rng.standard_normal((3, 2, 8)), 1 + 0.3 * rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    pos, turns = np.array([0, 5, 100]), _turns(3)
    f = lambda: np.sum(dz * O.norm_forward(x, w, pos, turns, norm, 1e-3, interleaved))
    dx, dw = O.norm_backward(x, w, dz, pos, turns, norm, 1e-3, interleaved)
    assert O.rel2(dx, _numeric(f, x)) < 1e-8
    assert O.rel2(dw, _numeric(f, w)) < 1e-8


def test_rotation_is_a_rotation():
    """Lengths are kept, position 0 is the identity, inner products depend on
    the difference of positions only, and far positions wrap exactly."""
    rng = np.random.default_rng(4)
    x, y = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    t = _turns(4)
    turned = lambda z, p: O._turned(z, np.array([p]), t, False, 1.0)
    assert np.allclose(turned(x, 0), x)
    assert np.allclose(np.linalg.norm(turned(x, 77)), np.linalg.norm(x))
    a = np.sum(turned(x, 3) * turned(y, 10))
    assert np.allclose(a, np.sum(turned(x, 2 ** 30 + 3) * turned(y, 2 ** 30 + 10)))
    quarter = O._turned(x, np.array([1]), [1 << 62] * 4, True, 1.0)
    assert np.allclose(quarter[..., 0::2], -x[..., 1::2]) and np.allclose(quarter[..., 1::2], x[..., 0::2])


@pytest.mark.parametrize("per_token", [False, True])
def test_attention_gradients(per_token):
    rng = np.random.default_rng(5)
    T, H, Hk, dk, dv = 5, 4, 2, 3, 2
    q, k, v = rng.standard_normal((T, H, dk)), rng.standard_normal((T, Hk, dk)), rng.standard_normal((T, Hk, dv))
    g = -rng.random((T, H)) if per_token else -rng.random(H)
    S0, dST = rng.standard_normal((H, dv, dk)), rng.standard_normal((H, dv, dk))
    dO = rng.standard_normal((T, H, dv))

    def f():
        o, S = O.attend(q, k, v, g, S0, 0.7)
        return np.sum(dO * o) + np.sum(dST * S)

    got = O.attend_backward(q, k, v, g, dO, S0, dST, 0.7)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dS0", S0)):
        assert O.rel2(got[name], _numeric(f, x)) < 1e-8, name


def test_attention_without_decay_is_a_masked_product():
    rng = np.random.default_rng(6)
    q, k, v = (rng.standard_normal((6, 1, 4)) for _ in range(3))
    o, S = O.attend(q, k, v, np.zeros(1))
    assert np.allclose(o[:, 0], np.tril(q[:, 0] @ k[:, 0].T) @ v[:, 0])
    assert np.allclose(S[0], v[:, 0].T @ k[:, 0])


def test_attention_forgets_all_behind_a_reset():
    rng = np.random.default_rng(7)
    q, k, v = (rng.standard_normal((6, 1, 4)) for _ in range(3))
    g = np.zeros((6, 1))
    g[3] = -np.inf
    o, S = O.attend(q, k, v, g, S0=rng.standard_normal((1, 4, 4)))
    o2, S2 = O.attend(q[3:], k[3:], v[3:], np.zeros((3, 1)))
    assert np.allclose(o[3:], o2) and np.allclose(S, S2)
