"""float64 oracle of the query / key normalisation and of the linear attention.

The attention goes token by token through the recurrence and its hand-derived
adjoint, so it shares neither the chunked sums of the kernels nor a pairwise
form.  Test infrastructure only; pinned in test_operators_oracle.py.
"""
import numpy as np


def rel2(x, y):
    """2-norm of the difference over the 2-norm of y."""
    x, y = np.asarray(x, np.float64), np.asarray(y, np.float64)
    n = np.sqrt(np.sum(y * y))
    d = np.sqrt(np.sum((x - y) ** 2))
    return float(d / n) if n > 0 else float(d)


# ------------------------------------------------------------------ norm
def _turned(x, positions, turns, interleaved, sign):
    """First 2 len(turns) values of each row of x [.., H, d] turned in pairs."""
    half = len(turns)
    z = x.copy()
    if half == 0:
        return z
    # the phase mod one turn in integers, as Python has them
    ph = np.array([[((int(p) * int(f)) % (1 << 64)) / 2.0 ** 64 for f in turns]
                   for p in np.asarray(positions).ravel()])
    th = sign * 2.0 * np.pi * ph.reshape(np.shape(positions) + (1, half))
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z[..., a] = np.cos(th) * x[..., a] - np.sin(th) * x[..., b]
    z[..., b] = np.sin(th) * x[..., a] + np.cos(th) * x[..., b]
    return z


def norm_forward(x, w, positions, turns, norm, eps, interleaved):
    c = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    y = x / np.sqrt(c * np.sum(x * x, -1, keepdims=True) + eps)
    return _turned(y if w is None else y * w, positions, turns, interleaved, 1.0)


def norm_backward(x, w, dz, positions, turns, norm, eps, interleaved):
    c = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    r = 1.0 / np.sqrt(c * np.sum(x * x, -1, keepdims=True) + eps)
    dy = _turned(dz, positions, turns, interleaved, -1.0)
    dw = np.sum(dy * x * r, axis=tuple(range(x.ndim - 1)))
    h = dy if w is None else dy * w
    return r * h - c * r ** 3 * x * np.sum(x * h, -1, keepdims=True), dw


# ------------------------------------------------------------- attention
def _wide(x, H):
    return np.repeat(x, H // x.shape[-2], axis=-2)


def attend(q, k, v, g, S0=None, scale=1.0):
    """One sequence: q [T,H,dk], k [T,Hk,dk], v [T,Hk,dv], g [T,H] or [H],
    S0 [H,dv,dk].  Returns o [T,H,dv], S_T."""
    T, H, dk = q.shape
    k, v = _wide(k, H), _wide(v, H)
    g = np.broadcast_to(g, (T, H))
    S = np.zeros((H, v.shape[-1], dk)) if S0 is None else S0.astype(np.float64)
    o = np.zeros((T, H, v.shape[-1]))
    for t in range(T):
        S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
        o[t] = scale * np.einsum("hvk,hk->hv", S, q[t])
    return o, S


def attend_backward(q, k, v, g, dO, S0=None, dST=None, scale=1.0):
    """Gradients of <dO, o> + <dST, S_T>: dq, dk, dv, dg, dS0 (dg in g's shape)."""
    T, H, dk = q.shape
    Hk, dv = k.shape[1], v.shape[-1]
    kw, vw = _wide(k, H), _wide(v, H)
    gw = np.broadcast_to(g, (T, H))
    S = np.zeros((H, dv, dk)) if S0 is None else S0.astype(np.float64)
    states = [S]
    for t in range(T):
        S = np.exp(gw[t])[:, None, None] * S + vw[t][:, :, None] * kw[t][:, None, :]
        states.append(S)
    dS = np.zeros((H, dv, dk)) if dST is None else dST.astype(np.float64)
    dq, dkw, dvw = np.zeros(q.shape), np.zeros(kw.shape), np.zeros(vw.shape)
    dg = np.zeros((T, H))
    for t in range(T - 1, -1, -1):
        dq[t] = scale * np.einsum("hvk,hv->hk", states[t + 1], dO[t])
        dS = dS + scale * dO[t][:, :, None] * q[t][:, None, :]
        dkw[t] = np.einsum("hvk,hv->hk", dS, vw[t])
        dvw[t] = np.einsum("hvk,hk->hv", dS, kw[t])
        e = np.exp(gw[t])[:, None, None]
        dg[t] = np.sum(dS * e * states[t], axis=(1, 2))
        dS = e * dS
    dk_ = dkw.reshape(T, Hk, H // Hk, dk).sum(2)
    dv_ = dvw.reshape(T, Hk, H // Hk, dv).sum(2)
    return {"dq": dq, "dk": dk_, "dv": dv_, "dg": dg if np.ndim(g) == 2 else dg.sum(0), "dS0": dS}
