"""float64 oracle of layer norm, short convolution and gated recurrence.

Rows one by one, the convolution and the recurrence token by token with
hand-derived adjoints, so nothing of the kernels' strips, tiles or scans is
shared.  Test infrastructure only; pinned in test_block_oracle.py.
"""
import numpy as np

from tests.operators_oracle import rel2  # noqa: F401


def sigma(z):
    return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


# ------------------------------------------------------------- layer norm
def _unit(s, norm, eps):
    m = s.mean(-1, keepdims=True) if norm == "layer" else np.zeros(s.shape[:-1] + (1,))
    r = 1.0 / np.sqrt(((s - m) ** 2).mean(-1, keepdims=True) + eps)
    return (s - m) * r, r


def layer_norm(x, w=None, b=None, residual=None, norm="layer", eps=1e-5):
    s = x if residual is None else x + residual
    y = _unit(s, norm, eps)[0]
    y = y if w is None else y * w
    return (y if b is None else y + b), s


def layer_norm_backward(x, dy, w=None, dh=None, norm="layer", eps=1e-5):
    u, r = _unit(x, norm, eps)
    g = dy if w is None else dy * w
    dx = g - u * (g * u).mean(-1, keepdims=True)
    if norm == "layer":
        dx = dx - g.mean(-1, keepdims=True)
    over = tuple(range(x.ndim - 1))
    return {"dx": r * dx + (0 if dh is None else dh), "dw": (dy * u).sum(over), "db": dy.sum(over)}


# ------------------------------------------------------ short convolution
def short_conv(x, w, b=None, hist=None, activation="identity"):
    """One sequence: x [T,D], w [D,K], hist [K-1,D].  Returns y and the last K - 1
    tokens."""
    T, D = x.shape
    K = w.shape[1]
    full = np.concatenate([np.zeros((K - 1, D)) if hist is None else hist, x])
    y = np.zeros((T, D))
    for t in range(T):
        z = np.zeros(D) if b is None else b.copy()
        for j in range(K):
            z = z + w[:, j] * full[K - 1 + t - j]
        y[t] = z * sigma(z) if activation == "silu" else z
    return y, full[T:]


def short_conv_backward(x, w, dy, b=None, hist=None, activation="identity"):
    T, D = x.shape
    K = w.shape[1]
    full = np.concatenate([np.zeros((K - 1, D)) if hist is None else hist, x])
    dfull, dw, db = np.zeros(full.shape), np.zeros(w.shape), np.zeros(D)
    for t in range(T):
        z = np.zeros(D) if b is None else b.copy()
        for j in range(K):
            z = z + w[:, j] * full[K - 1 + t - j]
        g = dy[t]
        if activation == "silu":
            g = g * sigma(z) * (1.0 + z * sigma(-z))
        for j in range(K):
            dfull[K - 1 + t - j] += w[:, j] * g
            dw[:, j] += g * full[K - 1 + t - j]
        db += g
    return {"dx": dfull[K - 1:], "dw": dw, "db": db, "dhist": dfull[:K - 1]}


# ------------------------------------------------------- gated recurrence
def gates(f, lam, gate):
    """a and c of u = c sigma(i) x."""
    if gate == "log":
        return np.exp(f), np.ones_like(f)
    if gate == "sigmoid":
        return sigma(f), sigma(-f)
    e = -lam * sigma(f)
    return np.exp(e), np.sqrt(-np.expm1(2.0 * e))


def recur(x, f, i=None, lam=None, h0=None, gate="sigmoid"):
    """One sequence: x, f, i [T,D], lam, h0 [D].  Returns h [T,D], h_T."""
    T, D = x.shape
    a, c = gates(f, lam, gate)
    u = c * x if i is None else c * x * sigma(i)
    h = np.zeros(D) if h0 is None else h0.astype(np.float64)
    out = np.zeros((T, D))
    for t in range(T):
        h = a[t] * h + u[t]
        out[t] = h
    return out, h


def recur_backward(x, f, dh, h=None, i=None, lam=None, h0=None, dhT=None, gate="sigmoid"):
    """Gradients of <dh, h> + <dhT, h_T>; h: the forward's output as it is read
    for h_{t-1} (None: the exact one)."""
    T, D = x.shape
    a, c = gates(f, lam, gate)
    s = np.ones_like(x) if i is None else sigma(i)
    first = np.zeros(D) if h0 is None else h0.astype(np.float64)
    if h is None:
        h = recur(x, f, i, lam, h0, gate)[0]
    before = np.concatenate([first[None], h])[:T]
    g = np.zeros((T, D))
    carry = np.zeros(D) if dhT is None else dhT.astype(np.float64)
    for t in range(T - 1, -1, -1):
        g[t] = dh[t] + carry
        carry = a[t] * g[t]
    out = {"dx": g * c * s, "di": g * c * x * s * (1.0 - s), "dh0": carry}
    p, q = sigma(f), sigma(-f)
    if gate == "log":
        out["df"] = g * before * a
    elif gate == "sigmoid":
        out["df"] = g * (before - s * x) * p * q
    else:
        # log a = -lam p; dc/dlog a = -a^2 / c (0 where c is)
        slope = np.divide(a * a, c, out=np.zeros_like(c), where=c > 0)
        d = g * (before * a - slope * s * x)
        out["df"] = -lam * d * p * q
        out["dlam"] = -(d * p).sum(0)
    return out
