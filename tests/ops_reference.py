"""Plain float64 numpy forms of the sequence-block operators, written from
their formulas, for the tests."""

import math

import numpy as np


def logistic(a):
    with np.errstate(over="ignore"):
        return np.where(a >= 0, 1.0 / (1.0 + np.exp(-np.abs(a))),
                        np.exp(-np.abs(a)) / (1.0 + np.exp(-np.abs(a))))


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------

def scan(gx, h0, D, gate, lengths=None):
    """gx [T, N, D*G*H] -> y [T, N, D*H], hy [D, N, H], tape."""
    T, N, width = gx.shape
    G = 3 if gate else 2
    H = width // (D * G)
    g = gx.reshape(T, N, D, G, H)
    lens = np.full(N, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    y = np.zeros((T, N, D, H))
    hy = np.zeros((D, N, H))
    before = np.zeros((T, N, D, H))
    after = np.zeros((T, N, D, H))
    for d in range(D):
        for n in range(N):
            h = np.zeros(H) if h0 is None else h0[d, n].astype(np.float64).copy()
            steps = range(lens[n]) if d == 0 else range(lens[n] - 1, -1, -1)
            for t in steps:
                before[t, n, d] = h
                f = logistic(g[t, n, d, 0])
                i = logistic(-g[t, n, d, 0])
                h = f * h + i * g[t, n, d, 1]
                after[t, n, d] = h
                y[t, n, d] = h * logistic(g[t, n, d, 2]) if gate else h
            hy[d, n] = h
    return y.reshape(T, N, D * H), hy, (before, after, lens)


def scan_backward(gx, tape, dy, dhy, D, gate):
    before, after, lens = tape
    T, N, width = gx.shape
    G = 3 if gate else 2
    H = width // (D * G)
    g = gx.reshape(T, N, D, G, H)
    dyr = dy.reshape(T, N, D, H)
    dgx = np.zeros((T, N, D, G, H))
    dh0 = np.zeros((D, N, H))
    for d in range(D):
        for n in range(N):
            c = np.zeros(H) if dhy is None else dhy[d, n].astype(np.float64).copy()
            steps = range(lens[n] - 1, -1, -1) if d == 0 else range(lens[n])
            for t in steps:
                f, i = logistic(g[t, n, d, 0]), logistic(-g[t, n, d, 0])
                o = logistic(g[t, n, d, 2]) if gate else 1.0
                dh = o * dyr[t, n, d] + c
                dgx[t, n, d, 0] = dh * (before[t, n, d] - g[t, n, d, 1]) * f * i
                dgx[t, n, d, 1] = dh * i
                if gate:
                    dgx[t, n, d, 2] = (dyr[t, n, d] * after[t, n, d] * o *
                                       logistic(-g[t, n, d, 2]))
                c = f * dh
            dh0[d, n] = c
    return dgx.reshape(T, N, D * G * H), dh0


# ---------------------------------------------------------------------------
# gated feed-forward
# ---------------------------------------------------------------------------

C0, C1 = math.sqrt(2.0 / math.pi), 0.044715


def activation(g, act):
    """act(g) and act'(g)."""
    if act == "gelu":
        th = np.tanh(C0 * (g + C1 * g ** 3))
        return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th ** 2) * C0 * (1 + 3 * C1 * g ** 2)
    s = logistic(g)
    if act == "silu":
        return g * s, s + g * s * logistic(-g)
    assert act == "sigmoid"
    return s, s * logistic(-g)


def glu(x, W, act):
    F = W.shape[0] // 2
    g, u = x @ W[:F].T, x @ W[F:].T
    return activation(g, act)[0] * u


def glu_backward(x, W, dy, act):
    F = W.shape[0] // 2
    g, u = x @ W[:F].T, x @ W[F:].T
    v, dv = activation(g, act)
    dg, du = dy * u * dv, dy * v
    return dg @ W[:F] + du @ W[F:], np.concatenate([dg.T @ x, du.T @ x])


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------

def w4_weights(q, scales, zeros, K, group):
    """The weights that packed rows stand for: [R, K]."""
    k = np.arange(K)
    nib = (q[:, k // 2].astype(np.int64) >> (4 * (k % 2))) & 15
    z = 8 if zeros is None else zeros.astype(np.int64)[:, k // group]
    return (nib - z) * scales[:, k // group].astype(np.float64)
