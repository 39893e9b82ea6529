"""Plain float64 oracle of the layer's operators: linear attention with a decay for each head (token
by token from its recurrence, and its gradients from theirs) and the norm of query and key heads with
the position rotation. NumPy loops over time, no code shared with the GPU path.

Inputs are arrays of any float type; everything is computed in float64 and returned unrounded.
``*_size`` functions return, for each output entry, the sum of the absolute values of the terms that
make it up: rounding a term by a relative u moves the entry by at most u times that.
"""

from __future__ import annotations

import numpy as np

__all__ = ["linattn", "linattn_bwd", "linattn_size", "linattn_bwd_size", "linattn_step", "qknorm", "qknorm_bwd"]


def _f(x):
    return np.asarray(x, dtype=np.float64)


def _group(x, HV):
    return np.repeat(x, HV // x.shape[-2], axis=-2)


def linattn(q, k, v, log_decay, scale, init=None):
    """(o, final state) of one batch: q, k [B, T, H, Dk]; v [B, T, HV, Dv]; init [B, HV, Dk, Dv]."""
    v, a = _f(v), np.exp(_f(log_decay))[:, None, None]
    B, T, HV, Dv = v.shape
    q, k = _group(_f(q), HV), _group(_f(k), HV)
    S = np.zeros((B, HV, q.shape[-1], Dv)) if init is None else _f(init).copy()
    o = np.zeros((B, T, HV, Dv))
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * np.matmul(q[:, t, :, None, :], S)[:, :, 0]
    return o, S


def linattn_bwd(q, k, v, log_decay, scale, do, init=None, dfinal=None):
    """(dq, dk, dv, d_init) for the gradients do of o and dfinal of the final state."""
    v, do, a = _f(v), _f(do), np.exp(_f(log_decay))[:, None, None]
    B, T, HV, Dv = v.shape
    H, Dk = np.shape(q)[-2:]
    q, k = _group(_f(q), HV), _group(_f(k), HV)
    S = np.zeros((B, HV, Dk, Dv)) if init is None else _f(init).copy()
    G = np.zeros((B, HV, Dk, Dv)) if dfinal is None else _f(dfinal).copy()
    dq, dk, dv = np.zeros((B, T, HV, Dk)), np.zeros((B, T, HV, Dk)), np.zeros((B, T, HV, Dv))
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * np.matmul(S, do[:, t, :, :, None])[..., 0]
    for t in reversed(range(T)):  # G: the gradient of the state after row t
        G = G + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = np.matmul(G, v[:, t, :, :, None])[..., 0]
        dv[:, t] = np.matmul(k[:, t, :, None, :], G)[:, :, 0]
        G = a * G
    shared = lambda x: x.reshape(B, T, H, HV // H, Dk).sum(3)  # noqa: E731
    return shared(dq), shared(dk), dv, G


def linattn_size(q, k, v, log_decay, scale, init=None):
    z = lambda x: None if x is None else np.abs(_f(x))  # noqa: E731
    return linattn(z(q), z(k), z(v), log_decay, abs(scale), z(init))


def linattn_bwd_size(q, k, v, log_decay, scale, do, init=None, dfinal=None):
    z = lambda x: None if x is None else np.abs(_f(x))  # noqa: E731
    return linattn_bwd(z(q), z(k), z(v), log_decay, abs(scale), z(do), z(init), z(dfinal))


def linattn_step(q, k, v, log_decay, scale, pool, idx):
    """One token of rows q, k [N, H, Dk], v [N, HV, Dv] on a copy of pool: (o, pool). idx None: slot n."""
    v, pool, a = _f(v), _f(pool).copy(), np.exp(_f(log_decay))[:, None, None]
    N, HV, _ = v.shape
    q, k = _group(_f(q), HV), _group(_f(k), HV)
    o = np.zeros(v.shape)
    for n in range(N):
        i = n if idx is None else int(idx[n])
        if i >= 0:
            pool[i] = a * pool[i] + k[n, :, :, None] * v[n, :, None, :]
            o[n] = scale * np.matmul(q[n, :, None, :], pool[i])[:, 0]
    return o, pool


def _rotation(table, pos, R, D, interleaved):
    """[rows, D, D] matrices that turn a row's channels."""
    m = np.zeros((len(pos), D, D))
    m[:, range(D), range(D)] = 1.0
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = table[pos, i], table[pos, R // 2 + i]
        m[:, a, a] = c
        m[:, b, b] = c
        m[:, a, b] = -s
        m[:, b, a] = s
    return m


def qknorm(x, w, table, positions, eps, interleaved):
    """One side: x [B, T, H, D], w [D], table [P, R] or None, positions [B, T] or None."""
    x, w = _f(x), _f(w)
    B, T, H, D = x.shape
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    if table is None:
        return y
    pos = np.tile(np.arange(T), B) if positions is None else np.asarray(positions).reshape(-1)
    m = _rotation(_f(table), pos, table.shape[1], D, interleaved)
    return np.einsum("rij,rhj->rhi", m, y.reshape(B * T, H, D)).reshape(x.shape)


def qknorm_bwd(x, w, table, positions, eps, interleaved, dy):
    """(dx, dw) of one side."""
    x, w, u = _f(x), _f(w), _f(dy)
    B, T, H, D = x.shape
    if table is not None:
        pos = np.tile(np.arange(T), B) if positions is None else np.asarray(positions).reshape(-1)
        m = _rotation(_f(table), pos, table.shape[1], D, interleaved)
        u = np.einsum("rij,rhi->rhj", m, u.reshape(B * T, H, D)).reshape(x.shape)
    s = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x / s
    g = u * w
    return (g - n * np.mean(g * n, -1, keepdims=True)) / s, (u * n).reshape(-1, D).sum(0)
