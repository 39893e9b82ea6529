"""The float64 oracle of linear attention and of the per-head norm with rotation, held against
finite differences, the closed sums of their definitions, and each other (CPU)."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import layer

RNG = np.random.default_rng(7)


def _case(B, T, H, HV, Dk, Dv):
    n = RNG.standard_normal
    return (n((B, T, H, Dk)), n((B, T, H, Dk)), n((B, T, HV, Dv)), -np.abs(n(HV)), 0.37, n((B, HV, Dk, Dv)))


def test_recurrence_equals_the_closed_sum():
    q, k, v, g, scale, S0 = _case(2, 9, 2, 4, 3, 5)
    o, S = layer.linattn(q, k, v, g, scale, S0)
    a = np.exp(g)
    for b in range(2):
        for h in range(4):
            for t in range(9):
                want = a[h] ** (t + 1) * q[b, t, h // 2] @ S0[b, h]
                for j in range(t + 1):
                    want = want + a[h] ** (t - j) * (q[b, t, h // 2] @ k[b, j, h // 2]) * v[b, j, h]
                assert np.allclose(o[b, t, h], scale * want, rtol=1e-12, atol=1e-12)
    zero = layer.linattn(q[:, :0], k[:, :0], v[:, :0], g, scale, S0)
    assert zero[0].shape == (2, 0, 4, 5) and np.array_equal(zero[1], S0)


def _differences(f, x, d):
    """Central differences of the scalar f along every entry of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += d
        hi = f(y)
        y[i] -= 2 * d
        g[i] = (hi - f(y)) / (2 * d)
    return g


def test_linattn_gradients_against_differences():
    q, k, v, g, scale, S0 = _case(1, 5, 1, 2, 2, 3)
    do, F = RNG.standard_normal(v.shape), RNG.standard_normal(S0.shape)

    def loss(q=q, k=k, v=v, S0=S0):
        o, S = layer.linattn(q, k, v, g, scale, S0)
        return float((o * do).sum() + (S * F).sum())

    dq, dk, dv, dS0 = layer.linattn_bwd(q, k, v, g, scale, do, S0, F)
    # the loss is at most cubic in each operand's entries alone (linear, in fact): differences are
    # exact but for rounding, about 1e-16 / 1e-4 of the loss
    for name, have, x in (("q", dq, q), ("k", dk, k), ("v", dv, v), ("S0", dS0, S0)):
        assert np.allclose(_differences(lambda y: loss(**{name: y}), x, 1e-4), have, rtol=1e-8, atol=1e-8), name


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(6, 6), (7, 4), (5, 0)])
def test_qknorm_gradients_against_differences(D, R, interleaved):
    x, w = RNG.standard_normal((1, 3, 2, D)), RNG.standard_normal(D)
    angle = RNG.standard_normal((8, R // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], -1) if R else None
    pos, dy = np.array([[5, 0, 7]]), RNG.standard_normal(x.shape)
    f = lambda x, w: float((layer.qknorm(x, w, table, pos, 1e-3, interleaved) * dy).sum())  # noqa: E731
    dx, dw = layer.qknorm_bwd(x, w, table, pos, 1e-3, interleaved, dy)
    assert np.allclose(_differences(lambda y: f(y, w), x, 1e-5), dx, rtol=1e-6, atol=1e-7)
    assert np.allclose(_differences(lambda y: f(x, y), w, 1e-5), dw, rtol=1e-6, atol=1e-7)


def test_rotation_keeps_lengths_and_turns_by_the_difference():
    """q_i . k_j of rotated rows depends on the positions' difference alone."""
    D = 8
    inv = 10.0 ** (-np.arange(D // 2) / D)
    angle = np.arange(64)[:, None] * inv
    table = np.concatenate([np.cos(angle), np.sin(angle)], -1)
    x, y, one = RNG.standard_normal((1, 1, 1, D)), RNG.standard_normal((1, 1, 1, D)), np.ones(D)
    for inter in (False, True):
        at = lambda z, p: layer.qknorm(z, one, table, np.array([[p]]), 0.0, inter).reshape(-1)  # noqa: E731
        assert np.isclose(at(x, 30) @ at(x, 30), D)
        assert np.isclose(at(x, 30) @ at(y, 17), at(x, 53) @ at(y, 40))


def test_steps_reproduce_the_sequence():
    q, k, v, g, scale, S0 = _case(2, 6, 1, 3, 4, 2)
    o, S = layer.linattn(q, k, v, g, scale, S0)
    pool = np.zeros((5, *S0.shape[1:]))
    pool[[3, 1]] = S0
    for t in range(6):
        y, pool = layer.linattn_step(q[:, t], k[:, t], v[:, t], g, scale, pool, [3, 1])
        assert np.allclose(y, o[:, t], rtol=1e-13, atol=1e-13)
    assert np.allclose(pool[[3, 1]], S, rtol=1e-13, atol=1e-13) and not pool[[0, 2, 4]].any()
