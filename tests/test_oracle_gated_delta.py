"""Pins of the gated delta rule's fp64 oracle (CPU): closed forms of the
forward and central differences of every gradient entry."""

import numpy as np
import pytest

from oracle import gated_delta as O


def case(T, d_k, d_v, seed):
    r = np.random.default_rng(seed)
    q, k = r.normal(size=(T, d_k)), r.normal(size=(T, d_k))
    q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
    return (q, k, r.normal(size=(T, d_v)), -np.abs(r.normal(size=T)), r.uniform(size=T),
            r.normal(size=(d_k, d_v)))


def test_first_token_from_zero():
    q, k, v, g, beta, _ = case(1, 5, 3, 0)
    o, S = O.forward(q, k, v, g, beta)
    np.testing.assert_allclose(o[0], beta[0] * (q[0] @ k[0]) * v[0], atol=1e-14)
    np.testing.assert_allclose(S, beta[0] * np.outer(k[0], v[0]), atol=1e-14)


def test_orthogonal_keys_are_additive_with_decay():
    _, _, v, g, beta, _ = case(4, 4, 3, 1)
    o, S = O.forward(np.eye(4), np.eye(4), v, g, beta)
    G = np.cumsum(g)
    np.testing.assert_allclose(S, np.exp(G[-1] - G)[:, None] * beta[:, None] * v, atol=1e-13)
    np.testing.assert_allclose(o, beta[:, None] * v, atol=1e-13)


def test_full_strength_overwrites_and_padding_keeps():
    q, k, v, g, beta, S0 = case(3, 6, 2, 2)
    beta[:], g[:] = 1.0, 0.0
    k[2] = k[0]
    _, S = O.forward(q, k, v, g, beta, S0)
    np.testing.assert_allclose(S.T @ k[0], v[2], atol=1e-13)
    _, same = O.forward(q, k, v, np.zeros(3), np.zeros(3), S0)
    np.testing.assert_array_equal(same, S0)


def test_reset_forgets():
    q, k, v, g, beta, S0 = case(9, 4, 3, 3)
    g[5] = -np.inf
    o, S = O.forward(q, k, v, g, beta, S0)
    o2, S2 = O.forward(q[5:], k[5:], v[5:], g[5:], beta[5:])
    np.testing.assert_allclose(o[5:], o2, atol=1e-14)
    np.testing.assert_allclose(S, S2, atol=1e-14)


@pytest.mark.parametrize("seed", [0, 1])
def test_gradient_against_central_differences(seed):
    T, d_k, d_v = 7, 4, 3
    q, k, v, g, beta, S0 = case(T, d_k, d_v, seed)
    r = np.random.default_rng(seed + 9)
    dout, dS = r.normal(size=(T, d_v)), r.normal(size=(d_k, d_v))
    args = [q, k, v, g, beta, S0]

    def loss():
        o, S = O.forward(*args)
        return np.sum(o * dout) + np.sum(S * dS)
    got = O.backward(q, k, v, g, beta, dout, S0, dS)
    h = 1e-6
    for x, grad in zip(args, got):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + h
            up = loss()
            x[i] = keep - h
            down = loss()
            x[i] = keep
            # central differences: h^2 truncation plus eps |loss| / h rounding
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-7 * max(1.0, abs(loss())), i


def test_a_planted_mistake_fails():
    """The gradient without the decay's factor in the carried state is caught."""
    q, k, v, g, beta, S0 = case(5, 4, 3, 4)
    dout = np.random.default_rng(1).normal(size=v.shape)
    good = O.backward(q, k, v, g, beta, dout, S0)
    bad = O.backward(q, k, v, np.zeros_like(g), beta, dout, S0)
    assert np.max(np.abs(good[2] - bad[2])) > 1e-3


def test_shared_heads_sum_their_gradients():
    r = np.random.default_rng(5)
    B, Hk, H, T, d_k, d_v = 2, 2, 4, 5, 4, 3
    q, k = r.normal(size=(B, Hk, T, d_k)), r.normal(size=(B, Hk, T, d_k)) * 0.5
    v, dout = r.normal(size=(B, H, T, d_v)), r.normal(size=(B, H, T, d_v))
    g, beta = -r.uniform(size=(B, H, T)), r.uniform(size=(B, H, T))
    shared = O.backward_heads(q, k, v, g, beta, dout)
    full = O.backward_heads(np.repeat(q, 2, 1), np.repeat(k, 2, 1), v, g, beta, dout)
    for i in range(2):
        np.testing.assert_allclose(shared[i], full[i].reshape(B, Hk, 2, T, d_k).sum(2), atol=1e-12)
    for i in range(2, 6):
        np.testing.assert_allclose(shared[i], full[i], atol=1e-12)
