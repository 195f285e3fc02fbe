"""The checks of the gated delta rule's gradient reject wrong gradients (CPU): a
term left out of the adjoint, one at a time, fails the central differences that
pin the oracle and the tolerance that the GPU is held to."""

import numpy as np
import pytest
import torch

from oracle import gated_delta as O
from test_gpu_gated_delta import close

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")
MISTAKES = {
    "the decay of the carried gradient": ("dg", "dS0"),
    "the write's share of the carried gradient": ("dg", "dS0"),
    "the query's share of the carried gradient": ("dv", "dbeta"),
    "dq's own write": ("dq",),
    "dk's read of the state": ("dk",),
    "dk's write": ("dk",),
    "dg's decayed state": ("dg",),
    "dbeta's read of the state": ("dbeta",),
}


def backward(q, k, v, g, beta, dout, S0, dS, without=None):
    """The adjoint of the recurrence, last token first, but for what `without` names."""
    def keep(name):
        assert name in MISTAKES
        return name != without
    before, S = [], S0
    for t in range(len(g)):
        before.append(S)
        S = np.exp(g[t]) * S
        S = S + np.outer(k[t], beta[t] * (v[t] - S.T @ k[t]))
    dq, dk, dv = (np.zeros(x.shape) for x in (q, k, v))
    dg, dbeta, D = np.zeros(len(g)), np.zeros(len(g)), dS
    for t in reversed(range(len(g))):
        kept = np.exp(g[t]) * before[t]
        miss = v[t] - kept.T @ k[t]
        write = np.outer(k[t], beta[t] * miss)
        dq[t] = (kept + (write if keep("dq's own write") else 0)) @ dout[t]
        if keep("the query's share of the carried gradient"):
            D = D + np.outer(q[t], dout[t])
        dd = D.T @ k[t]
        dbeta[t] = dd @ (miss if keep("dbeta's read of the state") else v[t])
        dv[t] = beta[t] * dd
        dk[t] = (D @ (beta[t] * miss) if keep("dk's write") else 0) - \
            (kept @ dv[t] if keep("dk's read of the state") else 0)
        if keep("the write's share of the carried gradient"):
            D = D - np.outer(k[t], dv[t])
        dg[t] = np.sum((kept if keep("dg's decayed state") else before[t]) * D)
        if keep("the decay of the carried gradient"):
            D = np.exp(g[t]) * D
    return dq, dk, dv, dg, dbeta, D


def case(T=7, d_k=4, d_v=3, seed=0):
    r = np.random.default_rng(seed)
    q, k = r.normal(size=(T, d_k)), r.normal(size=(T, d_k))
    q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
    return [q, k, r.normal(size=(T, d_v)), -np.abs(r.normal(size=T)), r.uniform(size=T),
            r.normal(size=(d_k, d_v))], r.normal(size=(T, d_v)), r.normal(size=(d_k, d_v))


def off_differences(args, dout, dS, got):
    """The names of the gradients with an entry that central differences reject: h^2
    truncation plus eps |loss| / h rounding, as for the oracle's own pin."""
    def loss():
        o, S = O.forward(*args)
        return np.sum(o * dout) + np.sum(S * dS)
    h, wrong = 1e-6, set()
    for name, x, grad in zip(NAMES, args, got):
        for i in np.ndindex(x.shape):
            kept = x[i]
            x[i] = kept + h
            up = loss()
            x[i] = kept - h
            down = loss()
            x[i] = kept
            if abs((up - down) / (2 * h) - grad[i]) > 1e-7 * max(1.0, abs(loss())):
                wrong.add(name)
    return wrong


def off_tolerance(got, ref, d_k, d_v, split):
    wrong = set()
    for name, x, r in zip(NAMES, got, ref):
        try:
            close(torch.from_numpy(x).float(), r, d_k, d_v, split, name)
        except AssertionError:
            wrong.add(name)
    return wrong


def test_the_right_gradient_passes():
    args, dout, dS = case()
    got = backward(*args[:5], dout, args[5], dS)
    for x, y in zip(got, O.backward(*args[:5], dout, args[5], dS)):
        np.testing.assert_array_equal(x, y)
    assert off_differences(args, dout, dS, got) == set()
    assert off_tolerance(got, got, 4, 3, False) == set()


@pytest.mark.parametrize("mistake", MISTAKES)
def test_a_missing_term_is_rejected(mistake):
    args, dout, dS = case()
    bad = backward(*args[:5], dout, args[5], dS, without=mistake)
    right = backward(*args[:5], dout, args[5], dS)
    assert set(MISTAKES[mistake]) <= off_differences(args, dout, dS, bad)
    for split in (False, True):
        assert set(MISTAKES[mistake]) <= off_tolerance(bad, right, 128, 128, split)
