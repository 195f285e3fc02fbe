"""fp64 oracle of the gated delta rule and its gradient (test infrastructure).

One value head, token by token, from the definition:
    S_t = e^{g_t} S_{t-1} + k_t d_t^T,  d_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),
    o_t = S_t^T q_t.
The gradient is the adjoint of that recurrence, last token first. The batched
forms read query / key head h // (H / H_k) for value head h.
"""

import numpy as np


def forward(q, k, v, g, beta, S0=None):
    """(o [T, d_v], S [d_k, d_v]) of one head."""
    S = np.zeros((q.shape[1], v.shape[1])) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.empty((q.shape[0], v.shape[1]))
    for t in range(q.shape[0]):
        S = np.exp(g[t]) * S
        S = S + np.outer(k[t], beta[t] * (v[t] - S.T @ k[t]))
        o[t] = S.T @ q[t]
    return o, S


def backward(q, k, v, g, beta, dout, S0=None, dS=None):
    """(dq, dk, dv, dg, dbeta, dS0) of sum(dout * o) + sum(dS * S) of one head."""
    T = q.shape[0]
    S = np.zeros((q.shape[1], v.shape[1])) if S0 is None else np.array(S0, dtype=np.float64)
    before = []
    for t in range(T):
        before.append(S)
        S = np.exp(g[t]) * S
        S = S + np.outer(k[t], beta[t] * (v[t] - S.T @ k[t]))
    dq, dk, dv = (np.zeros(x.shape) for x in (q, k, v))
    dg, dbeta = np.zeros(T), np.zeros(T)
    D = np.zeros(S.shape) if dS is None else np.array(dS, dtype=np.float64)
    for t in reversed(range(T)):
        kept = np.exp(g[t]) * before[t]
        miss = v[t] - kept.T @ k[t]
        d = beta[t] * miss
        dq[t] = (kept + np.outer(k[t], d)) @ dout[t]
        D = D + np.outer(q[t], dout[t])
        dd = D.T @ k[t]
        dbeta[t] = dd @ miss
        dv[t] = beta[t] * dd
        dk[t] = D @ d - kept @ dv[t]
        D = D - np.outer(k[t], dv[t])
        dg[t] = np.sum(kept * D)
        D = np.exp(g[t]) * D
    return dq, dk, dv, dg, dbeta, D


def forward_heads(q, k, v, g, beta, S0=None):
    """(o [B, H, T, d_v], S [B, H, d_k, d_v]) of q, k [B, H_k, T, d_k], v
    [B, H, T, d_v], g, beta [B, H, T]."""
    B, H = v.shape[:2]
    r = H // q.shape[1]
    got = [[forward(q[b, h // r], k[b, h // r], v[b, h], g[b, h], beta[b, h],
                    None if S0 is None else S0[b, h]) for h in range(H)] for b in range(B)]
    return tuple(np.array([[x[i] for x in row] for row in got]) for i in range(2))


def backward_heads(q, k, v, g, beta, dout, S0=None, dS=None):
    """The gradients with the shapes of the inputs; a shared head's dq, dk are
    sums over its value heads."""
    B, H = v.shape[:2]
    r = H // q.shape[1]
    got = [[backward(q[b, h // r], k[b, h // r], v[b, h], g[b, h], beta[b, h], dout[b, h],
                     None if S0 is None else S0[b, h], None if dS is None else dS[b, h])
            for h in range(H)] for b in range(B)]
    dq, dk, dv, dg, db, dS0 = (np.array([[x[i] for x in row] for row in got]) for i in range(6))
    dq, dk = (x.reshape((B, -1, r) + x.shape[2:]).sum(2) for x in (dq, dk))
    return dq, dk, dv, dg, db, dS0
