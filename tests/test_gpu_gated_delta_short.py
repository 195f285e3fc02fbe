"""The bf16 gradient of short sequences: a head's own tokens decide on its
arithmetic (fp32 below 32 of them), not the heads beside it.

Tolerance of the comparison with 64 bits, fixed before the first run: an fp32
gradient of a gate is a sum of n = d_k + d_v + 4 * 64 terms at most, each addition
off by half a step 2^-24 of what the terms' sizes add up to, and each term is a
product of at most 2 factors in three TF32 parts, off by 2^-22 (four half steps)
each: (n + 8) 2^-24 of the sum of the sizes, which the definition gives with
every value positive and every difference a sum.
"""

import numpy as np
import pytest
import torch

from test_gpu_gated_delta import GRADS, IN, make, n64, on_gpu, oracle_backward

from kernelized_linear_attention_kata_b200 import api
from kernelized_linear_attention_kata_b200 import build as kbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kbuild.build()
    api.lib()


def gradient(d):
    return dict(zip(GRADS, api.bwd_gated_delta(*(d[n] for n in IN), d["dout"], S0=d["S0"], dS=d["dS"])))


def sizes(q, k, v, g, beta, dout, S0, dS):
    """(dg, dbeta) of one head with every value positive and every difference a sum."""
    q, k, v, dout, S, D = (np.abs(x) for x in (q, k, v, dout, S0, dS))
    a, before = np.exp(g), []
    for t in range(len(g)):
        before.append(S)
        S = a[t] * S
        S = S + np.outer(k[t], beta[t] * (v[t] + S.T @ k[t]))
    dg, dbeta = np.zeros(len(g)), np.zeros(len(g))
    for t in reversed(range(len(g))):
        kept = a[t] * before[t]
        D = D + np.outer(q[t], dout[t])
        dd = D.T @ k[t]
        dbeta[t] = dd @ (v[t] + kept.T @ k[t])
        D = D + np.outer(k[t], beta[t] * dd)
        dg[t] = np.sum(kept * D)
        D = a[t] * D
    return dg, dbeta


@pytest.mark.parametrize("d_k, d_v", [(16, 32), (64, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 31])
def test_few_tokens_of_many_heads_run_in_fp32(T, d_k, d_v):
    """The same values as fp32 tensors give the same bits."""
    d = on_gpu(make(4, 40, 40, T, d_k, d_v, "bf16", seed=T))
    got = gradient(d)
    ref = gradient({n: x.float() for n, x in d.items()})
    for name in GRADS:
        assert torch.equal(got[name], ref[name].to(got[name].dtype)), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 5, 31, 32, 40, 64])
def test_a_head_has_the_same_gradient_in_any_batch(T, d):
    t = on_gpu(make(2, 70, 70, T, d, d, "bf16", seed=100 + T))
    batch = gradient(t)
    for b, h in ((0, 0), (1, 37), (1, 69)):
        alone = gradient({n: x[b:b + 1, h:h + 1].contiguous() for n, x in t.items()})
        for name in GRADS:
            assert torch.equal(alone[name], batch[name][b:b + 1, h:h + 1]), name


@pytest.mark.parametrize("d_k, d_v", [(16, 32), (64, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 3, 4])
def test_each_heads_gates_against_64_bits(T, d_k, d_v):
    t = make(2, 70, 70, T, d_k, d_v, "bf16", seed=200 + T)
    got, a = gradient(on_gpu(t)), n64(t)
    ref = dict(zip(GRADS, oracle_backward(t)))
    tol = (d_k + d_v + 4 * 64 + 8) * 2.0 ** -24
    for b in range(2):
        for h in range(70):
            size = sizes(*(a[n][b, h] for n in IN + ("dout", "S0", "dS")))
            for name, s in zip(("dg", "dbeta"), size):
                err = np.abs(got[name][b, h].double().cpu().numpy() - ref[name][b, h])
                assert np.all(err <= tol * s), (name, b, h, float(np.max(err / s)))
