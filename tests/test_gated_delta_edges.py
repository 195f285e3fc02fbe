"""Calls of the gated delta rule at the edges of what its header allows."""

import ctypes
import types

import pytest
import torch

from test_gated_delta_refusals import bwd, fwd, lib, step  # noqa: F401

from kernelized_linear_attention_kata_b200 import _lib as L
from kernelized_linear_attention_kata_b200 import api

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def test_no_value_heads_on_the_host(lib):  # noqa: F811
    """dq and dk are written (with zeros) although no head is: they may not be null."""
    assert bwd(lib, H=0, Hk=2, dq=None) == L.KATA_ERR_INVALID_ARGUMENT
    for call in (fwd, bwd, step):
        assert call(lib, B=1 << 30, H=0, Hk=64) == L.KATA_ERR_UNSUPPORTED
    assert step(lib, H=0, Hk=2, y=ctypes.c_void_p(None)) == L.KATA_OK


def test_no_tensor_with_a_stream_given():
    """The refusal is the same with a stream as without."""
    stream = types.SimpleNamespace(device_index=0, device="cuda:0")
    t = torch.zeros(1, 1, 8, 64)
    gate = torch.zeros(1, 1, 8)
    with pytest.raises(TypeError, match="q must be a tensor"):
        api.kata_fwd_gated_delta(None, t, t, gate, gate, t, stream=stream)
    with pytest.raises(TypeError, match="q must be a tensor"):
        api.kata_bwd_gated_delta(1.0, t, t, gate, gate, t, t, t, t, gate, gate, stream=stream)
    with pytest.raises(TypeError, match="q must be a tensor"):
        api.kata_gated_delta_step(None, t[:, :, 0], t[:, :, 0], gate[:, :, 0], gate[:, :, 0],
                                  torch.zeros(1, 1, 64, 64), t[:, :, 0], stream=stream)
    with pytest.raises(ValueError, match="stream"):
        api.kata_fwd_gated_delta(t, t, t, gate, gate, t, stream=stream)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_value_heads(dtype):
    """Key heads that no value head reads: nothing comes out, their gradients are 0."""
    B, Hk, T, d = 2, 3, 40, 64
    dt = TYPES[dtype]
    q, k = (torch.full((B, Hk, T, d), x, dtype=dt, device="cuda") for x in (0.5, 0.25))
    v, gate = torch.empty(B, 0, T, d, dtype=dt, device="cuda"), torch.empty(B, 0, T, device="cuda")
    S = torch.empty(B, 0, d, d, device="cuda")
    o, S1 = api.fwd_gated_delta(q, k, v, gate, gate, S0=S, return_state=True)
    assert o.shape == v.shape and S1.shape == S.shape
    dq, dk, dv, dg, dbeta, dS0 = (torch.full_like(x, float("nan")) for x in (q, k, v, gate, gate, S))
    api.kata_bwd_gated_delta(q, k, v, gate, gate, v, dq, dk, dv, dg, dbeta, S0=S, dS=S, dS0=dS0)
    assert (dq == 0).all() and (dk == 0).all()
    got = api.bwd_gated_delta(q, k, v, gate, gate, v, S0=S, dS=S)
    assert (got[0] == 0).all() and (got[1] == 0).all() and got[2].shape == v.shape
