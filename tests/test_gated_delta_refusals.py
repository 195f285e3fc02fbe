"""The gated delta rule's refusals, on the host (no GPU needed): the C ABI's
status codes and the Python binding's errors come before any launch."""

import ctypes

import pytest
import torch

from kernelized_linear_attention_kata_b200 import _lib as L
from kernelized_linear_attention_kata_b200 import api
from kernelized_linear_attention_kata_b200 import build as kbuild

P = ctypes.c_void_p(256)
BF16, F32 = L.KATA_DTYPE_BF16, L.KATA_DTYPE_F32


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return L.lib()


def fwd(lib, B=1, Hk=1, H=1, T=16, d_k=64, d_v=64, dtype=BF16, S0=None, S_out=None, ws=P,
        ws_bytes=1 << 30, q=P):
    return lib.kata_fwd_gated_delta(q, P, P, P, P, P, B, Hk, H, T, d_k, d_v, dtype, S0, S_out, ws,
                                    ws_bytes, None)


def bwd(lib, B=1, Hk=1, H=1, T=16, d_k=64, d_v=64, dtype=BF16, dS=None, dS0=None, ws=P,
        ws_bytes=1 << 30, dq=P):
    return lib.kata_bwd_gated_delta(P, P, P, P, P, P, None, dS, dq, P, P, P, P, dS0, B, Hk, H, T, d_k,
                                    d_v, dtype, ws, ws_bytes, None)


def step(lib, B=1, Hk=1, H=1, d_k=64, d_v=64, dtype=BF16, S=P, y=P):
    return lib.kata_gated_delta_step(P, P, P, P, P, S, y, B, Hk, H, d_k, d_v, dtype, None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_shapes_and_types(lib, call):
    assert call(lib, d_k=48) == L.KATA_ERR_UNSUPPORTED
    assert call(lib, d_v=256) == L.KATA_ERR_UNSUPPORTED
    assert call(lib, d_k=0) == L.KATA_ERR_UNSUPPORTED
    assert call(lib, dtype=7) == L.KATA_ERR_UNSUPPORTED
    assert call(lib, B=-1) == L.KATA_ERR_INVALID_ARGUMENT
    assert call(lib, H=-2) == L.KATA_ERR_INVALID_ARGUMENT
    assert call(lib, Hk=2, H=3) == L.KATA_ERR_INVALID_ARGUMENT
    assert call(lib, Hk=0, H=3) == L.KATA_ERR_INVALID_ARGUMENT
    assert call(lib, B=1 << 30, H=64, Hk=64) == L.KATA_ERR_UNSUPPORTED      # beyond the grid


@pytest.mark.parametrize("call", [fwd, bwd])
def test_lengths_and_workspaces(lib, call):
    assert call(lib, T=-1) == L.KATA_ERR_INVALID_ARGUMENT
    assert call(lib, T=0x7fffffff) == L.KATA_ERR_UNSUPPORTED
    assert call(lib, ws=None) == L.KATA_ERR_WORKSPACE
    assert call(lib, ws=ctypes.c_void_p(256 + 16)) == L.KATA_ERR_WORKSPACE
    size = {fwd: lib.kata_fwd_gated_delta_workspace_bytes,
            bwd: lib.kata_bwd_gated_delta_workspace_bytes}[call]
    need = size(1, 1, 1, 16, 64, 64, BF16)
    assert need >= 256
    assert call(lib, ws_bytes=need - 1) == L.KATA_ERR_WORKSPACE
    assert size(1, 1, 1, 16, 48, 64, BF16) == 0
    assert size(1, 2, 3, 16, 64, 64, BF16) == 0
    assert size(1, 1, 1, -1, 64, 64, BF16) == 0


def test_null_and_overlapping_pointers(lib):
    assert fwd(lib, q=None) == L.KATA_ERR_INVALID_ARGUMENT
    assert fwd(lib, S0=P, S_out=P) == L.KATA_ERR_INVALID_ARGUMENT
    assert fwd(lib, S0=P, S_out=ctypes.c_void_p(256 + 64)) == L.KATA_ERR_INVALID_ARGUMENT
    assert bwd(lib, dq=None) == L.KATA_ERR_INVALID_ARGUMENT
    assert bwd(lib, dS=P, dS0=P) == L.KATA_ERR_INVALID_ARGUMENT
    assert step(lib, y=None) == L.KATA_ERR_INVALID_ARGUMENT
    assert step(lib, S=ctypes.c_void_p(264)) == L.KATA_ERR_INVALID_ARGUMENT
    assert step(lib, B=0) == L.KATA_OK                          # nothing to do


def tensors(T=8, **change):
    t = {"q": torch.zeros(2, 2, T, 64), "k": torch.zeros(2, 2, T, 64), "v": torch.zeros(2, 4, T, 64),
         "g": torch.zeros(2, 4, T), "beta": torch.zeros(2, 4, T)}
    t.update(change)
    return t


@pytest.mark.parametrize("change, error", [
    ({"k": torch.zeros(2, 2, 9, 64)}, ValueError),
    ({"v": torch.zeros(2, 4, 9, 64)}, ValueError),
    ({"v": torch.zeros(2, 3, 8, 64), "g": torch.zeros(2, 3, 8), "beta": torch.zeros(2, 3, 8)}, ValueError),
    ({"v": torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)}, TypeError),
    ({"g": torch.zeros(2, 2, 8)}, ValueError),
    ({"beta": torch.zeros(2, 4)}, ValueError),
    ({"q": torch.zeros(2, 2, 8, 64, dtype=torch.float64), "k": torch.zeros(2, 2, 8, 64, dtype=torch.float64),
      "v": torch.zeros(2, 4, 8, 64, dtype=torch.float64)}, TypeError),
    ({}, ValueError),                                           # CPU tensors: there is no fallback
])
def test_binding_refuses(change, error):
    t = tensors(**change)
    with pytest.raises(error):
        api.fwd_gated_delta(**t)
    with pytest.raises(error):
        api.bwd_gated_delta(**t, dout=torch.zeros_like(t["v"]))


def test_binding_refuses_states_and_outputs():
    t = tensors()
    o = torch.zeros_like(t["v"])
    with pytest.raises(ValueError):
        api.kata_fwd_gated_delta(**t, o=o, S0=torch.zeros(2, 4, 64, 32))
    with pytest.raises(ValueError):
        api.kata_fwd_gated_delta(**t, o=o, S_out=torch.zeros(2, 4, 64, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        api.kata_fwd_gated_delta(**t, o=torch.zeros(2, 4, 8, 32))
    with pytest.raises(ValueError):
        api.gated_delta_step(t["q"], t["k"], t["v"], t["g"], t["beta"], torch.zeros(2, 4, 64, 64))
    with pytest.raises(ValueError):
        api.gated_delta_step(*(t[n][:, :, 0] for n in ("q", "k", "v", "g", "beta")),
                             torch.zeros(2, 2, 64, 64))


def test_binding_refuses_what_is_no_tensor():
    t = tensors()
    for name in t:
        with pytest.raises(TypeError):
            api.fwd_gated_delta(**{**t, name: None})
        with pytest.raises(TypeError):
            api.bwd_gated_delta(**{**t, name: 1.0}, dout=t["v"])
    with pytest.raises(TypeError):
        api.bwd_gated_delta(**t, dout=None)
    with pytest.raises(TypeError):
        api.fwd_gated_delta(**t, S0="none")
    with pytest.raises(TypeError):
        api.kata_fwd_gated_delta(**t, o=None)
    with pytest.raises(TypeError):
        api.kata_bwd_gated_delta(**t, dout=t["v"], dq=t["q"], dk=None, dv=t["v"], dg=t["g"], dbeta=t["g"])
    token = [t[n][:, :, 0] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(TypeError):
        api.kata_gated_delta_step(*token, torch.zeros(2, 4, 64, 64), None)
    with pytest.raises(TypeError):
        api.gated_delta_step(*token, None)


def test_binding_refuses_sizes_beyond_32_bits():
    n = 1 << 31
    q = torch.zeros(1, 1, 1, 64).expand(1, 1, n, 64)
    gate = torch.zeros(1, 1, 1).expand(1, 1, n)
    with pytest.raises(ValueError):
        api.fwd_gated_delta(q, q, q, gate, gate)
