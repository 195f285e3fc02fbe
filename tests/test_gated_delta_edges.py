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


def inputs(B, Hk, H, T, d_k, d_v, dtype, seed, state):
    from test_gpu_gated_delta import make, on_gpu
    t = make(B, Hk, H, T, d_k, d_v, dtype, seed=seed, state=state)
    t["g"] *= 0.05                                  # the carry matters over many chunks
    return t, on_gpu(t)


IN = ("q", "k", "v", "g", "beta")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", [(16, 32), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("B, Hk, H, T", [(1, 1, 2, 129), (1, 2, 2, 2500)])
@pytest.mark.parametrize("given", ["nothing", "S0", "dS"])
def test_segments_without_all_states(dtype, d_k, d_v, B, Hk, H, T, given):
    """A sequence cut into segments that starts from nothing, or whose last state
    has no gradient."""
    from test_gpu_gated_delta import GRADS, close, oracle_backward, oracle_forward
    t, d = inputs(B, Hk, H, T, d_k, d_v, dtype, T + d_k, True)
    for name in {"S0", "dS"} - {given}:
        del t[name], d[name]
    split = dtype == "bf16"
    o, S = api.fwd_gated_delta(*(d[n] for n in IN), S0=d.get("S0"), return_state=True)
    ref_o, ref_S = oracle_forward(t)
    close(o, ref_o, d_k, d_v, split, "o")
    close(S, ref_S, d_k, d_v, split, "S")
    assert torch.equal(api.fwd_gated_delta(*(d[n] for n in IN), S0=d.get("S0")), o)
    got = api.bwd_gated_delta(*(d[n] for n in IN), d["dout"], S0=d.get("S0"), dS=d.get("dS"))
    ref = oracle_backward(t)
    for name, x, r in zip(GRADS, got, ref):
        if x is not None:
            close(x, r, d_k, d_v, split, name)
    assert (got[5] is None) == ("S0" not in d)
    if "S0" not in d:                               # the starting state's gradient, asked for by itself
        out = [torch.empty_like(x) for x in got[:5]]
        dS0 = torch.empty(B, H, d_k, d_v, device="cuda")
        api.kata_bwd_gated_delta(*(d[n] for n in IN), d["dout"], *out, dS=d.get("dS"), dS0=dS0)
        close(dS0, ref[5], d_k, d_v, split, "dS0")
        for x, y in zip(out, got):
            assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_and_step_on_a_given_stream(dtype):
    """Two gradients and two steps at once on two streams, none of them the current one."""
    sets = [inputs(1, 2, 4, 333, 128, 64, dtype, s, True)[1] for s in (1, 2)]
    want, want_y, want_S = [], [], []
    for d in sets:
        want.append(api.bwd_gated_delta(*(d[n] for n in IN), d["dout"], S0=d["S0"], dS=d["dS"]))
        d["token"] = [d[n][:, :, 5].contiguous() for n in IN]
        want_S.append(d["S0"].clone())
        want_y.append(api.gated_delta_step(*d["token"], want_S[-1]))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in sets], []
    for s, d, w in zip(streams, sets, want):
        s.wait_stream(torch.cuda.current_stream())
        out = [torch.full_like(x, float("nan")) for x in w]
        S, y = d["S0"].clone(), torch.full_like(d["token"][2], float("nan"))
        s.wait_stream(torch.cuda.current_stream())
        api.kata_bwd_gated_delta(*(d[n] for n in IN), d["dout"], *out[:5], S0=d["S0"], dS=d["dS"], dS0=out[5], stream=s)
        api.kata_gated_delta_step(*d["token"], S, y, stream=s)
        outs.append((out, S, y))
    torch.cuda.synchronize()
    for (out, S, y), w, wS, wy in zip(outs, want, want_S, want_y):
        assert torch.equal(S, wS) and torch.equal(y, wy)
        for a, b in zip(out, w):
            assert torch.equal(a, b)


def moved(x):
    """A contiguous copy that starts one entry off its allocation's border."""
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
    flat[1:].copy_(x.reshape(-1))
    return flat[1:].view(x.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v, T", [(64, 64, 90), (32, 128, 1000), (128, 16, 20)])
def test_unaligned_gradients(dtype, d_k, d_v, T):
    """Inputs and outputs off a 16-byte border: fp32 tensors all, of a bf16 call those
    that are fp32 (its own are refused)."""
    _, d = inputs(1, 1, 2, T, d_k, d_v, dtype, 7, True)
    want = api.bwd_gated_delta(*(d[n] for n in IN), d["dout"], S0=d["S0"], dS=d["dS"])
    o, S = api.fwd_gated_delta(*(d[n] for n in IN), S0=d["S0"], return_state=True)
    u = {n: moved(x) if x.dtype == torch.float32 else x for n, x in d.items()}
    out = [moved(torch.full_like(x, float("nan"))) if x.dtype == torch.float32 else torch.empty_like(x) for x in want]
    api.kata_bwd_gated_delta(*(u[n] for n in IN), u["dout"], *out[:5], S0=u["S0"], dS=u["dS"], dS0=out[5])
    for x, y in zip(out, want):
        assert torch.equal(x, y)
    S1 = moved(torch.full_like(S, float("nan")))
    o1 = moved(torch.zeros_like(o)) if o.dtype == torch.float32 else torch.empty_like(o)
    api.kata_fwd_gated_delta(*(u[n] for n in IN), o1, S0=u["S0"], S_out=S1)
    assert torch.equal(o1, o) and torch.equal(S1, S)
    if dtype == "bf16":
        for i, name in enumerate(("dq", "dk", "dv")):
            bad = [torch.empty_like(x) for x in want]
            bad[i] = moved(bad[i])
            with pytest.raises(L.KataError):
                api.kata_bwd_gated_delta(*(d[n] for n in IN), d["dout"], *bad[:5])
        with pytest.raises(L.KataError):
            api.bwd_gated_delta(*(d[n] for n in IN), moved(d["dout"]))
