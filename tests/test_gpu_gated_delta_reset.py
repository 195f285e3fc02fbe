"""A reset (a log decay of -inf, or of -110 and below) drops the state: what
follows has the bits of a start from nothing, in the forward and in the step,
however large the state was. e^-110 is 1.7e-48, an eight-hundredth of fp32's least
value 1.4e-45, and rounds to 0; 0 times a finite state is 0, and adding it
changes no bit."""

import pytest
import torch

from test_gpu_gated_delta import IN, make, on_gpu

from kernelized_linear_attention_kata_b200 import api
from kernelized_linear_attention_kata_b200 import build as kbuild

pytestmark = pytest.mark.gpu
RESETS = [-float("inf"), -1e30, -200.0, -110.0]


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kbuild.build()
    api.lib()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g", RESETS)
@pytest.mark.parametrize("T", [1, 70])
def test_forward_drops_the_state(dtype, g, T):
    d = on_gpu(make(2, 2, 2, T, 64, 64, dtype, seed=T))
    d["g"][:, :, 0] = g
    args = [d[n] for n in IN]
    want = api.fwd_gated_delta(*args, S0=torch.zeros_like(d["S0"]), return_state=True)
    got = api.fwd_gated_delta(*args, S0=1e37 * d["S0"], return_state=True)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g", RESETS)
def test_step_drops_the_state(dtype, g):
    d = on_gpu(make(2, 2, 2, 1, 64, 64, dtype, seed=3))
    d["g"][:] = g
    args = [d[n][:, :, 0].contiguous() for n in IN]
    old, none = 1e37 * d["S0"], torch.zeros_like(d["S0"])
    assert torch.equal(api.gated_delta_step(*args, old), api.gated_delta_step(*args, none))
    assert torch.equal(old, none)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_reset_in_a_prompt_and_in_a_step_agree(dtype):
    """The reset as the last token of a prompt, and as a step behind the prompt: the
    states differ by the rounding of one token's write at most. S = beta k v^T: the
    product in the forward is off by 2^-16 (bf16 halves of the write) of its
    largest entry, in the step by two roundings of 2^-24."""
    d = on_gpu(make(1, 2, 2, 9, 64, 64, dtype, seed=5))
    d["g"][:, :, 8] = -float("inf")
    _, whole = api.fwd_gated_delta(*(d[n] for n in IN), S0=1e37 * d["S0"], return_state=True)
    _, S = api.fwd_gated_delta(*(d[n][:, :, :8].contiguous() for n in IN), S0=1e37 * d["S0"], return_state=True)
    api.gated_delta_step(*(d[n][:, :, 8].contiguous() for n in IN), S)
    assert float((whole - S).abs().max()) <= 2.0 ** -15 * float(S.abs().max())
