"""Tensors of more than 2^31 elements: the last heads of a call that large against
the same heads in a call of their own (the heads are independent).

With at least as many heads as SMs no sequence is cut into segments, and the
results have the same bits. A gradient of fewer heads may be cut, which changes the order
of its sums: both calls are then within the gradients' 64-bit tolerance of each
other's exact value, 2 (4 (d_k + d_v + 256) 2^-24 + 8 * 2^-16) of the largest
entry = 5e-4, and a bf16 value has one rounding step of 2^-7 on top."""

import pytest
import torch

from kernelized_linear_attention_kata_b200 import api
from kernelized_linear_attention_kata_b200 import build as kbuild

pytestmark = pytest.mark.gpu
D = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kbuild.build()
    api.lib()
    yield
    torch.cuda.empty_cache()


def inputs(H, T, dtype, seed):
    """q, k, v, g, beta of one sequence; made head by head, to need no more than they take."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = (torch.empty(1, H, T, D, dtype=TYPES[dtype], device="cuda") for _ in range(3))
    for h in range(H):
        for i, x in enumerate((q, k, v)):
            y = torch.randn(T, D, device="cuda", generator=gen)
            x[0, h] = y if i == 2 else y / torch.linalg.vector_norm(y, dim=-1, keepdim=True)
    g = -0.1 * torch.rand(1, H, T, device="cuda", generator=gen)
    return [q, k, v, g, torch.rand(1, H, T, device="cuda", generator=gen)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(dtype):
    H, T, n = 300, 57 * 1024 + 5, 150
    assert H * T * D > 2 ** 31
    t = inputs(H, T, dtype, 1)
    o, S = api.fwd_gated_delta(*t, return_state=True)
    o1, S1 = api.fwd_gated_delta(*(x[:, -n:].contiguous() for x in t), return_state=True)
    assert torch.equal(o[:, -n:], o1) and torch.equal(S[:, -n:], S1)


def test_gradient(dtype="bf16"):
    H, T, n = 280, 61 * 1024, 2
    assert H * T * D > 2 ** 31
    torch.cuda.empty_cache()
    need = 12 * 2 * H * T * D + api.bwd_gated_delta_workspace_bytes(1, H, H, T, D, D)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of free device memory")
    t = inputs(H, T, dtype, 2)
    do = t[2].flip(1)
    part = [x[:, -n:].contiguous() for x in t + [do]]
    got = [x[:, -n:].clone() for x in api.bwd_gated_delta(*t, do)[:5]]
    del t, do
    torch.cuda.empty_cache()
    for x, y in zip(got, api.bwd_gated_delta(*part)[:5]):
        x, y = x.float(), y.float()
        bound = 5e-4 * y.abs().max() + 2.0 ** -7 * y.abs()
        assert ((x - y).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step(dtype):
    BH, n = 131072 + 40, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(BH, 1, D, device="cuda", generator=gen).to(TYPES[dtype]) for _ in range(3))
    g, beta = -torch.rand(BH, 1, device="cuda", generator=gen), torch.rand(BH, 1, device="cuda", generator=gen) / D
    S = torch.randn(BH, 1, D, D, device="cuda", generator=gen)
    assert S.numel() > 2 ** 31
    part = [x[-n:].clone() for x in (q, k, v, g, beta, S)]
    y = api.gated_delta_step(q, k, v, g, beta, S)
    y1 = api.gated_delta_step(*part)
    assert torch.equal(y[-n:], y1) and torch.equal(S[-n:], part[5])
