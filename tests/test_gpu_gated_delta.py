"""GPU parity of the gated delta rule (chunked forward, gradient, one-token
step) against the fp64 oracle, token by token, on the same inputs.

Tolerances, fixed before the first run. Errors are relative to the largest
entry of the exact tensor. With unit keys and 0 <= beta <= 1 the rule is a
contraction, so partial sums stay within a few times the result's largest
entry. fp32: a value passes through at most n = d_k + d_v + 4 * 64 additions
(a product with the state, the solve, a product with the writes, the update;
for a gradient also the value axis), each off by at most half a step 2^-24 of
a partial sum, taken as 4 times the largest entry: 4 n 2^-24 <= 1.3e-4.
Products of fp32 are made of three TF32 parts and off by at most 2^-22, four
half steps of one of the n terms; the bound's 4 covers them as well. bf16:
the tensor-core kernels take fp32 operands as two bf16 halves, off by at most
2^-16 of the operand; a value meets at most 8 such operands in a row, 8 * 2^-16
= 1.3e-4 on top. An output held in bf16 is rounded once more, half a step,
2^-8 of its value.
"""

import numpy as np
import pytest
import torch

from oracle import gated_delta as O
from kernelized_linear_attention_kata_b200 import api
from kernelized_linear_attention_kata_b200 import build as kbuild
from kernelized_linear_attention_kata_b200._lib import KATA_OK, KataError

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
IN = ("q", "k", "v", "g", "beta")
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kbuild.build()
    api.lib()


def make(B, Hk, H, T, d_k, d_v, dtype, seed, state=True):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    def unit(x):
        return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    dt = TYPES[dtype]
    t = {"q": unit(normal(B, Hk, T, d_k)).to(dt), "k": unit(normal(B, Hk, T, d_k)).to(dt),
         "v": normal(B, H, T, d_v).to(dt), "g": -0.3 * normal(B, H, T).abs(),
         "beta": torch.rand((B, H, T), generator=gen), "dout": normal(B, H, T, d_v).to(dt)}
    if state:
        t["S0"], t["dS"] = normal(B, H, d_k, d_v), normal(B, H, d_k, d_v)
    return t


def on_gpu(t):
    return {n: x.cuda() for n, x in t.items()}


def n64(t):
    return {n: x.double().numpy() for n, x in t.items()}


def oracle_forward(t):
    a = n64(t)
    return O.forward_heads(*(a[n] for n in IN), S0=a.get("S0"))


def oracle_backward(t):
    a = n64(t)
    return O.backward_heads(*(a[n] for n in IN), a["dout"], S0=a.get("S0"), dS=a.get("dS"))


def close(got, ref, d_k, d_v, split, name="", scale=None):
    """|got - ref| <= tol max|ref| (+ 2^-8 |ref| for a bf16 tensor); `split`:
    whether bf16 halves may have been used."""
    tol = 4 * (d_k + d_v + 4 * 64) * 2.0 ** -24 + (8 * 2.0 ** -16 if split else 0.0)
    big = max(np.max(np.abs(ref)), 1e-30) if scale is None else scale
    bound = tol * big + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0.0)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound), (name, float(np.max(err / big)), tol)


def forward(t, **kw):
    return api.fwd_gated_delta(*(t[n] for n in IN), S0=t.get("S0"), return_state=True, **kw)


def backward(t):
    return api.bwd_gated_delta(*(t[n] for n in IN), t["dout"], S0=t.get("S0"), dS=t.get("dS"))


SHAPES = [(16, 16), (16, 128), (32, 64), (64, 32), (64, 64), (64, 128), (128, 16), (128, 64), (128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", SHAPES)
@pytest.mark.parametrize("B, Hk, H, T, state", [(1, 1, 1, 1, True), (2, 1, 1, 2, False), (1, 2, 2, 63, True),
                                                (1, 1, 3, 64, False), (1, 1, 1, 65, True),
                                                (2, 2, 4, 200, True)])
def test_forward_and_gradient(dtype, d_k, d_v, B, Hk, H, T, state):
    t = make(B, Hk, H, T, d_k, d_v, dtype, seed=T + d_k + 3 * d_v, state=state)
    d = on_gpu(t)
    o, S = forward(d)
    ref_o, ref_S = oracle_forward(t)
    split = dtype == "bf16"
    # outputs of short sequences are compared with the values that make them
    close(o, ref_o, d_k, d_v, split, "o")
    close(S, ref_S, d_k, d_v, split, "S")
    got, ref = backward(d), oracle_backward(t)
    big = max(np.max(np.abs(r)) for r in ref[:5])
    for name, x, r in zip(GRADS, got, ref):
        if x is not None:
            # an exact zero (dq from no state ...) is held to the other gradients' size
            close(x, r, d_k, d_v, split, name, scale=max(np.max(np.abs(r)), 1e-3 * big))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_chunks_and_heads(dtype):
    """More chunks than one block holds at a time, with heads to fill the GPU
    unevenly; two heads against the oracle."""
    t = make(2, 5, 5, 1500, 64, 64, dtype, seed=4)
    d = on_gpu(t)
    o, S = forward(d)
    got = backward(d)
    pick = {n: (x[1:, 3:4] if n not in ("g", "beta") else x[1:, 3:4]) for n, x in t.items()}
    ref_o, ref_S = oracle_forward(pick)
    close(o[1:, 3:4], ref_o, 64, 64, dtype == "bf16", "o")
    close(S[1:, 3:4], ref_S, 64, 64, dtype == "bf16", "S")
    for name, x, r in zip(GRADS, got, oracle_backward(pick)):
        close(x[1:, 3:4], r, 64, 64, dtype == "bf16", name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", [(128, 128), (64, 64), (32, 32)])
def test_one_long_head(dtype, d_k, d_v):
    """One head, 70 chunks: the sequence itself is what fills the GPU."""
    t = make(1, 1, 1, 70 * 64 - 5, d_k, d_v, dtype, seed=8)
    t["g"] *= 0.02                                  # a slow decay: the carry matters across all chunks
    d = on_gpu(t)
    o, S = forward(d)
    ref_o, ref_S = oracle_forward(t)
    close(o, ref_o, d_k, d_v, dtype == "bf16", "o")
    close(S, ref_S, d_k, d_v, dtype == "bf16", "S")
    for name, x, r in zip(GRADS, backward(d), oracle_backward(t)):
        close(x, r, d_k, d_v, dtype == "bf16", name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", [(16, 128), (32, 16), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("B, Hk, H, T", [(1, 1, 3, 1000), (2, 1, 2, 129), (1, 4, 60, 540), (1, 2, 2, 2500)])
def test_sequences_in_segments(dtype, d_k, d_v, B, Hk, H, T):
    """Few enough heads for the sequence to be cut: states and their gradients
    pass over the borders of segments, the last of which is short, with shared
    keys and padded head sizes; the first and the last head of the last batch."""
    t = make(B, Hk, H, T, d_k, d_v, dtype, seed=T + d_k + d_v)
    t["g"] *= 0.05                                  # the carry matters over many chunks
    d = on_gpu(t)
    o, S = forward(d)
    got = dict(zip(GRADS, backward(d)))
    for h in (0, H - 1):
        k = h // (H // Hk)
        pick = {n: x[B - 1:, k:k + 1] if n in ("q", "k") else x[B - 1:, h:h + 1] for n, x in t.items()}
        ref_o, ref_S = oracle_forward(pick)
        close(o[B - 1:, h:h + 1], ref_o, d_k, d_v, dtype == "bf16", "o")
        close(S[B - 1:, h:h + 1], ref_S, d_k, d_v, dtype == "bf16", "S")
        ref = dict(zip(GRADS, oracle_backward(pick)))
        for name in ("dv", "dg", "dbeta", "dS0"):
            close(got[name][B - 1:, h:h + 1], ref[name], d_k, d_v, dtype == "bf16", name)
    if H // Hk <= 3:                                # the sums over a shared head's value heads
        last = {n: x[B - 1:] for n, x in t.items()}
        for name, r in zip(GRADS[:2], oracle_backward(last)):
            close(got[name][B - 1:], r, d_k, d_v, dtype == "bf16", name)


@pytest.mark.parametrize("d_k, d_v", [(16, 32), (64, 64), (128, 128)])
@pytest.mark.parametrize("B, Hk, H, T", [(1, 1, 3, 7), (2, 2, 4, 9), (1, 1, 2, 1), (1, 2, 4, 31), (1, 2, 4, 32)])
def test_gradient_of_few_tokens(d_k, d_v, B, Hk, H, T):
    """Shared heads below and at the size from which the bf16 gradient runs on the
    tensor cores; below it the sums are fp32's."""
    t = make(B, Hk, H, T, d_k, d_v, "bf16", seed=5 * T + d_k)
    ref = oracle_backward(t)
    for name, x, r in zip(GRADS, backward(on_gpu(t)), ref):
        close(x, r, d_k, d_v, B * H * T >= 128, name)


@pytest.mark.parametrize("d_k, d_v", [(128, 64), (128, 128), (64, 64)])
def test_shared_heads_of_many_chunks(d_k, d_v):
    """Three value heads a key head and more chunks than blocks: the gradients of
    the keys are added up inside a block; one key head and its value heads."""
    t = make(2, 5, 15, 1990, d_k, d_v, "bf16", seed=23)
    got = dict(zip(GRADS, backward(on_gpu(t))))
    for b, k in ((0, 0), (1, 4)):
        pick = {n: x[b:b + 1, k:k + 1] if n in ("q", "k") else x[b:b + 1, 3 * k:3 * k + 3] for n, x in t.items()}
        for name, r in zip(GRADS, oracle_backward(pick)):
            part = slice(k, k + 1) if name in ("dq", "dk") else slice(3 * k, 3 * k + 3)
            close(got[name][b:b + 1, part], r, d_k, d_v, True, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", [(128, 128), (64, 32)])
def test_more_heads_than_run_at_once(dtype, d_k, d_v):
    """200 heads: blocks take chunks of several heads one after another."""
    t = make(40, 5, 5, 130, d_k, d_v, dtype, seed=17)
    d = on_gpu(t)
    o, S = forward(d)
    got = backward(d)
    for b, h in ((0, 0), (29, 3), (39, 4)):
        pick = {n: x[b:b + 1, h:h + 1] for n, x in t.items()}
        ref_o, ref_S = oracle_forward(pick)
        close(o[b:b + 1, h:h + 1], ref_o, d_k, d_v, dtype == "bf16", "o")
        close(S[b:b + 1, h:h + 1], ref_S, d_k, d_v, dtype == "bf16", "S")
        for name, x, r in zip(GRADS, got, oracle_backward(pick)):
            close(x[b:b + 1, h:h + 1], r, d_k, d_v, dtype == "bf16", name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 128])
def test_gates_at_their_limits(dtype, d):
    """No decay, full overwrites of repeated keys, tokens that write nothing,
    resets (-inf, and a decay far below the type's range) inside chunks and at
    their borders, and many strong decays in one chunk."""
    t = make(1, 1, 4, 150, d, d, dtype, seed=2)
    t["g"][0, 0] = 0.0
    t["k"][0, 0, 20:60] = t["k"][0, 0, 5:6]
    t["beta"][0, 0, 20:60] = 1.0
    t["beta"][0, 1, 10:100] = 0.0
    for at in (0, 17, 64, 65, 127, 149):
        t["g"][0, 2, at] = -float("inf") if at % 2 else -1e30
    t["g"][0, 3] = -50.0 * torch.rand(150)
    dv = on_gpu(t)
    o, S = forward(dv)
    ref_o, ref_S = oracle_forward(t)
    got, ref = backward(dv), oracle_backward(t)
    for h in range(4):
        close(o[:, h], ref_o[:, h], d, d, dtype == "bf16", f"o {h}")
        close(S[:, h], ref_S[:, h], d, d, dtype == "bf16", f"S {h}")
        for name, x, r in zip(GRADS[2:], got[2:], ref[2:]):
            if h == 2 and name == "dg":             # a dropped state has no gradient: e^-100 of it
                r = np.where(np.isfinite(r), r, 0.0)
            big = max(np.max(np.abs(r[:, h])), 1e-3 * np.max(np.abs(ref[2])))
            close(x[:, h], r[:, h], d, d, dtype == "bf16", f"{name} {h}", scale=big)
    for name, x, r in zip(GRADS[:2], got, ref):
        close(x, r, d, d, dtype == "bf16", name)


def test_padding_tokens_leave_the_state():
    """A batch of two lengths: beta = 0 and g = 0 behind the shorter one's end
    give the state of the shorter sequence, and whatever stands in the padded
    q, k, v rows does not matter to it."""
    t = make(2, 2, 2, 140, 64, 64, "bf16", seed=6)
    n = 77
    t["g"][1, :, n:] = 0.0
    t["beta"][1, :, n:] = 0.0
    d = on_gpu(t)
    o, S = forward(d)
    short = {x: (y[1:, :, :n] if y.shape[2:3] == (140,) else y[1:]) for x, y in t.items()}
    ref_o, ref_S = oracle_forward(short)
    close(o[1:, :, :n], ref_o, 64, 64, True, "o")
    close(S[1:], ref_S, 64, 64, True, "S")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_head(dtype):
    """A NaN token poisons its head from there on and no other."""
    t = make(1, 2, 2, 130, 64, 64, dtype, seed=3)
    t["v"][0, 0, 70] = float("nan")
    d = on_gpu(t)
    o, S = forward(d)
    ref_o, ref_S = oracle_forward(t)
    assert torch.isnan(o[0, 0, 70:]).all() and torch.isnan(S[0, 0]).all()
    close(o[0, 0, :64], ref_o[0, 0, :64], 64, 64, True, "before its chunk")
    close(o[0, 1], ref_o[0, 1], 64, 64, dtype == "bf16", "other head")
    close(S[0, 1], ref_S[0, 1], 64, 64, dtype == "bf16", "other head")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", SHAPES)
@pytest.mark.parametrize("B, Hk, H", [(1, 1, 1), (3, 2, 4), (67, 1, 3)])
def test_step(dtype, d_k, d_v, B, Hk, H):
    t = make(B, Hk, H, 1, d_k, d_v, dtype, seed=B + d_k + d_v)
    ref_o, ref_S = oracle_forward(t)
    d = on_gpu(t)
    S = d["S0"].clone()
    y = api.gated_delta_step(*(d[n][:, :, 0].contiguous() for n in IN), S)
    close(y, ref_o[:, :, 0], d_k, d_v, False, "y")
    close(S, ref_S, d_k, d_v, False, "S")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_k, d_v", [(128, 128), (64, 64), (32, 16)])
def test_prompt_then_tokens(dtype, d_k, d_v):
    """Serving: a prompt through the forward, a continuation through a second
    forward from its state, then tokens through the step."""
    T, cut, tail = 150, 83, 5
    t = make(2, 2, 4, T, d_k, d_v, dtype, seed=11)
    d = on_gpu(t)
    ref_o, ref_S = oracle_forward(t)

    def part(a, b):
        return [d[n][:, :, a:b].contiguous() for n in IN]
    o1, S = api.fwd_gated_delta(*part(0, cut), S0=d["S0"], return_state=True)
    o2, S = api.fwd_gated_delta(*part(cut, T - tail), S0=S, return_state=True)
    os = [o1, o2]
    for i in range(T - tail, T):
        os.append(api.gated_delta_step(*(x[:, :, 0].contiguous() for x in part(i, i + 1)), S)[:, :, None])
    close(torch.cat(os, 2), ref_o, d_k, d_v, dtype == "bf16", "o")
    close(S, ref_S, d_k, d_v, dtype == "bf16", "S")


@pytest.mark.parametrize("d", [32, 64])
def test_gradient_against_differences(d):
    """The gradient against central differences of the fp64 forward, along
    random directions of every input: a training step's forward and backward."""
    t = make(1, 1, 2, 100, d, d, "f32", seed=21)
    got = [x.double().cpu() for x in backward(on_gpu(t))]
    a = {n: x.double() for n, x in t.items()}

    def loss(b):
        o, S = O.forward_heads(*(b[n].numpy() for n in IN), S0=b["S0"].numpy())
        return float(np.sum(o * a["dout"].numpy()) + np.sum(S * a["dS"].numpy()))
    gen = torch.Generator().manual_seed(1)
    for name, grad in zip(IN + ("S0",), got):
        dirn = torch.randn(a[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, down = dict(a), dict(a)
        up[name], down[name] = a[name] + h * dirn, a[name] - h * dirn
        slope, said = (loss(up) - loss(down)) / (2 * h), float((grad * dirn).sum())
        # fp32 entries off by 1.3e-4 of the largest at most, added in quadrature, far above
        # the differences' own error of h^2
        size = float(grad.abs().max() * dirn.norm())
        assert abs(slope - said) <= 1.3e-4 * size + 1e-6 * abs(slope), name


def test_results_repeat_bit_for_bit():
    for dtype in ("f32", "bf16"):
        d = on_gpu(make(2, 2, 4, 700, 64, 64, dtype, seed=5))
        first = forward(d) + backward(d)
        for _ in range(2):
            for x, y in zip(forward(d) + backward(d), first):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_own_stream_and_captured_graph(dtype):
    """A call on another stream than the current one, two calls at once on two
    streams, and a captured training step replayed on new inputs."""
    d1, d2 = (on_gpu(make(1, 2, 4, 333, 128, 64, dtype, seed=s)) for s in (1, 2))
    ref1, ref2 = forward(d1), forward(d2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s, d in ((s1, d1), (s2, d2)):
        o, S = torch.full_like(d["v"], float("nan")), torch.full_like(d["S0"], float("nan"))
        s.wait_stream(torch.cuda.current_stream())
        api.kata_fwd_gated_delta(*(d[n] for n in IN), o, S0=d["S0"], S_out=S, stream=s)
        outs.append((o, S))
    torch.cuda.synchronize()
    for got, ref in zip(outs, (ref1, ref2)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])

    live = {n: x.clone() for n, x in d1.items()}
    eager = forward(d2) + backward(d2)
    forward(live), backward(live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(live) + backward(live)
    for n in live:
        live[n].copy_(d2[n])
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(out, eager):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_captured_training_steps(dtype):
    """Two graphs of forward and gradient, replayed by turns and at once on two
    streams: their workspaces are their own."""
    sets = [on_gpu(make(1, 1, 2, 700, 64, 128, dtype, seed=s)) for s in (31, 32)]
    want = [forward(d) + backward(d) for d in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(forward(d) + backward(d))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for out in outs:
            for x in out:
                x.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            for x, y in zip(got, ref):
                assert torch.equal(x, y)


def test_captured_step():
    t = on_gpu(make(3, 1, 2, 1, 64, 64, "bf16", seed=9))
    args = [t[n][:, :, 0].contiguous() for n in IN]
    S, ref = t["S0"].clone(), t["S0"].clone()
    ys = [api.gated_delta_step(*args, ref) for _ in range(2)]
    y = torch.empty_like(args[2])
    api.kata_gated_delta_step(*args, S.clone(), y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.kata_gated_delta_step(*args, S, y)
    for want in ys:
        graph.replay()
        assert torch.equal(y, want)
    assert torch.equal(S, ref)


def test_rows_outside_are_left_as_they_were():
    """Outputs inside larger buffers: what lies before and behind stays."""
    t = on_gpu(make(1, 1, 1, 70, 64, 64, "bf16", seed=1))
    pad = 8 * 64
    buf = torch.full((70 * 64 + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[pad:pad + 70 * 64].view(1, 1, 70, 64)
    api.kata_fwd_gated_delta(*(t[n] for n in IN), o, S0=t["S0"])
    ref, _ = forward(t)
    assert torch.equal(o, ref)
    assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()


def test_unaligned_tensors():
    """Contiguous tensors that start off a 16-byte border: taken in fp32,
    refused in bf16, whose tiles TMA loads."""
    for dtype, d in (("bf16", 64), ("bf16", 32), ("f32", 64)):
        t = on_gpu(make(1, 2, 2, 90, d, d, dtype, seed=12))
        ref, ref_S = forward(t)
        for n in ("q", "k", "v"):
            flat = torch.empty(t[n].numel() + 1, dtype=t[n].dtype, device="cuda")
            moved = flat[1:].view(t[n].shape)
            moved.copy_(t[n])
            u = dict(t)
            u[n] = moved
            if dtype == "bf16":
                with pytest.raises(KataError):
                    forward(u)
                continue
            o, S = forward(u)
            assert torch.equal(o, ref) and torch.equal(S, ref_S)


def test_empty_problems():
    t = on_gpu(make(2, 1, 2, 3, 64, 64, "bf16", seed=1))
    e = {n: (x[:, :, :0].contiguous() if n in IN + ("dout",) else x) for n, x in t.items()}
    o, S = forward(e)
    assert o.numel() == 0 and torch.equal(S, t["S0"])
    got = backward(e)
    assert torch.equal(got[5], t["dS"])
    del e["S0"], e["dS"]
    assert (forward(e)[1] == 0).all()
    none = {n: x[:0].contiguous() for n, x in t.items()}
    assert forward(none)[0].shape == (0, 2, 3, 64)


def test_workspace_status_and_refusals():
    t = on_gpu(make(1, 1, 2, 40, 64, 64, "bf16", seed=1))
    n = api.fwd_gated_delta_workspace_bytes(1, 1, 2, 40, 64, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o = torch.empty_like(t["v"])
    api.kata_fwd_gated_delta(*(t[x] for x in IN), o, workspace=ws)
    assert api.kata_workspace_status(ws) == KATA_OK
    with pytest.raises(KataError):
        api.kata_fwd_gated_delta(*(t[x] for x in IN), o, workspace=ws[:-256].contiguous()[:256])
    with pytest.raises(KataError):
        api.kata_fwd_gated_delta(*(t[x] for x in IN), o, S0=t["S0"], S_out=t["S0"])
    with pytest.raises(ValueError):
        api.kata_fwd_gated_delta(t["q"].transpose(2, 3), t["k"].transpose(2, 3), t["v"], t["g"], t["beta"], o)
    wide = torch.zeros(1, 1, 40, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        api.kata_fwd_gated_delta(wide[..., :64], wide[..., :64], t["v"], t["g"], t["beta"], o)
