"""Cases of the gated delta rule: the chunked forward, its gradient and the
one-token step, timed against their plain form in elementary torch operations.

Per value head, with a state S [d_k, d_v] and per token a log decay g <= 0 and
a write strength beta:
    S_t = exp(g_t) S_(t-1) + k_t d_t^T,  d_t = beta_t (v_t - exp(g_t) S_(t-1)^T k_t)
    o_t = S_t^T q_t
Query / key head h // (heads / key_heads) serves value head h.
"""

import math

import torch

own = False

CHUNK = 64                      # tokens a chunk of the plain form
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, dtype, B, key_heads, heads, T, d_k, d_v, state):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "key_heads": key_heads,
            "heads": heads, "T": T, "d_k": d_k, "d_v": d_v, "state": state}


def listed():
    return [
        # the shortest prompt: one head, where launches and latency count
        _case("forward, tiny, f32", "forward", "f32", 1, 1, 1, 256, 16, 16, True),
        # one layer of a training step's forward: many sequences, many heads
        _case("forward, layer, bf16", "forward", "bf16", 8, 16, 16, 2048, 64, 64, False),
        # a long document in one sequence: few heads, a long carry
        _case("forward, 131k, bf16", "forward", "bf16", 1, 16, 16, 131072, 128, 128, True),
        # prompts continued from a state, shared key heads, an odd length
        _case("forward, shared keys, bf16", "forward", "bf16", 3, 4, 12, 1237, 128, 64, True),
        # full precision, a batch of ordinary sequences
        _case("forward, batch, f32", "forward", "f32", 4, 8, 8, 1023, 64, 64, True),
        # the gradient of one layer of a training step
        _case("gradient, layer, bf16", "backward", "bf16", 4, 8, 8, 4096, 64, 64, False),
        # the gradient of a longer sequence with wide heads and shared keys
        _case("gradient, long, bf16", "backward", "bf16", 1, 8, 16, 16384, 128, 128, True),
        # full precision, shared keys, an odd length
        _case("gradient, shared keys, f32", "backward", "f32", 2, 2, 4, 333, 32, 64, True),
        # serving: one token for one sequence, where latency counts
        _case("step, one sequence, bf16", "step", "bf16", 1, 8, 16, 1, 128, 128, True),
        # serving: one token for a full batch
        _case("step, batch 256, bf16", "step", "bf16", 256, 16, 16, 1, 128, 128, True),
        # serving in full precision, an odd batch
        _case("step, batch 37, f32", "step", "f32", 37, 8, 8, 1, 64, 64, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("forward", "backward", "step"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    key_heads, group = _log_int(rng, 1, 16), rng.choice((1, 1, 2, 3, 4))
    d_k, d_v = rng.choice(((64, 64), (128, 128), (128, 64), (64, 128), (32, 64), (16, 32), (128, 16)))
    if op == "step":
        B, T = _log_int(rng, 1, 256), 1
        B = max(1, min(B, 4096 // (key_heads * group)))
    else:
        B, T = _log_int(rng, 1, 8), _log_int(rng, 1, 16384 if op == "forward" else 8192)
        B = max(1, min(B, 2 ** 18 // (key_heads * group * T)))
    state = op == "step" or rng.random() < 0.5
    return {"op": op, "dtype": dtype, "B": B, "key_heads": key_heads, "heads": key_heads * group,
            "T": T, "d_k": d_k, "d_v": d_v, "state": state}


def _inputs(case, seed):
    """Unit-length queries and keys, a tenth of the keys repeats of an earlier
    one (bindings that are written again), decays from slow to fast heads, and
    write strengths as a sigmoid gives them."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    B, Hk, H, T, d_k, d_v = (case[n] for n in ("B", "key_heads", "heads", "T", "d_k", "d_v"))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).sqrt()

    dt = TYPES[case["dtype"]]
    q, k, v = unit(normal(B, Hk, T, d_k)), unit(normal(B, Hk, T, d_k)), normal(B, H, T, d_v)
    if T > 8:
        earlier = torch.randint(0, T, (T,), generator=gen, device="cuda") % torch.arange(1, T + 1, device="cuda")
        again = torch.rand(T, generator=gen, device="cuda") < 0.1
        k = torch.where(again[:, None], k[:, :, earlier], k)
    rate = torch.exp(torch.rand(H, 1, generator=gen, device="cuda") * math.log(64.0)) / 64
    g = -rate * torch.log1p(torch.exp(normal(B, H, T)))
    beta = 1 / (1 + torch.exp(-normal(B, H, T)))
    s = {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "g": g, "beta": beta}
    if case["state"]:
        s["S0"] = 0.3 * normal(B, H, d_k, d_v)
    if case["op"] == "backward":
        s["dout"] = normal(B, H, T, d_v).to(dt)
        if case["state"]:
            s["dS"] = 0.3 * normal(B, H, d_k, d_v)
    if case["op"] == "step":
        for n in ("q", "k", "v", "g", "beta"):
            s[n] = s[n][:, :, 0].contiguous()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"], s["start"] = case["op"], s.get("S0")
    return s


def run(state):
    s = state
    if own:
        from kernelized_linear_attention_kata_b200 import api
        if s["op"] == "forward":
            if s["start"] is None:
                return {"o": api.fwd_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"])}
            o, S = api.fwd_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], S0=s["start"],
                                       return_state=True)
            return {"o": o, "S": S}
        if s["op"] == "backward":
            names = ("dq", "dk", "dv", "dg", "dbeta", "dS0")
            got = api.bwd_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"],
                                      S0=s["start"], dS=s.get("dS"))
            return {n: x for n, x in zip(names, got) if x is not None}
        o = api.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["start"])
        return {"o": o, "S": s["start"]}           # updated in place
    if s["op"] == "forward":
        return _forward(s)
    if s["op"] == "backward":
        return _backward(s)
    return _step(s)


def _step(s):
    group = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    S = s["start"] * torch.exp(s["g"])[..., None, None]
    d = s["beta"][..., None] * (s["v"].float() - (k[..., None, :] @ S)[..., 0, :])
    s["start"] = S = S + k[..., :, None] * d[..., None, :]
    return {"o": (q[..., None, :] @ S)[..., 0, :].to(s["v"].dtype), "S": S}


def _chunked(x, N):
    """[B, H, T, ...] as N chunks [B, H, N, CHUNK, ...], zeros behind the end."""
    B, H, T = x.shape[:3]
    full = x.new_zeros((B, H, N * CHUNK) + tuple(x.shape[3:]))
    full[:, :, :T] = x
    return full.reshape((B, H, N, CHUNK) + tuple(x.shape[3:]))


def _unit_lower_inverse(L):
    """(I + L)^-1 of strictly lower triangular L: diagonal blocks of doubling
    size, inv [[A, 0], [X, B]] = [[A', 0], [-B' X A', B']]."""
    i = torch.arange(CHUNK, device=L.device)
    M = torch.eye(CHUNK, device=L.device).expand_as(L)
    for b in (1, 2, 4, 8, 16, 32):
        corner = (i[:, None] // (2 * b) == i[None, :] // (2 * b)) & (i[:, None] // b > i[None, :] // b)
        M = M - M @ (L * corner) @ M
    return M


def _chunk_terms(s):
    """What the chunks have before their starting state is known, in 32 bits
    (the sums of log decays and their differences in 64)."""
    group, T = s["v"].shape[1] // s["q"].shape[1], s["v"].shape[2]
    N = -(-T // CHUNK)
    t = {"N": N, "T": T, "group": group}
    t["q"], t["k"] = (_chunked(s[n].float(), N).repeat_interleave(group, 1) for n in ("q", "k"))
    t["v"], t["beta"] = _chunked(s["v"].float(), N), _chunked(s["beta"], N)[..., None]
    G = _chunked(s["g"], N).double().cumsum(-1)
    i = torch.arange(CHUNK, device=G.device)
    causal = i[:, None] >= i[None, :]
    t["decay"] = torch.exp(torch.where(causal, G[..., :, None] - G[..., None, :], -math.inf)).float()
    t["from_start"] = torch.exp(G).float()[..., None]
    t["to_end"] = torch.exp(G[..., -1:] - G).float()[..., None]
    t["whole"] = t["from_start"][..., -1:, :]
    t["kk"] = t["k"] @ t["k"].mT
    t["L"] = torch.tril(t["beta"] * t["decay"] * t["kk"], -1)
    t["M"] = _unit_lower_inverse(t["L"])
    t["P"] = (t["q"] @ t["k"].mT) * t["decay"]
    return t


def _states(s, t):
    """Each chunk's starting state and its tokens' writes, and the last state."""
    B, H, d_k, d_v = t["v"].shape[0], t["v"].shape[1], t["k"].shape[-1], t["v"].shape[-1]
    mv, mk = t["M"] @ (t["beta"] * t["v"]), t["M"] @ (t["beta"] * t["from_start"] * t["k"])
    k_end = (t["to_end"] * t["k"]).mT
    S = s["start"] if s["start"] is not None else mv.new_zeros(B, H, d_k, d_v)
    starts, writes = mv.new_empty(B, H, t["N"], d_k, d_v), torch.empty_like(mv)
    for n in range(t["N"]):
        starts[:, :, n] = S
        writes[:, :, n] = mv[:, :, n] - mk[:, :, n] @ S
        S = t["whole"][:, :, n] * S + k_end[:, :, n] @ writes[:, :, n]
    return starts, writes, S


def _flat(x, t):
    B, H, N, C = x.shape[:4]
    return x.reshape((B, H, N * C) + tuple(x.shape[4:]))[:, :, :t["T"]]


def _forward(s):
    t = _chunk_terms(s)
    starts, writes, S = _states(s, t)
    o = _flat(t["from_start"] * (t["q"] @ starts) + t["P"] @ writes, t).to(s["v"].dtype)
    return {"o": o} if s["start"] is None else {"o": o, "S": S}


def _backward(s):
    t = _chunk_terms(s)
    starts, writes, _ = _states(s, t)
    do = _chunked(s["dout"].float(), t["N"])
    q, k, beta, M, P, decay = (t[n] for n in ("q", "k", "beta", "M", "P", "decay"))
    q_start, k_start, k_end = t["from_start"] * q, t["from_start"] * k, t["to_end"] * k
    # the gradient of each chunk's last state, last chunk first
    dS = s["dS"] if "dS" in s else torch.zeros_like(starts[:, :, 0])
    p_do, q_do, m_t, k_t = P.mT @ do, q_start.mT @ do, beta * M.mT, k_start.mT
    ends, d_v = torch.empty_like(starts), torch.empty_like(writes)
    for n in reversed(range(t["N"])):
        ends[:, :, n] = dS
        d_v[:, :, n] = m_t[:, :, n] @ (p_do[:, :, n] + k_end[:, :, n] @ dS)
        dS = t["whole"][:, :, n] * dS + q_do[:, :, n] - k_t[:, :, n] @ d_v[:, :, n]
    # d_v = beta dR, R = beta (v - k_start S) and writes = M R
    d_r = M.mT @ (p_do + k_end @ ends)
    miss = t["v"] - k_start @ starts
    d_P = do @ writes.mT
    d_L = -torch.tril(d_r @ writes.mT, -1)
    d_qk, d_kk = d_P * decay, d_L * beta * decay
    d_q_start, d_k_start, d_k_end = do @ starts.mT, -d_v @ starts.mT, writes @ ends.mT
    dq = t["from_start"] * d_q_start + d_qk @ k
    dk = t["from_start"] * d_k_start + t["to_end"] * d_k_end + d_qk.mT @ q + (d_kk + d_kk.mT) @ k
    dbeta = (d_r * miss).sum(-1) + (d_L * decay * t["kk"]).sum(-1)
    to_end = (k_end * d_k_end).sum(-1)
    pairs = d_P * P + d_L * t["L"]
    dG = (q_start * d_q_start + k_start * d_k_start).sum(-1) - to_end + pairs.sum(-1) - pairs.sum(-2)
    last = to_end.sum(-1) + t["whole"][..., 0, 0] * (starts * ends).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1) + last[..., None]
    dq, dk = (_flat(x.unflatten(1, (-1, t["group"])).sum(2), t).to(s["q"].dtype) for x in (dq, dk))
    out = {"dq": dq, "dk": dk, "dv": _flat(d_v, t).to(s["v"].dtype), "dg": _flat(dg, t),
           "dbeta": _flat(dbeta, t)}
    if s["start"] is not None:
        out["dS0"] = dS
    return out


def work(case):
    B, Hk, H, T, d_k, d_v = (case[n] for n in ("B", "key_heads", "heads", "T", "d_k", "d_v"))
    e = 2 if case["dtype"] == "bf16" else 4
    qk, v, gates, S = B * Hk * T * d_k * e, B * H * T * d_v * e, B * H * T * 4, B * H * d_k * d_v * 4
    if case["op"] == "backward":
        # q, k, v, dout and the gates in, five gradients out; the state is rebuilt (2 products with
        # it a token), its gradient carried (2), and 4 more give dq, dk and the write's gradient
        n = 4 * qk + 3 * v + 4 * gates + (3 * S if case["state"] else 0)
        return {"bytes": n, "flops": 16 * B * H * T * d_k * d_v}
    # the state is read with the key, written to, and read with the query
    states = 2 * S if case["state"] else 0
    return {"bytes": 2 * qk + 2 * v + 2 * gates + states, "flops": 6 * B * H * T * d_k * d_v}


def exact(case, seed):
    """The definition, token by token, in 64 bits; the gradient by its adjoint,
    last token first."""
    s = _inputs(case, seed)
    group = case["heads"] // case["key_heads"]
    T, step = case["T"], case["op"] == "step"
    if step:
        s.update({n: s[n].unsqueeze(2) for n in ("q", "k", "v", "g", "beta")})
    B, H, d_k, d_v = case["B"], case["heads"], case["d_k"], case["d_v"]

    def by_time(x, repeat=1):                       # [T, B * H, ...]
        x = x.double().repeat_interleave(repeat, 1)
        return x.permute(2, 0, 1, *range(3, x.dim())).reshape((T, B * H) + tuple(x.shape[3:])).contiguous()

    def by_head(x):
        x = x.reshape((T, B, H) + tuple(x.shape[2:]))
        return x.permute(1, 2, 0, *range(3, x.dim())).contiguous()

    q, k = by_time(s["q"], group), by_time(s["k"], group)
    v, beta, a = by_time(s["v"]), by_time(s["beta"])[..., None], torch.exp(by_time(s["g"]))[..., None, None]
    S = s["S0"].double().reshape(B * H, d_k, d_v).clone() if "S0" in s else \
        torch.zeros(B * H, d_k, d_v, dtype=torch.float64, device="cuda")
    grad = case["op"] == "backward"
    o = torch.empty_like(v)
    before = torch.empty((T,) + tuple(S.shape), dtype=S.dtype, device="cuda") if grad else None
    rows, cols = k[:, :, None, :], k[..., None]
    for i in range(T):
        if grad:
            before[i] = S
        S *= a[i]
        d = torch.baddbmm(v[i][:, None], rows[i], S, alpha=-1).mul_(beta[i][:, None])
        S.baddbmm_(cols[i], d)
        if not grad:
            torch.bmm(q[i][:, None], S, out=o[i][:, None])
    if not grad:
        out = {"o": by_head(o)}
        if case["state"]:
            out["S"] = S.reshape(B, H, d_k, d_v)
        if step:
            out["o"] = out["o"][:, :, 0]
        return out
    do = by_time(s["dout"])
    dS = s["dS"].double().reshape(B * H, d_k, d_v) if "dS" in s else torch.zeros_like(S)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = (torch.empty(T, B * H, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in reversed(range(T)):
        decayed = before[i] * a[i]
        miss = v[i][:, None] - rows[i] @ decayed                     # [B H, 1, d_v]
        d = beta[i][:, None] * miss
        after = decayed + cols[i] @ d
        dq[i] = (after @ do[i][..., None])[..., 0]
        dS = dS + q[i][..., None] @ do[i][:, None]
        dd = rows[i] @ dS
        db[i] = (dd * miss).sum((-1, -2))
        du = beta[i][:, None] * dd
        dv[i] = du[:, 0]
        dk[i] = (dS @ d.mT - decayed @ du.mT)[..., 0]
        dS = dS - cols[i] @ du
        dg[i] = (decayed * dS).sum((-1, -2))
        dS = dS * a[i]
    dq, dk = (by_head(x).unflatten(1, (-1, group)).sum(2) for x in (dq, dk))
    out = {"dq": dq, "dk": dk, "dv": by_head(dv), "dg": by_head(dg), "dbeta": by_head(db)}
    if case["state"]:
        out["dS0"] = dS.reshape(B, H, d_k, d_v)
    return out
