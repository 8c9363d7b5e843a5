"""The workloads of linear attention with decay and of the fused projections.

Two operators around the mixer, each with a plain form in elementary torch
operations (``own = False``) and the library's entry points (``own = True``):

  linear attention with a log decay g per value head (value head h reads key
  head h // (Hv // Hk)), state S [Dv][Dk]:
      S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
    "prefill": T tokens of B sequences from S0 (fixed length, or packed back
    to back); "decode": T new tokens from the cached state, in place.
    g is given per token ("token") or is a constant of the head ("head").

  projections p[t, n] = sum_k x[t, k] w[n, k] + bias[n] with, per output
  column range, an activation and a residual:  y = act(p) + residual, and the
  gated form  y[t, n] = act(p[t, n]) p[t, N/2 + n] + residual  (n < N/2).
"""
import math
import random

import torch

own = False
D = 128  # head width


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # Single-user generation, one token through a 16-head layer with the
        # constant per-head decays: all latency.
        dict(name="decode 1x16 heads", op="decode", B=1, T=1, Hk=16, Hv=16, gate="head", io="bf16"),
        # Batched generation at the 16/48-head shape: streams 805 MB of state.
        dict(name="decode 256x48 heads", op="decode", B=256, T=1, Hk=16, Hv=48, gate="token", io="bf16"),
        # Four drafted tokens per sequence verified from the cache.
        dict(name="decode 4 tokens 64x48", op="decode", B=64, T=4, Hk=16, Hv=48, gate="token", io="bf16"),
        # A batch of long prompts at the 16/32-head shape.
        dict(name="prefill 4x8192 32 heads", op="prefill", B=4, T=8192, Hk=16, Hv=32, gate="token", io="bf16"),
        # One very long prompt: few (sequence, head) pairs, a thousand chunks.
        dict(name="prefill 1x65536 48 heads", op="prefill", B=1, T=65536, Hk=16, Hv=48, gate="head", io="bf16"),
        # A serving batch of prompts of ragged lengths, packed back to back.
        dict(name="prefill packed 24 seqs", op="packed", B=24, T=4000, lens_seed=7, Hk=16, Hv=32, gate="token", io="bf16"),
        # fp32 tensors (checks, small models): fp32 arithmetic throughout.
        dict(name="prefill fp32 2x1001", op="prefill", B=2, T=1001, Hk=4, Hv=8, gate="token", io="f32"),
        # One token through the in-projection (q|k and gate columns activated).
        dict(name="linear 1 token 5120-16480", op="linear", M=1, K=5120, N=16480, bias=True, ranges="in_proj"),
        # A decode batch through the out-projection, added to the residual stream.
        dict(name="linear 64 tokens 6144-5120", op="linear", M=64, K=6144, N=5120, bias=False, ranges="residual"),
        # Prompts through the in-projection: tensor-core bound.
        dict(name="linear 8192 tokens 5120-16480", op="linear", M=8192, K=5120, N=16480, bias=True, ranges="in_proj"),
        # The gated feed-forward's first product, gate and up in one call.
        dict(name="gated 2048 tokens 5120-24576", op="linear", M=2048, K=5120, N=24576, bias=False, ranges="gated"),
        # Odd sizes: ragged tiles on every side, rows that are not 16-byte aligned.
        dict(name="linear odd 777x1000x519", op="linear", M=777, K=1000, N=519, bias=True, ranges="residual"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("decode", "prefill", "packed", "linear", "linear"))
    if op == "linear":
        ranges = rng.choice(("in_proj", "residual", "gated"))
        M, K = _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 768)
        N = _log_int(rng, 16, 16480)
        if ranges == "gated":
            N += N % 2
        return dict(op="linear", M=M, K=K, N=N, bias=rng.random() < 0.5, ranges=ranges)
    Hk = rng.choice((1, 2, 4, 8, 16))
    Hv = Hk * rng.choice((1, 2, 3))
    gate = rng.choice(("token", "head"))
    if op == "decode":
        B = _log_int(rng, 1, 256)
        T = rng.choice((1, 1, 1, 2, 3, 4, 5, 8))
        return dict(op=op, B=B if T == 1 else max(1, B // 4), T=T, Hk=Hk, Hv=Hv, gate=gate,
                    io=rng.choice(("bf16", "bf16", "f32")))
    if op == "packed":
        return dict(op=op, B=rng.randint(2, 24), T=_log_int(rng, 64, 4000), lens_seed=rng.randint(1, 1 << 20), Hk=Hk,
                    Hv=Hv, gate=gate, io="bf16")
    if rng.random() < 0.2:
        return dict(op=op, B=rng.randint(1, 4), T=_log_int(rng, 16, 1024), Hk=min(Hk, 4), Hv=min(Hk, 4) * (Hv // Hk),
                    gate=gate, io="f32")
    B = rng.choice((1, 1, 2, 3, 4))
    return dict(op=op, B=B, T=_log_int(rng, 17, 32768 // B), Hk=Hk, Hv=Hv, gate=gate, io="bf16")


def _lengths(case):
    """Ragged lengths of a packed batch: log-uniform, the last token counts of real prompts."""
    r = random.Random(case["lens_seed"])
    return [_log_int(r, max(1, case["T"] // 40), case["T"]) for _ in range(case["B"])]


def _ranges(case):
    """(col_begin, col_end, activation, residual?) of the outputs of a projection."""
    N, kind = case["N"], case["ranges"]
    if kind == "gated":
        return [(0, N // 2, "silu", False)]
    if kind == "residual":
        return [(0, N, "none", True)]
    a, b = (N * 2 // 8) // 8 * 8, (N * 5 // 8) // 8 * 8   # q|k, v, output gate
    return [r for r in ((0, a, "silu", False), (a, b, "none", False), (b, N, "sigmoid", False)) if r[0] < r[1]]


def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        out = sum((e - b) * M * 2 * (2 if res else 1) for b, e, _, res in _ranges(case))
        return {"bytes": 2 * K * (M + N) + out + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    e = 2 if case["io"] == "bf16" else 4
    Hk, Hv = case["Hk"], case["Hv"]
    tokens = sum(_lengths(case)) if case["op"] == "packed" else case["B"] * case["T"]
    state = case["B"] * Hv * D * D * 4
    gates = tokens * Hv * 4 if case["gate"] == "token" else Hv * 4
    # per token and head: one rank-1 update and one product of the state with a vector
    return {"bytes": tokens * (2 * Hk + 2 * Hv) * D * e + 2 * state + gates, "flops": 4 * tokens * Hv * D * D}


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = torch.randn(M, K, device=dev, generator=g).bfloat16()
        w = (torch.randn(N, K, device=dev, generator=g) / math.sqrt(K)).bfloat16()
        bias = (0.1 * torch.randn(N, device=dev, generator=g)).bfloat16() if case["bias"] else None
        outs = [(b, e, torch.empty(M, e - b, device=dev, dtype=torch.bfloat16), act,
                 torch.randn(M, e - b, device=dev, generator=g).bfloat16() if res else None)
                for b, e, act, res in _ranges(case)]
        return dict(case=case, x=x, w=w, bias=bias, outs=outs)
    B, T, Hk, Hv = case["B"], case["T"], case["Hk"], case["Hv"]
    dt = torch.bfloat16 if case["io"] == "bf16" else torch.float32
    packed = case["op"] == "packed"
    lens = _lengths(case) if packed else None
    rows = sum(lens) if packed else B * T
    # one fused q|k|v buffer, q and k behind a SiLU as the in-projection leaves them
    qkv = torch.randn(rows, (2 * Hk + Hv) * D, device=dev, generator=g, dtype=dt)
    qk = qkv[:, :2 * Hk * D]
    qk.copy_(torch.nn.functional.silu(qk))
    lead = (rows,) if packed else (B, T)
    qkv = qkv.view(*lead, -1)
    st = dict(case=case, q=qkv[..., :Hk * D], k=qkv[..., Hk * D:2 * Hk * D], v=qkv[..., 2 * Hk * D:],
              o=torch.empty(*lead, Hv * D, device=dev, dtype=dt), g=None, log_decay=None)
    if case["gate"] == "token":
        st["g"] = -torch.nn.functional.softplus(-(3.0 + torch.randn(*lead, Hv, device=dev, generator=g)))
    else:  # a geometric ladder of decays over the heads
        st["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, Hv + 1, device=dev, dtype=torch.float32) / Hv)
    S = 0.02 * torch.randn(B, Hv, D, D, device=dev, generator=g)
    if case["op"] == "decode":
        st["S"] = S
    else:
        st["S0"], st["S_T"] = S, torch.empty_like(S)
    if packed:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    return st


# ----------------------------------------------------------------- plain form
def _act(p, act):
    return p * torch.sigmoid(p) if act == "silu" else torch.sigmoid(p) if act == "sigmoid" else p


def _plain_linear(st):
    p = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        p = p + st["bias"].float()
    out = []
    for b, e, y, act, res in st["outs"]:
        v = _act(p[:, b:e], act)
        if st["case"]["ranges"] == "gated":
            v = v * p[:, e:2 * e]
        if res is not None:
            v = v + res.float()
        out.append(v.to(y.dtype))
    return out


def _heads(st, lead):
    """q, k (expanded to the value heads), v as [B, Hv, T, D] fp32 and g as [B, Hv, T] (64 bits: long sums)."""
    c = st["case"]
    Hk, Hv = c["Hk"], c["Hv"]
    B, T = lead
    q, k, v = (st[n].reshape(B, T, -1, D).float().transpose(1, 2) for n in "qkv")
    q, k = (x.repeat_interleave(Hv // Hk, dim=1) for x in (q, k))
    g = st["g"].reshape(B, T, Hv) if st["g"] is not None else st["log_decay"].expand(B, T, Hv)
    return q, k, v, g.transpose(1, 2).double()


def _plain_chunked(q, k, v, g, S):
    """The recurrence over chunks: inside a chunk one masked product, between chunks the carried state."""
    B, H, T, _ = q.shape
    C = min(256, max(16, 1 << max(0, T - 1).bit_length()))
    n = -(-T // C)
    pad = n * C - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, C, D) for x in (q, k, v))
    G = torch.nn.functional.pad(g, (0, pad)).view(B, H, n, C).cumsum(-1)
    last = G[..., -1:]
    R = (G[..., :, None] - G[..., None, :]).float()
    R = torch.exp(R.masked_fill_(torch.ones(C, C, dtype=torch.bool, device=q.device).triu(1), -math.inf))
    o = (q @ k.transpose(-1, -2) * R) @ v
    upd = (v * torch.exp(last - G).float()[..., None]).transpose(-1, -2) @ k      # [B, H, n, Dv, Dk]
    d = torch.exp(last[..., 0]).float()
    before = torch.empty_like(upd)
    for i in range(n):  # the state before each chunk
        before[:, :, i] = S
        S = d[:, :, i, None, None] * S + upd[:, :, i]
    o = o + (q * torch.exp(G).float()[..., None]) @ before.transpose(-1, -2)
    return o.reshape(B, H, n * C, D)[:, :, :T], S


def _plain_linattn(st):
    c, scale = st["case"], 1.0 / math.sqrt(D)
    B, T, Hv = c["B"], c["T"], c["Hv"]
    if c["op"] == "decode":
        q, k, v, g = _heads(st, (B, T))
        o = torch.empty_like(v)
        S = st["S"]
        a = torch.exp(g).float()
        for t in range(T):
            S.mul_(a[:, :, t, None, None]).add_(v[:, :, t, :, None] * k[:, :, t, None, :])
            o[:, :, t] = (S @ q[:, :, t, :, None])[..., 0]
        return (o * scale).transpose(1, 2).reshape(B, T, Hv * D).to(st["o"].dtype), S
    if c["op"] == "prefill":
        q, k, v, g = _heads(st, (B, T))
        o, S = _plain_chunked(q, k, v, g, st["S0"])
        return (o * scale).transpose(1, 2).reshape(B, T, Hv * D).to(st["o"].dtype), S
    # packed: rows gathered into a [B, longest] rectangle; rows past a sequence's end add nothing
    cu = st["cu"].long()
    n = cu[1:] - cu[:-1]
    at = torch.arange(max(_lengths(c)), device=cu.device)
    inside = at[None, :] < n[:, None]
    row = (cu[:-1, None] + at[None, :]).clamp_(max=st["q"].shape[0] - 1)
    part = dict(case=c, log_decay=st["log_decay"], g=None if st["g"] is None else st["g"][row],
                **{x: st[x][row] * inside[..., None].to(st[x].dtype) for x in "qkv"})
    q, k, v, g = _heads(part, tuple(row.shape))
    o, S = _plain_chunked(q, k, v, g * inside[:, None, :], st["S0"])
    return (o * scale).transpose(1, 2).reshape(*row.shape, Hv * D)[inside].to(st["o"].dtype), S


# ------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "linear":
            return _plain_linear(state)
        o, S = _plain_linattn(state)
        return {"o": o, "S": S}
    from gated_deltanet_mixer_gb300 import gdn

    if case["op"] == "linear":
        gdn.gdn_linear_ex(state["x"], state["w"], state["outs"], bias=state["bias"], gated=case["ranges"] == "gated")
        return [o[2] for o in state["outs"]]
    if case["op"] == "decode":
        gdn.gdn_linattn_decode(state["q"], state["k"], state["v"], state["S"], state["o"], Hk=case["Hk"], Hv=case["Hv"],
                               g=state["g"], log_decay=state["log_decay"])
        return {"o": state["o"], "S": state["S"]}
    if "ws" not in state:  # the scratch that a program keeps across its calls
        B, T, packed = case["B"], case["T"], case["op"] == "packed"
        state["ws"] = torch.empty(gdn.gdn_linattn_workspace_bytes(B, state["q"].shape[0] if packed else T, case["Hk"], case["Hv"],
                                                                  packed=packed), dtype=torch.uint8, device="cuda")
    gdn.gdn_linattn_prefill(state["q"], state["k"], state["v"], state["S0"], state["o"], state["S_T"], Hk=case["Hk"],
                            Hv=case["Hv"], g=state["g"], log_decay=state["log_decay"], cu_seqlens=state.get("cu"),
                            workspace=state["ws"])
    return {"o": state["o"], "S": state["S_T"]}


# ------------------------------------------------------- the definition, fp64
def _recur(q, k, v, g, S):
    """The token loop in 64 bits: q, k, v [T, units, D], g [T, units], S [units, Dv, Dk]; o, S."""
    o = torch.empty_like(v)
    a = g.exp()[..., None, None]
    for t in range(q.shape[0]):
        S = S * a[t]
        S.baddbmm_(v[t][:, :, None], k[t][:, None, :])
        torch.bmm(S, q[t][:, :, None], out=o[t][:, :, None])
    return o / math.sqrt(D), S


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        p = st["x"].double() @ st["w"].double().T
        if st["bias"] is not None:
            p += st["bias"].double()
        res = []
        for b, e, _, act, r in st["outs"]:
            y = p[:, b:e]
            if act == "silu":
                y = y / (1 + torch.exp(-y))
            elif act == "sigmoid":
                y = 1 / (1 + torch.exp(-y))
            if case["ranges"] == "gated":
                y = y * p[:, e:]
            res.append(y if r is None else y + r.double())
        return res
    B, Hk, Hv = case["B"], case["Hk"], case["Hv"]
    S0 = st["S" if case["op"] == "decode" else "S0"].double()
    r = Hv // Hk

    def part(rows, S, seqs, T):  # rows: token rows of `seqs` sequences of T tokens
        f = {}
        for n, H in (("q", Hk), ("k", Hk), ("v", Hv)):
            x = st[n].reshape(-1, H, D)[rows].double().view(seqs, T, H, D)
            x = x if n == "v" else x[:, :, torch.arange(Hv, device=x.device) // r]
            f[n] = x.transpose(0, 1).reshape(T, seqs * Hv, D).contiguous()
        g = st["log_decay"].double().expand(seqs, T, Hv) if st["g"] is None else st["g"].reshape(-1, Hv)[rows].double().view(seqs, T, Hv)
        o, S = _recur(f["q"], f["k"], f["v"], g.transpose(0, 1).reshape(T, seqs * Hv), S.reshape(seqs * Hv, D, D))
        return o.view(T, seqs, Hv * D).transpose(0, 1).reshape(seqs * T, Hv * D), S.view(seqs, Hv, D, D)

    if case["op"] != "packed":
        o, S = part(slice(None), S0, B, case["T"])
        return {"o": o.view(B, case["T"], Hv * D), "S": S}
    os_, Ss, at = [], [], 0
    for s, n in enumerate(_lengths(case)):
        o, S = part(slice(at, at + n), S0[s:s + 1], 1, n)
        os_.append(o)
        Ss.append(S)
        at += n
    return {"o": torch.cat(os_), "S": torch.cat(Ss)}
