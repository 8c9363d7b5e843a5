"""The workloads of softmax attention over a paged cache in 8 bits, and of what fills it.

Four operators, each with a plain form in elementary torch operations
(``own = False``) and the library's entry points (``own = True``):

  "pages"   block tables, slots and positions from request lengths: request b
      with kv cached and n new tokens owns ceil((kv + n) / page) pages; the ones
      it lacks come from the free list, requests in order.
  "rope"    rotary positions on the first `rot` of D elements of every head:
      the pair (a, b) at position p becomes m (a cos - b sin, b cos + a sin) of
      the angle p f_i, f_i = base^(-2i/rot), possibly scaled.
  "append"  new keys and values into pages of e4m3 values with a power of two
      as scale for each page and head: the smallest s with max |x| <= 448 s over
      the page's tokens, and not below the stored one where the page holds older
      tokens (which are expressed anew in the scale that holds).
  "attn"    o_i = sum_j softmax_j(scale q_i . k_j) v_j over the cached tokens j
      up to the query's own position; query head h reads key head h // (Hq // Hk).
"""
import math
import random

import numpy as np
import torch

own = False
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One decoding step of a batch: a token each, now and then a new page.
        dict(name="pages 64 requests, 1 token", op="pages", B=64, new=1, kv=4096, page=16, seed=1),
        # Many prompts admitted at once: tables and slots of some 20,000 tokens.
        dict(name="pages 512 prompts", op="pages", B=512, new=160, kv=64, page=16, seed=2),
        # One token of the 24/4-head attention layer, 64 of 256 dimensions rotated: all latency.
        dict(name="rope 1 token 24+4 heads", op="rope", tokens=1, Hq=24, Hk=4, D=256, rot=64, layout="half",
             scaling="none", far=4096, io="bf16", in_place=True),
        # A prompt through the same layer, in place in the projection's output.
        dict(name="rope 8192 tokens 24+4 heads", op="rope", tokens=8192, Hq=24, Hk=4, D=256, rot=64, layout="half",
             scaling="none", far=131072, io="bf16", in_place=True),
        # Whole heads in the interleaved layout, fp32, positions far out with frequencies scaled by parts.
        dict(name="rope 1003 tokens interleaved fp32", op="rope", tokens=1003, Hq=12, Hk=3, D=128, rot=128,
             layout="interleaved", scaling="parts", far=1 << 20, io="f32", in_place=False),
        # One decoding step of a batch: a token each into half-filled pages.
        dict(name="append 64 x 1 token", op="append", B=64, new=1, kv=2000, Hk=4, D=256, page=16, seed=3, io="bf16"),
        # Prompts of ragged lengths behind cached prefixes.
        dict(name="append 12 prompts", op="append", B=12, new=4000, kv=500, Hk=4, D=256, page=16, seed=4, io="bf16"),
        # Single-user generation: one token over a few thousand cached ones.
        dict(name="attn 1 x 1 over 4096", op="attn", B=1, new=1, kv=4096, Hq=24, Hk=4, D=256, page=16, ragged=False,
             seed=5, io="bf16"),
        # Batched generation: streams 1.07 GB of cache.
        dict(name="attn 64 x 1 over 8192", op="attn", B=64, new=1, kv=8192, Hq=24, Hk=4, D=256, page=16, ragged=False,
             seed=6, io="bf16"),
        # Four drafted tokens per sequence verified, lengths ragged.
        dict(name="attn 16 x 4 ragged", op="attn", B=16, new=4, kv=16000, Hq=32, Hk=8, D=128, page=32, ragged=True,
             seed=7, io="bf16"),
        # A long prompt's last chunk over what is cached of it: tensor-core bound.
        dict(name="attn 8192 over 24576", op="attn", B=1, new=8192, kv=24576, Hq=24, Hk=4, D=256, page=16, ragged=False,
             seed=8, io="bf16"),
        # A serving batch of prompts of ragged odd lengths, packed back to back.
        dict(name="attn 12 prompts packed", op="attn", B=12, new=2000, kv=700, Hq=16, Hk=2, D=128, page=64, ragged=True,
             seed=9, io="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    limit = max(work(c)["flops"] for c in listed()), max(work(c)["bytes"] for c in listed())
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= limit[0] and w["bytes"] <= limit[1]:
            return c


def _draw(rng):
    op = rng.choice(("pages", "rope", "append", "attn", "attn", "attn"))
    page = rng.choice((16, 16, 32, 64, 128))
    seed = rng.randint(10, 1 << 20)
    D = rng.choice((64, 128, 256))
    Hk = rng.choice((1, 2, 3, 4, 8))
    Hq = Hk * rng.choice((1, 2, 3, 4, 6, 8))
    io = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "pages":
        return dict(op=op, B=_log_int(rng, 1, 512), new=rng.choice((1, 4, _log_int(rng, 1, 160))),
                    kv=_log_int(rng, 1, 4096), page=page, seed=seed)
    if op == "rope":
        scaling = rng.choice(("none", "linear", "ntk", "parts"))
        return dict(op=op, tokens=_log_int(rng, 1, 8192), Hq=Hq, Hk=Hk, D=D, rot=rng.choice((D // 4, D // 2, D)),
                    layout=rng.choice(("half", "interleaved")), scaling=scaling, far=_log_int(rng, 4096, 1 << 20),
                    io=io, in_place=scaling != "parts" and rng.random() < 0.5)
    if op == "append":
        return dict(op=op, B=_log_int(rng, 1, 64), new=rng.choice((1, 3, _log_int(rng, 1, 4000))),
                    kv=_log_int(rng, 1, 4000), Hk=Hk, D=D, page=page, seed=seed, io=io)
    if io == "f32":  # checks, small models
        return dict(op=op, B=rng.randint(1, 4), new=_log_int(rng, 1, 64), kv=_log_int(rng, 1, 2000), Hq=Hq, Hk=Hk, D=D,
                    page=page, ragged=True, seed=seed, io=io)
    if rng.random() < 0.5:
        return dict(op=op, B=_log_int(rng, 1, 64), new=rng.choice((1, 1, 1, 2, 4, 7)), kv=_log_int(rng, 1, 32768), Hq=Hq,
                    Hk=Hk, D=D, page=page, ragged=rng.random() < 0.7, seed=seed, io=io)
    return dict(op=op, B=rng.randint(1, 8), new=_log_int(rng, 8, 8192), kv=_log_int(rng, 1, 24576), Hq=Hq, Hk=Hk, D=D,
                page=page, ragged=rng.random() < 0.7, seed=seed, io=io)


def _lengths(case):
    """(cached, new) tokens of each request; ragged ones spread log-uniformly below the case's numbers."""
    r = random.Random(case["seed"])
    B, kv, new = case["B"], case["kv"], case["new"]
    if case["op"] == "attn" and not case["ragged"]:
        return [(kv, new)] * B
    few = case["op"] == "attn" and new < 8 or new == 1  # a decoding step: as many new tokens each
    return [(_log_int(r, max(1, kv // 20), kv), new if few else _log_int(r, max(1, new // 20), new)) for _ in range(B)]


def _element(case):
    return 2 if case["io"] == "bf16" else 4


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * (case["Hq"] + case["Hk"])
        width = case["rot"] if case["in_place"] else case["D"]
        return {"bytes": 2 * n * width * _element(case) + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    lens = _lengths(case)
    tokens = sum(n for _, n in lens)
    if op == "pages":
        pages = sum(-(-(kv + n) // case["page"]) + -kv // case["page"] for kv, n in lens)
        # lengths, new counts, new lengths, offsets; slot and position of a token; page out of the list into the table
        return {"bytes": 16 * case["B"] + 12 * tokens + 8 * pages, "flops": 4 * tokens}
    if op == "append":
        return {"bytes": 2 * tokens * case["Hk"] * case["D"] * (_element(case) + 1), "flops": 6 * tokens * case["Hk"] * case["D"]}
    e, Hq, Hk, D = _element(case), case["Hq"], case["Hk"], case["D"]
    seen = sum(n * kv + n * (n + 1) // 2 for kv, n in lens)
    blocks = sum(-(-(kv + n) // case["page"]) for kv, n in lens)
    cache = sum(kv + n for kv, n in lens) * Hk * D * 2 + blocks * (Hk * 8 + 4)
    return {"bytes": cache + 2 * tokens * Hq * D * e, "flops": 4 * seen * Hq * D}


# --------------------------------------------------------------------- inputs
def _cu(lens):
    cu = [0]
    for _, n in lens:
        cu.append(cu[-1] + n)
    return cu


def _scaling(case):
    return {"none": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=4.0),
            "parts": dict(kind="parts", factor=8.0, original=32768, fast=32.0, slow=1.0)}[case["scaling"]]


def _pow2(e):
    """2^e of 32-bit numbers, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [pages, Hk, page, D] as e4m3 values and the power of two of each page and head."""
    amax = x.abs().amax(dim=(2, 3)).float()
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    s = _pow2(e)
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)
    op = case["op"]
    dt = torch.float32 if case.get("io") == "f32" else torch.bfloat16

    def rand(*shape, dtype=torch.float32):
        return torch.randn(*shape, device=dev, generator=g, dtype=dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if op == "rope":
        Hq, Hk, D, T = case["Hq"], case["Hk"], case["D"], case["tokens"]
        qkv = rand(T, (Hq + 2 * Hk) * D, dtype=dt)  # q, k: views of the projection's output
        first = torch.randint(0, max(1, case["far"] - T), (1,), device=dev, generator=g)
        st = dict(case=case, q=qkv[:, :Hq * D], k=qkv[:, Hq * D:(Hq + Hk) * D],
                  pos=(first + torch.arange(T, device=dev)).to(torch.int32))
        st["qo"], st["ko"] = (st["q"], st["k"]) if case["in_place"] else (torch.empty(T, Hq * D, device=dev, dtype=dt),
                                                                          torch.empty(T, Hk * D, device=dev, dtype=dt))
        if own:
            from gated_deltanet_mixer_gb300 import gdn
            st["plan"] = gdn.gdn_rope_plan(case["rot"], base=1e6, layout=case["layout"], scaling=_scaling(case))
        return st
    lens, page = _lengths(case), case["page"]
    B, cu = len(lens), _cu(lens)
    tokens = cu[-1]
    blocks = [-(-(kv + n) // page) for kv, n in lens]
    width = max(blocks)
    order = torch.randperm(sum(blocks) + 5, device=dev, generator=g).to(torch.int32)  # pages, scattered as in a long-running server
    if op == "pages":
        have = [-(-kv // page) for kv, _ in lens]
        table, at = np.full((B, width), -1, dtype=np.int32), 0
        pages = order.cpu().numpy()
        for b, n in enumerate(have):
            table[b, :n] = pages[at:at + n]
            at += n
        return dict(case=case, kv=ints([kv for kv, _ in lens]), new=ints([n for _, n in lens]),
                    free=torch.from_numpy(pages[at:].copy()).to(dev), used=ints([0]),
                    table=torch.from_numpy(table).to(dev), kv_out=ints([0] * B), used_out=ints([0]), cu=ints([0] * (B + 1)),
                    slots=torch.empty(tokens, dtype=torch.int64, device=dev),
                    positions=torch.empty(tokens, dtype=torch.int32, device=dev))
    table, at = torch.full((B, width), -1, dtype=torch.int32, device=dev), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    P, Hk, D = order.numel(), case["Hk"], case["D"]
    st = dict(case=case, table=table, cu=ints(cu), kv=ints([kv + n for kv, n in lens]), max_new=max(n for _, n in lens),
              max_kv=max(kv + n for kv, n in lens))
    # heads differ in size, pages a little; a head's keys share a mean, as real ones do
    size = torch.exp2(rand(1, Hk, 1, 1)).to(torch.bfloat16)
    mean = rand(1, Hk, 1, D, dtype=torch.bfloat16) * 0.5
    for n in "kv":
        x = rand(P, Hk, page, D, dtype=torch.bfloat16)
        if n == "k" and op == "attn":
            x += mean
        x *= size
        st[n + "8"], st["s" + n] = torch.empty(P, Hk, page, D, dtype=torch.float8_e4m3fn, device=dev), torch.empty(P, Hk, device=dev)
        for lo in range(0, P, 4096):
            st[n + "8"][lo:lo + 4096], st["s" + n][lo:lo + 4096] = _quantise(x[lo:lo + 4096])
        del x
    if op == "append":
        kv_rows = rand(tokens, 2 * Hk * D, dtype=dt) * 2.0
        st["k"], st["v"] = kv_rows[:, :Hk * D], kv_rows[:, Hk * D:]
        return st
    Hq = case["Hq"]
    r = Hq // Hk
    # queries of the size that makes scores of a few units
    st["q"] = ((1.5 * rand(tokens, Hk, r, D)) / size.view(1, Hk, 1, 1)).reshape(tokens, Hq * D).to(dt)
    st["o"] = torch.empty(tokens, Hq * D, device=dev, dtype=dt)
    return st


# ----------------------------------------------------------------- plain form
def _plain_pages(st):
    page = st["case"]["page"]
    kv, new = st["kv"].long(), st["new"].long()
    n = kv + new
    need, have = (n + page - 1) // page, (kv + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have) + st["used"].long()
    j = torch.arange(st["table"].shape[1], device=kv.device)
    fresh = (j[None] >= have[:, None]) & (j[None] < need[:, None])
    at = (first[:, None] + j[None] - have[:, None]).clamp_(0, st["free"].numel() - 1)
    table = torch.where(fresh, st["free"][at], st["table"])
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    t = torch.arange(st["slots"].numel(), device=kv.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = kv[b] + t - cu[b]
    slots = table[b, pos // page].long() * page + pos % page
    return dict(table=table, kv=n.to(torch.int32), used=(st["used"] + (need - have).sum()).to(torch.int32),
                cu=cu.to(torch.int32), slots=slots, positions=pos.to(torch.int32))


def _frequencies(case, dev):
    """The pairs' frequencies in 64 bits, and the factor on cosine and sine."""
    rot, s, base = case["rot"], _scaling(case), 1e6
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    if s is None:
        return base ** (-2 * i / rot), 1.0
    if s["kind"] == "linear":
        return base ** (-2 * i / rot) / s["factor"], 1.0
    if s["kind"] == "ntk":
        return (base * s["factor"] ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0

    def pair(turns):  # the pair that makes so many turns over the original context
        return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(s["fast"])), 0), min(math.ceil(pair(s["slow"])), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    f = base ** (-2 * i / rot)
    return f * (1 - ramp) + f / s["factor"] * ramp, 0.1 * math.log(s["factor"]) + 1


def _plain_rope(st):
    c = st["case"]
    rot, D = c["rot"], c["D"]
    f, m = _frequencies(c, st["pos"].device)
    angle = st["pos"].double()[:, None] * f
    cos, sin = (torch.cos(angle) * m).float()[:, None], (torch.sin(angle) * m).float()[:, None]
    for x, y in ((st["q"], st["qo"]), (st["k"], st["ko"])):
        h = x.unflatten(1, (-1, D))
        if c["layout"] == "half":
            a, b = h[..., :rot // 2].float(), h[..., rot // 2:rot].float()
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = h[..., 0:rot:2].float(), h[..., 1:rot:2].float()
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        out = y.unflatten(1, (-1, D))
        out[..., :rot] = r.to(y.dtype)
        if not c["in_place"]:
            out[..., rot:] = h[..., rot:]
    return st["qo"], st["ko"]


def _touched(st):
    """(request, block) of the pages that a call writes, and where the old and new tokens of each lie."""
    page, pairs = st["case"]["page"], []
    for b, (kv, n) in enumerate(_lengths(st["case"])):
        pairs += [(b, j, kv, kv + n) for j in range(kv // page, -(-(kv + n) // page))]
    return torch.tensor(pairs, device=st["cu"].device)


def _plain_append(st):
    c = st["case"]
    page, Hk, D = c["page"], c["Hk"], c["D"]
    b, j, kv, end = _touched(st).unbind(1)
    pages = st["table"][b, j].long()
    pos = j[:, None] * page + torch.arange(page, device=b.device)
    new, old = (pos >= kv[:, None]) & (pos < end[:, None]), pos < kv[:, None]
    row = (st["cu"].long()[b, None] + pos - kv[:, None]).clamp_(0, st["k"].shape[0] - 1)
    for x, c8, s in ((st["k"], st["k8"], st["sk"]), (st["v"], st["v8"], st["sv"])):
        h = x[row].unflatten(2, (Hk, D)).float().transpose(1, 2)                       # [units, Hk, page, D]
        fresh, kept = new[:, None, :, None], old[:, None, :, None]
        m, e = torch.frexp((h * fresh).abs().amax(dim=(2, 3)))
        need = _pow2(e - 9 + (m > 0.875).to(e.dtype))
        before = s[pages]
        scale = torch.where(old.any(1)[:, None], torch.maximum(need, before), need)
        was = c8[pages].float()
        again = (was * (before / scale)[:, :, None, None]).to(torch.float8_e4m3fn).float()
        now = (h / scale[:, :, None, None]).to(torch.float8_e4m3fn).float()
        c8[pages] = torch.where(fresh, now, torch.where(kept, again, was)).to(torch.float8_e4m3fn)
        s[pages] = scale
    return dict(k=st["k8"], v=st["v8"], sk=st["sk"], sv=st["sv"])


def _rows(st, b, n, dtype):
    """The n cached keys and values of request b, [Hk, n, D]."""
    page = st["case"]["page"]
    p = st["table"][b, :-(-n // page)].long()
    return ((c8[p].to(dtype) * s[p].to(dtype)[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
            for c8, s in ((st["k8"], st["sk"]), (st["v8"], st["sv"])))


def _plain_attn(st, dtype=torch.float32):
    c = st["case"]
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    out = torch.empty_like(st["q"]) if dtype == torch.float32 else torch.empty_like(st["q"], dtype=dtype)
    at = 0
    for b, (kv, n) in enumerate(_lengths(c)):
        k, v = _rows(st, b, kv + n, dtype)
        step = max(1, min(n, (1 << 28) // (Hq * (kv + n))))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            q = st["q"][at + lo:at + hi].to(dtype).view(hi - lo, Hk, Hq // Hk, D).permute(1, 2, 0, 3)  # [Hk, r, rows, D]
            s = q.reshape(Hk, -1, D) @ k.transpose(1, 2) / math.sqrt(D)
            s = s.view(Hk, Hq // Hk, hi - lo, kv + n)
            hidden = torch.arange(kv + n, device=s.device)[None] > (kv + torch.arange(lo, hi, device=s.device))[:, None]
            s.masked_fill_(hidden, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = p.view(Hk, -1, kv + n) @ v / p.sum(-1).view(Hk, -1, 1)
            out[at + lo:at + hi] = o.view(Hk, Hq // Hk, hi - lo, D).permute(2, 0, 1, 3).reshape(hi - lo, Hq * D).to(out.dtype)
        at += n
    return out


# ------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"pages": _plain_pages, "rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](state)
    from gated_deltanet_mixer_gb300 import gdn

    st = state
    if op == "pages":
        gdn.gdn_kv_pages(st["kv"], st["new"], st["free"], st["used"], st["table"], st["kv_out"], st["used_out"], st["cu"],
                         st["slots"], st["positions"], page=st["case"]["page"])
        return dict(table=st["table"], kv=st["kv_out"], used=st["used_out"], cu=st["cu"], slots=st["slots"],
                    positions=st["positions"])
    if op == "rope":
        gdn.gdn_rope(st["plan"], st["pos"], [(st["q"], st["qo"]), (st["k"], st["ko"])], D=st["case"]["D"])
        return st["qo"], st["ko"]
    if op == "append":
        gdn.gdn_kv_append(st["k"], st["v"], st["kv"], st["table"], st["k8"], st["v8"], st["sk"], st["sv"],
                          cu_seqlens=st["cu"], max_new=st["max_new"])
        return dict(k=st["k8"], v=st["v8"], sk=st["sk"], sv=st["sv"])
    if "ws" not in st:  # the scratch that a program keeps across its calls
        st["ws"] = torch.empty(gdn.gdn_attn_workspace_bytes(len(st["kv"]), st["q"].shape[0], st["case"]["Hq"],
                                                            st["case"]["Hk"], st["case"]["D"], max_new=st["max_new"],
                                                            max_kv=st["max_kv"]), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn(st["q"], st["o"], st["kv"], st["table"], st["k8"], st["v8"], st["sk"], st["sv"], Hq=st["case"]["Hq"],
                 cu_seqlens=st["cu"], max_new=st["max_new"], max_kv=st["max_kv"], workspace=st["ws"])
    return st["o"]


# ------------------------------------------------------- the definition, fp64
def _e4m3(x):
    """x to the nearest value of 1 sign, 4 exponent and 3 fraction bits (bias 7), ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    q = ((torch.clamp(e.long() - 4, min=-9) + 1023) << 52).view(torch.float64)
    return torch.round(x / q) * q


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pages":
        table, slots, positions = st["table"].cpu().numpy().copy(), [], []
        free, used, page = st["free"].cpu().tolist(), 0, case["page"]
        for b, (kv, n) in enumerate(_lengths(case)):
            for pos in range(kv, kv + n):
                if pos % page == 0:
                    table[b, pos // page] = free[used]
                    used += 1
                slots.append(int(table[b, pos // page]) * page + pos % page)
                positions.append(pos)
        lens = _lengths(case)
        return dict(table=torch.from_numpy(table), kv=torch.tensor([kv + n for kv, n in lens], dtype=torch.int32),
                    used=torch.tensor([used], dtype=torch.int32), cu=torch.tensor(_cu(lens), dtype=torch.int32),
                    slots=torch.tensor(slots), positions=torch.tensor(positions, dtype=torch.int32))
    if op == "rope":
        f, m = _frequencies(case, st["pos"].device)
        turn = torch.polar(torch.full((), m, device=f.device, dtype=torch.float64), st["pos"].double()[:, None] * f)[:, None]
        res = []
        for x in (st["q"], st["k"]):
            h = x.double().unflatten(1, (-1, case["D"])).clone()
            part = h[..., :case["rot"]]
            z = part.unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (-1, 2))
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            h[..., :case["rot"]] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
            res.append(h.flatten(1))
        return tuple(res)
    if op == "append":
        page, Hk, D = case["page"], case["Hk"], case["D"]
        res, at = {}, 0
        for n in "kv":
            res[n], res["s" + n] = st[n + "8"].double(), st["s" + n].double()
        for b, (kv, new) in enumerate(_lengths(case)):
            blocks = list(range(kv // page, -(-(kv + new) // page)))
            pages = st["table"][b, blocks[0]:blocks[-1] + 1].long()
            lead = kv - blocks[0] * page                                  # old tokens in the first block
            pad = len(blocks) * page - lead - new
            for n in "kv":
                x = st[n][at:at + new].double().view(new, Hk, D)
                x = torch.nn.functional.pad(x, (0, 0, 0, 0, lead, pad)).view(len(blocks), page, Hk, D).transpose(1, 2)
                val = res[n][pages] * res["s" + n][pages][:, :, None, None]
                amax = x.abs().amax(dim=(2, 3))
                s = torch.exp2(torch.floor(torch.log2(amax)) - 9)             # at most half of what is wanted
                for _ in range(3):
                    s = torch.where(s * E4M3_MAX < amax, 2 * s, s)
                if lead:
                    s[0] = torch.maximum(s[0], res["s" + n][pages[0]])
                    x[0, :, :lead] = val[0, :, :lead]
                y = _e4m3(x / s[:, :, None, None])
                if pad:
                    y[-1, :, page - pad:] = res[n][pages[-1], :, page - pad:]
                res[n][pages], res["s" + n][pages] = y, s
            at += new
        return res
    return _exact_attn(st)


def _exact_attn(st):
    """Each query block against the whole cache in 64 bits, by log-sum-exp."""
    c = st["case"]
    Hq, Hk, D, page = c["Hq"], c["Hk"], c["D"], c["page"]
    res, at = [], 0
    for b, (kv, n) in enumerate(_lengths(c)):
        p = st["table"][b, :-(-(kv + n) // page)].long()
        cached = []
        for c8, s in ((st["k8"], st["sk"]), (st["v8"], st["sv"])):
            x = c8[p].double().mul_(s[p].double()[:, :, None, None])     # [blocks, Hk, page, D]
            cached.append(x.permute(1, 0, 2, 3).reshape(Hk, -1, D))
        where = torch.arange(cached[0].shape[1], device=p.device)
        o = torch.empty(n, Hq, D, device=p.device, dtype=torch.float64)
        step = max(1, min(n, (1 << 27) // where.numel()))
        for h in range(Hq):
            k, v = (x[h // (Hq // Hk)] for x in cached)
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                q = st["q"][at + lo:at + hi, h * D:(h + 1) * D].double()
                last = (kv + torch.arange(lo, hi, device=p.device))[:, None]
                s = torch.where(where[None] <= last, q @ k.T * D ** -0.5, -math.inf)
                o[lo:hi, h] = torch.exp(s - torch.logsumexp(s, 1, keepdim=True)) @ v
        res.append(o.view(n, Hq * D))
        at += n
    return torch.cat(res)
