"""Softmax attention over a paged 8-bit cache, appending to it and rotary
positions, from their formulas in 64 bits; and problems for their tests."""
import math

import torch

E4M3_MAX = 448.0


def e4m3(x):
    """The nearest e4m3 value (1 sign, 4 exponent, 3 fraction bits, bias 7), ties to even, saturated."""
    x = x.double().clamp(-E4M3_MAX, E4M3_MAX)
    _, e = torch.frexp(x)
    q = ((torch.clamp(e.long() - 4, min=-9) + 1023) << 52).view(torch.float64)  # 2^.., from its bits
    return torch.round(x / q) * q


def scale_for(amax):
    """The smallest power of two s in [2^-120, 2^7] with amax <= 448 s, NaN where amax is not finite."""
    s = torch.full_like(amax, 2.0 ** -120, dtype=torch.float64)
    for _ in range(127):
        s = torch.where(amax > E4M3_MAX * s, 2 * s, s)
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, math.nan))


class Cache:
    """Pages on one device: bytes, scales, tables of `lens` tokens, pages in random order."""

    def __init__(self, lens, Hk, D, page, seed=0, device="cpu", fill=0x7f, extra=3, blocks=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.page, self.Hk, self.D, self.lens = page, Hk, D, list(lens)
        order = torch.randperm(sum(need) + extra, generator=g).to(torch.int32)
        width = blocks or max(1, max(need))
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        P = order.numel()
        # what no token has written: NaN bytes, and NaN scales where no page is used
        self.k8 = torch.full((P, Hk, page, D), fill, dtype=torch.uint8)
        self.v8 = self.k8.clone()
        self.sk = torch.full((P, Hk), math.nan)
        self.sv = self.sk.clone()
        self.to(device)

    def to(self, device):
        for n in ("table", "k8", "v8", "sk", "sv"):
            setattr(self, n, getattr(self, n).to(device))
        self.kv = torch.tensor(self.lens, dtype=torch.int32, device=device)
        return self

    def args(self):
        return self.kv, self.table, self.k8, self.v8, self.sk, self.sv

    def fill(self, seed=1, mean=0.5):
        """Random keys and values in every token of the sequences."""
        g = torch.Generator().manual_seed(seed)
        for b, n in enumerate(self.lens):
            for j in range(-(-n // self.page)):
                p, m = int(self.table[b, j]), min(self.page, n - j * self.page)
                for c8, s, mu in ((self.k8, self.sk, mean), (self.v8, self.sv, 0.0)):
                    x = torch.randn(self.Hk, m, self.D, generator=g) + mu * torch.sin(torch.arange(self.D) * 1.7)
                    s[p] = 2.0 ** torch.randint(-8, -4, (self.Hk,), generator=g).float()
                    c8[p, :, :m] = (x / s[p].cpu()[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(
                        torch.uint8).to(c8.device)
        return self

    def rows(self, b, n):
        """k, v [n, Hk, D] of sequence b in 64 bits."""
        out = []
        for c8, s in ((self.k8, self.sk), (self.v8, self.sv)):
            x = c8.view(torch.float8_e4m3fn).double() * s.double()[:, :, None, None]
            p = self.table[b, :-(-n // self.page)].long()
            out.append(x[p].transpose(1, 2).reshape(-1, self.Hk, self.D)[:n])
        return out


def attend(q, k, v, n, causal, scale):
    """q [n, Hq, D] over k, v [kv, Hk, D], the new tokens the last n: o, sum_j p_j |v_j|, and the largest
    scale sum_d |q_d k_d| of a row (what rounding errors of scores grow with)."""
    q, k, v = q.double(), k.double(), v.double()
    Hq, Hk, kv = q.shape[1], k.shape[1], k.shape[0]
    head = torch.arange(Hq, device=q.device) // (Hq // Hk)
    k, v = k[:, head], v[:, head]
    s = torch.einsum("nhd,khd->hnk", q, k) * scale
    size = (torch.einsum("nhd,khd->hnk", q.abs(), k.abs()) * abs(scale)).amax(-1) if kv else s.new_zeros(Hq, n)
    seen = torch.ones(n, kv, dtype=torch.bool, device=q.device)
    if causal:
        seen = torch.arange(kv, device=q.device)[None] <= (kv - n + torch.arange(n, device=q.device))[:, None]
    s = s.masked_fill(~seen, -math.inf)
    p = torch.softmax(s, -1) if kv else s
    p = torch.where(seen.any(-1)[None, :, None], p, torch.zeros_like(p))
    return torch.einsum("hnk,khd->nhd", p, v), torch.einsum("hnk,khd->nhd", p, v.abs()), size.T


def least(cache, b, n, kv, Hq, causal):
    """What bf16 io may be off by however small a weight is: weights stand in fp16 with the page's value scale as
    a factor, so that the row's largest weight so far under the largest scale so far (2^-100 at least) is 2^11 or more,
    and fp16 rounds to within 2^-25: 2^-36 of that weight and scale for each token's value over its scale.  The sum of
    weights that they are divided by is no less than the row's largest weight."""
    p = cache.table[b, :-(-kv // cache.page)].long()
    codes = cache.v8.view(torch.float8_e4m3fn)[p].double().abs().nan_to_num(0.0).transpose(1, 2).reshape(-1, cache.Hk, cache.D)[:kv]
    scales = cache.sv[p].double().nan_to_num(0.0).clamp(min=2.0 ** -100).repeat_interleave(cache.page, 0)[:kv]
    x = 2.0 ** -36 * scales.cummax(0).values[:, :, None] * codes.cumsum(0) if kv else codes
    last = torch.full((n,), kv - 1) if not causal else kv - n + torch.arange(n)
    x = torch.cat((torch.zeros_like(x[:1]) if kv else codes.new_zeros(1, cache.Hk, cache.D), x))
    return x[(last + 1).clamp(min=0).to(x.device)].repeat_interleave(Hq // cache.Hk, 1)


def append(k, v, cache, lens, new):
    """The cache behind new tokens k, v (lists of [n, Hk, D] per sequence), in place, in 64 bits."""
    for b, (kv, n) in enumerate(zip(lens, new)):
        start = kv - n
        if n == 0:
            continue
        for x, c8, s in ((k[b], cache.k8, cache.sk), (v[b], cache.v8, cache.sv)):
            for j in range(start // cache.page, -(-kv // cache.page)):
                lo, hi = max(start, j * cache.page), min(kv, (j + 1) * cache.page)
                p, at = int(cache.table[b, j]), lo - j * cache.page
                part = x[lo - start:hi - start].double().transpose(0, 1)     # [Hk, rows, D]
                amax = part.abs().amax((1, 2))
                need = scale_for(torch.where(torch.isnan(part).any(2).any(1), torch.full_like(amax, math.inf), amax))
                old = s[p].double()
                scale = need if at == 0 else torch.where(need.isnan() | old.isnan(), torch.full_like(need, math.nan),
                                                         torch.maximum(need, old))
                by = c8[p].view(torch.float8_e4m3fn).double()
                if at:
                    anew = e4m3(by[:, :at] * (old / scale)[:, None, None])
                    by[:, :at] = torch.where((scale > old)[:, None, None], anew, by[:, :at])
                fresh = e4m3(part / scale[:, None, None])
                by[:, at:at + hi - lo] = torch.where(scale.isnan()[:, None, None], torch.zeros_like(fresh), fresh)
                now = by[:, :at + hi - lo].float().to(torch.float8_e4m3fn).view(torch.uint8)
                c8[p, :, :at + hi - lo] = now
                s[p] = scale.float()


def frequencies(rot, base, scaling=None):
    i = torch.arange(rot // 2, dtype=torch.float64)
    if not scaling:
        return base ** (-2 * i / rot), 1.0
    kind, factor = scaling["kind"], scaling["factor"]
    if kind == "linear":
        return base ** (-2 * i / rot) / factor, 1.0
    if kind == "ntk":
        return (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    f = base ** (-2 * i / rot)

    def c(n):
        return rot * math.log(scaling["original"] / (2 * math.pi * n)) / (2 * math.log(base))

    lo, hi = max(math.floor(c(scaling.get("fast", 32))), 0), min(math.ceil(c(scaling.get("slow", 1))), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1


def rope(x, positions, rot, D, f, m, layout, inverse=False):
    """x [tokens, heads * D] turned, in 64 bits."""
    x = x.double().unflatten(-1, (-1, D)).clone()
    a = positions.double()[:, None] * f.to(positions.device)
    cos, sin = (m * torch.cos(a))[:, None], (m * torch.sin(a) * (-1 if inverse else 1))[:, None]
    ia = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    u, w = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = u * cos - w * sin, w * cos + u * sin
    return x.flatten(-2)
