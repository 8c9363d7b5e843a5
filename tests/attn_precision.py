"""How far gdn_attn may be off in bf16 io, from what the header promises of its weights and queries; and problems that
fewer bits would fail."""
import math

import torch

import attn_reference as R


def attend(q, k, codes, scales, n, causal, scale, tile, hp=2.0 ** -11):
    """q [n, Hq, D] over k [kv, Hk, D] and values codes [kv, Hk, D] times scales [kv, Hk], all in 64 bits: the output
    and how far from it the library may be.

    A rounding to fp16 is off by at most 2^-11 of the value, or 2^-25 below its normal numbers; p stands in it with its
    page's value scale, times the power that brings the largest of these products to 2^11 or more: with w_j = p_j s_j,
        sum_j (2^-11 w_j + 2^-36 max_j w_j) |code_j|.
    A score is a sum of D products in fp32, off by (D + 8) 2^-24 of the sum A of their sizes; for tiles of 128 rows
    each element of q below 2^-8 of its row's largest is off by 2^-17 of that largest besides (above it, it is exact; for
    few rows the bits that fp16 has keep any element to 2^-39 of the largest): E in all.  Differences to a running
    maximum, with the logarithm of a scale in them (127 in size at most), are rounded to fp32 some four times: 2^-24 of A
    and of 127.  The exponential is good to 2^-22.  Each enters a weight as a factor, on the token and on the sum:
        2 (E + 4 2^-24 (A + 127) + 2^-22) sum_j w_j |code_j|,   twice over for the higher orders.
    Sums over L tokens in fp32: 2 (L + 8) 2^-24 of sum_j w_j |code_j|.  One rounding of the output: 2^-8 of it."""
    q, k = q.double(), k.double()
    Hq, Hk, kv, D = q.shape[1], k.shape[1], k.shape[0], q.shape[2]
    head = torch.arange(Hq, device=q.device) // (Hq // Hk)
    k, c, s = k[:, head], codes.double()[:, head], scales.double()[:, head]
    x = torch.einsum("nhd,khd->hnk", q, k) * scale
    A = (torch.einsum("nhd,khd->hnk", q.abs(), k.abs()) * abs(scale)).amax(-1)
    top = q.abs().amax(-1, keepdim=True)
    lost = torch.where(q.abs() < 2.0 ** -8 * top, torch.ones_like(q), torch.zeros_like(q)) if tile else torch.ones_like(q)
    E = (torch.einsum("nhd,khd->hnk", lost, k.abs()).amax(-1) * abs(scale)) * top[..., 0].T * 2.0 ** (-17 if tile else -39)
    E = E + (D + 8) * 2.0 ** -24 * A
    seen = torch.ones(n, kv, dtype=torch.bool, device=q.device)
    if causal:
        seen = torch.arange(kv, device=q.device)[None] <= (kv - n + torch.arange(n, device=q.device))[:, None]
    p = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
    p = torch.where(seen.any(-1)[None, :, None], p, torch.zeros_like(p))
    w = p * s.T[:, None]                                                    # [Hq, n, kv]
    o, S = torch.einsum("hnk,khd->hnd", w, c), torch.einsum("hnk,khd->hnd", w, c.abs())
    size = torch.einsum("hnk,khd->hnd", seen.double()[None].expand(Hq, n, kv), c.abs())
    tol = (hp + 4 * (E + 4 * 2.0 ** -24 * (A + 127) + 2.0 ** -22) + 2 * (kv + 8) * 2.0 ** -24)[..., None] * S
    tol = tol + 2.0 ** -36 * w.amax(-1)[..., None] * size + 2.0 ** -8 * o.abs()
    return o.transpose(0, 1), tol.transpose(0, 1)


def rounded(q, k, codes, scales, n, scale, weights):
    """The output with unnormalised weights, at most 1, times scales over the largest product, through `weights`; the rest
    in 64 bits (causal)."""
    q, k = q.double(), k.double()
    Hq, Hk, kv = q.shape[1], k.shape[1], k.shape[0]
    head = torch.arange(Hq, device=q.device) // (Hq // Hk)
    x = torch.einsum("nhd,khd->hnk", q, k[:, head]) * scale
    seen = torch.arange(kv)[None] <= (kv - n + torch.arange(n))[:, None]
    x = x.masked_fill(~seen, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    s = scales.double()[:, head].T[:, None]
    return torch.einsum("hnk,khd->nhd", weights(p, s), codes.double()[:, head]) / p.sum(-1).T[..., None]


def parts(cache, b, kv):
    """Keys in 64 bits, values' codes and their scales of sequence b, [kv, Hk, ..]."""
    k, _ = cache.rows(b, kv)
    p = cache.table[b, :-(-kv // cache.page)].long()
    codes = cache.v8.view(torch.float8_e4m3fn)[p].double().transpose(1, 2).reshape(-1, cache.Hk, cache.D)[:kv]
    return k, codes, cache.sv[p].double().repeat_interleave(cache.page, 0)[:kv]


def weights_against_scales(n, D, lead, drop, device="cpu", kv=None, late=True):
    """A page whose tokens have nearly all the weight and a value scale 2^-lead, and one of scale 1 whose weights are
    2^-drop of theirs, behind it (or before): with drop well above lead the first page's values are the output, although
    the second's are 2^lead times larger.  -> cache, q (4 heads on 2) and the scale of the scores."""
    kv = kv or 48 + n
    c = R.Cache([kv], 2, D, 16, device=device).fill(mean=0.0)
    t = c.table[0].long()
    c.k8[t] = 0
    far = t[1] if late else t[0]
    g = torch.Generator().manual_seed(lead)
    for p in t:                                       # what is heavy: about 1 in each dimension, so drop in powers of 2; else 0
        about = 1 + 0.125 * torch.randint(-1, 2, c.k8.shape[1:], generator=g)
        c.k8[p] = 0 if p == far else about.to(torch.float8_e4m3fn).view(torch.uint8).to(device)
    c.sk[t] = 1.0
    c.sv[t] = 2.0 ** -lead
    c.sv[far] = 1.0
    q = torch.full((n, 4 * D), 1.0, device=device).bfloat16()
    return c, q, drop * math.log(2.0) / D
