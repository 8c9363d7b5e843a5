"""A decoder layer of softmax attention over the paged 8-bit cache, on the library's operators: the layer that stands
between the linear ones of a hybrid decoder.

    python -m gated_deltanet_mixer_gb300.attn_layer --hidden 2048 --ffn 6144 --Hq 8 --Hk 2 --D 256 --rot 64 --T 1000 --new 4

Per step, for n_b new tokens of each of B requests, x [tokens, hidden] of the residual stream, packed:

    tables, offsets, positions   pages for the new tokens                gdn_kv_pages
    q | k | v = x W_in^T         one product, views of one buffer        gdn_linear_ex
    q, k                         turned in place                         gdn_rope
    cache     += k, v            e4m3, a scale per page and head         gdn_kv_append
    o         = attention        over all of a request's tokens          gdn_attn
    x        += o W_out^T        added in place                          gdn_linear_ex
    f         = silu(x W_g^T) (x W_u^T)                                  gdn_linear_ex, gated
    x        += f W_d^T          added in place                          gdn_linear_ex

(The norms in front of the two halves, those of q and k that such layers have ahead of the rotation, and the gate on o
are left out: the library has no call for them.)  Lengths and tables stay on the GPU: a step of
single tokens can be captured into a graph and replayed.  Run as a program it takes prompts of ragged lengths, then
single tokens from a captured graph, and checks them against the same tokens taken as one prompt.
"""
import argparse
import math

import torch

from . import gdn


class PagedCache:
    """Pages of one layer, the free list, and the tables and lengths of B requests."""

    def __init__(self, B, Hk, D, pages, page=16, max_blocks=None, device="cuda"):
        self.B, self.Hk, self.D, self.page = B, Hk, D, page
        self.k, self.v = (torch.zeros(pages, Hk, page, D, dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
        self.sk, self.sv = (torch.zeros(pages, Hk, device=device) for _ in range(2))
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.zeros(B, max_blocks or pages, **i32)
        self.kv_lens, self.used, self.free = torch.zeros(B, **i32), torch.zeros(1, **i32), torch.arange(pages, **i32)

    def args(self):
        return self.kv_lens, self.table, self.k, self.v, self.sk, self.sv


class AttnLayer:
    """Weights, the cache, and the buffers of a step kept across calls."""

    def __init__(self, hidden, ffn, Hq, Hk, D, rot, cache, base=1e6, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(rows, cols):
            return (torch.randn(rows, cols, device=device, generator=g) / math.sqrt(cols)).bfloat16()

        self.hidden, self.ffn, self.Hq, self.Hk, self.D, self.cache = hidden, ffn, Hq, Hk, D, cache
        self.w_in, self.w_out = w((Hq + 2 * Hk) * D, hidden), w(hidden, Hq * D)
        self.w_gate_up, self.w_down = w(2 * ffn, hidden), w(hidden, ffn)
        self.plan = gdn.gdn_rope_plan(rot, base=base)
        self.ws = torch.empty(0, dtype=torch.uint8, device=device)

    def step(self, tokens, max_new, max_kv=0):
        """Buffers for steps of up to `tokens` new tokens, up to max_new of a request, each request's tokens max_kv at most."""
        dev, B = self.ws.device, self.cache.B
        i32 = dict(dtype=torch.int32, device=dev)
        need = gdn.gdn_attn_workspace_bytes(B, tokens, self.Hq, self.Hk, self.D, max_new=max_new, max_kv=max_kv)
        if self.ws.numel() < need:
            self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        return dict(cu=torch.zeros(B + 1, **i32), positions=torch.zeros(tokens, **i32), max_new=max_new, max_kv=max_kv,
                    slots=torch.zeros(tokens, dtype=torch.int64, device=dev), ws=self.ws,
                    qkv=torch.empty(tokens, (self.Hq + 2 * self.Hk) * self.D, **bf),
                    o=torch.zeros(tokens, self.Hq * self.D, **bf), f=torch.empty(tokens, self.ffn, **bf))

    def forward(self, x, new_tokens, s):
        """x [tokens, hidden] bf16, updated in place; new_tokens [B] int32 on the device; s from step()."""
        c, q_cols, kv_cols = self.cache, self.Hq * self.D, self.Hk * self.D
        gdn.gdn_kv_pages(c.kv_lens, new_tokens, c.free, c.used, c.table, c.kv_lens, c.used, s["cu"], s["slots"], s["positions"],
                         page=c.page)
        gdn.gdn_linear_ex(x, self.w_in, [(0, q_cols + 2 * kv_cols, s["qkv"])])
        q, k, v = s["qkv"].split([q_cols, kv_cols, kv_cols], 1)
        gdn.gdn_rope(self.plan, s["positions"], [(q, q), (k, k)], D=self.D)
        gdn.gdn_kv_append(k, v, *c.args(), cu_seqlens=s["cu"], max_new=s["max_new"], max_kv=s["max_kv"])
        gdn.gdn_attn(q, s["o"], *c.args(), Hq=self.Hq, cu_seqlens=s["cu"], max_new=s["max_new"], max_kv=s["max_kv"],
                     workspace=s["ws"])
        gdn.gdn_linear_ex(s["o"], self.w_out, [(0, self.hidden, x, "none", x)])
        gdn.gdn_linear_ex(x, self.w_gate_up, [(0, self.ffn, s["f"], "silu")], gated=True)
        gdn.gdn_linear_ex(s["f"], self.w_down, [(0, self.hidden, x, "none", x)])
        return x


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("hidden", 2048), ("ffn", 6144), ("Hq", 8), ("Hk", 2), ("D", 256), ("rot", 64), ("B", 3), ("T", 1000),
                          ("new", 4)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    lens = [max(1, a.T * (b + 1) // a.B) for b in range(a.B)]  # ragged prompts
    most = max(lens) + a.new
    i32 = dict(dtype=torch.int32, device="cuda")
    one, two = (AttnLayer(a.hidden, a.ffn, a.Hq, a.Hk, a.D, a.rot,
                          PagedCache(a.B, a.Hk, a.D, sum(-(-(n + a.new) // 16) for n in lens), max_blocks=-(-most // 16)))
                for _ in range(2))
    tokens = [torch.randn(n + a.new, a.hidden, device="cuda").bfloat16() for n in lens]
    whole = one.forward(torch.cat(tokens), torch.tensor([n + a.new for n in lens], **i32),
                        one.step(sum(lens) + a.B * a.new, most, most)).split([n + a.new for n in lens])
    parts = [[x] for x in two.forward(torch.cat([x[:n] for x, n in zip(tokens, lens)]), torch.tensor(lens, **i32),
                                      two.step(sum(lens), max(lens), most)).split(lens)]
    x, ones, s = torch.empty(a.B, a.hidden, device="cuda", dtype=torch.bfloat16), torch.ones(a.B, **i32), two.step(a.B, 1, most)
    graph = None
    for t in range(a.new):
        x.copy_(torch.stack([y[n + t] for y, n in zip(tokens, lens)]))
        if t == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                two.forward(x, ones, s)
        if graph is None:
            two.forward(x, ones, s)
        else:
            graph.replay()
        for b in range(a.B):
            parts[b].append(x[b:b + 1].clone())
    torch.cuda.synchronize()
    if gdn.gdn_device_status() != gdn.GDN_OK:
        raise SystemExit("device status %d" % gdn.gdn_device_status())
    want, got = torch.cat(list(whole)).double(), torch.cat([torch.cat(p) for p in parts]).double()
    dx = ((want - got).norm() / want.norm()).item()
    print("prompts of %s tokens, then %d each: outputs differ by %.2e (relative)" % (lens, a.new, dx))
    # Keys and values of the last tokens are rounded to e4m3 with a scale that a page's later tokens may have raised in the
    # one prompt and not yet in the other: where they differ, by a subnormal's step, 2^-9 / 448 of the page's largest.  The
    # rest is bf16 rounding at seven places per token, a half step of 2^-9 of a value on average, which add up in squares.
    if not dx < 7 ** 0.5 * 2.0 ** -8:
        raise SystemExit("prompts and tokens disagree")


if __name__ == "__main__":
    main()
