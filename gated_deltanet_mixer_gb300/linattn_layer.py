"""A decoder layer of linear attention with a decay for each head, on the library's operators.

    python -m gated_deltanet_mixer_gb300.linattn_layer --hidden 2048 --ffn 6144 --Hk 16 --Hv 16 --T 1000 --new 4

Per token x [hidden] of the residual stream:

    q | k | v = x W_in^T + b_in      SiLU on q and k, none on v     one gdn_linear_ex, a range each
    o         = linear attention     state S [Hv][128][128]         gdn_linattn_prefill / _decode
    x        += o W_out^T            added in place                 gdn_linear_ex
    f         = silu(x W_g^T) (x W_u^T)                             gdn_linear_ex, gated
    x        += f W_d^T              added in place                 gdn_linear_ex

(The norms in front of the two halves are left out: they are the caller's.)
Run as a program it takes a prompt and then single tokens, and checks that the
state and the outputs agree with one longer prompt.
"""
import argparse
import math

import torch

from . import gdn

D = 128


class LinAttnLayer:
    """Weights, the cached state of B sequences, and the workspace kept across calls."""

    def __init__(self, hidden, ffn, Hk, Hv, B, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(rows, cols):
            return (torch.randn(rows, cols, device=device, generator=g) / math.sqrt(cols)).bfloat16()

        self.hidden, self.ffn, self.Hk, self.Hv, self.B = hidden, ffn, Hk, Hv, B
        self.w_in, self.w_out = w((2 * Hk + Hv) * D, hidden), w(hidden, Hv * D)
        self.b_in = torch.zeros(self.w_in.shape[0], device=device, dtype=torch.bfloat16)
        self.w_gate_up, self.w_down = w(2 * ffn, hidden), w(hidden, ffn)
        # a geometric ladder of decays over the heads
        self.log_decay = -torch.exp2(-8.0 * torch.arange(1, Hv + 1, device=device, dtype=torch.float32) / Hv)
        self.S = torch.zeros(B, Hv, D, D, device=device)
        self.ws = torch.empty(0, dtype=torch.uint8, device=device)

    def forward(self, x, decode=False):
        """x [B, T, hidden] bf16, updated in place; the state moves on by T tokens."""
        B, T, _ = x.shape
        rows = x.view(B * T, self.hidden)
        kq, kv = self.Hk * D, self.Hv * D
        qkv = torch.empty(B, T, 2 * kq + kv, device=x.device, dtype=x.dtype)
        flat = qkv.view(B * T, -1)
        gdn.gdn_linear_ex(rows, self.w_in, [(0, 2 * kq, flat[:, :2 * kq], "silu"), (2 * kq, 2 * kq + kv, flat[:, 2 * kq:])],
                          bias=self.b_in)
        q, k, v = qkv[..., :kq], qkv[..., kq:2 * kq], qkv[..., 2 * kq:]
        o = torch.empty(B, T, kv, device=x.device, dtype=x.dtype)
        if decode:
            gdn.gdn_linattn_decode(q, k, v, self.S, o, Hk=self.Hk, Hv=self.Hv, log_decay=self.log_decay)
        else:
            need = gdn.gdn_linattn_workspace_bytes(B, T, self.Hk, self.Hv)
            if self.ws.numel() < need:
                self.ws = torch.empty(need, dtype=torch.uint8, device=x.device)
            gdn.gdn_linattn_prefill(q, k, v, self.S, o, self.S, Hk=self.Hk, Hv=self.Hv, log_decay=self.log_decay,
                                    workspace=self.ws)
        gdn.gdn_linear_ex(o.view(B * T, kv), self.w_out, [(0, self.hidden, rows, "none", rows)])
        f = torch.empty(B * T, self.ffn, device=x.device, dtype=x.dtype)
        gdn.gdn_linear_ex(rows, self.w_gate_up, [(0, self.ffn, f, "silu")], gated=True)
        gdn.gdn_linear_ex(f, self.w_down, [(0, self.hidden, rows, "none", rows)])
        return x


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("hidden", 2048), ("ffn", 6144), ("Hk", 16), ("Hv", 16), ("B", 2), ("T", 1000), ("new", 4)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    x = torch.randn(a.B, a.T + a.new, a.hidden, device="cuda").bfloat16()
    one, two = (LinAttnLayer(a.hidden, a.ffn, a.Hk, a.Hv, a.B) for _ in range(2))
    whole = one.forward(x.clone())
    parts = [two.forward(x[:, :a.T].clone())]
    for t in range(a.T, a.T + a.new):
        parts.append(two.forward(x[:, t:t + 1].clone(), decode=True))
    parts = torch.cat(parts, dim=1)
    torch.cuda.synchronize()
    if gdn.gdn_device_status() != gdn.GDN_OK:
        raise SystemExit("device status %d" % gdn.gdn_device_status())
    dx = ((whole.double() - parts.double()).norm() / whole.double().norm()).item()
    dS = ((one.S.double() - two.S.double()).norm() / one.S.double().norm()).item()
    print("prompt of %d tokens, then %d: outputs differ by %.2e, states by %.2e (relative)" % (a.T, a.new, dx, dS))
    # both runs round the same values to bf16 at six places per token; a half
    # step is 2^-9 of a value on average, and the differences add up in squares
    if not (dx < 6 ** 0.5 * 2.0 ** -8 and dS < 2.0 ** -8):
        raise SystemExit("prompt and tokens disagree")


if __name__ == "__main__":
    main()
