"""Linear attention with decay and the fused projections in 64 bits, written
from the formulas, with the error scales that the tolerances are built from.

``recur`` returns beside o and S the same sums over absolute values (Ao, AS):
every rounding of an operand or a partial sum changes a result by at most that
rounding times the sum of the magnitudes that meet in it."""
import math

import torch

D = 128


def recur(q, k, v, g, S0, scale=None):
    """q, k [T, Hk, D], v [T, Hv, D], g [T, Hv], S0 [Hv, D, D] or None (fp64 CPU tensors)."""
    T, Hv = v.shape[:2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    r = Hv // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    S = torch.zeros(Hv, D, D, dtype=torch.float64) if S0 is None else S0.clone()
    AS = S.abs()
    o, Ao = torch.empty(T, Hv, D, dtype=torch.float64), torch.empty(T, Hv, D, dtype=torch.float64)
    for t in range(T):
        a = g[t].exp()[:, None, None]
        S = torch.where(a == 0, 0.0, a * S) + v[t][:, :, None] * k[t][:, None, :]
        AS = torch.where(a == 0, 0.0, a * AS) + v[t].abs()[:, :, None] * k[t].abs()[:, None, :]
        o[t] = scale * torch.einsum("hvk,hk->hv", S, q[t])
        Ao[t] = abs(scale) * torch.einsum("hvk,hk->hv", AS, q[t].abs())
    return o, S, Ao, AS


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x / math.sqrt(2.0)))
    if act == "sigmoid":
        return torch.sigmoid(x)
    return x


class Guarded:
    """A tensor inside a larger buffer whose bytes around it must not change."""

    def __init__(self, shape, dtype, ld=None, device="cuda"):
        rows, cols = (1, math.prod(shape)) if ld is None else (math.prod(shape[:-1]), shape[-1])
        self.buf = torch.full((2048 + rows * (ld or cols) + 2048,), 7.0, dtype=dtype, device=device)
        body = self.buf[2048:-2048]
        self.t = body.view(shape) if ld is None else body.view(*shape[:-1], ld)[..., :cols]
        self.inside = torch.zeros_like(self.buf, dtype=torch.bool)
        flag = self.inside[2048:-2048]
        (flag if ld is None else flag.view(*shape[:-1], ld)[..., :cols]).fill_(True)

    def intact(self):
        return bool((self.buf[~self.inside] == 7.0).all())
