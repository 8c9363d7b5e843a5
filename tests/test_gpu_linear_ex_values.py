"""gdn_linear_ex's activations over their whole range.  The contraction has one
product, by 1, so the sums are exact and only the activation is looked at."""
import math

import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert gdn.gdn_device_status(reset=True) == 0


def activated(values, act, M, up=None):
    """act(values), as the columns of M rows; gated with a constant up factor if one is given."""
    n = values.numel()
    x = torch.zeros(M, 8, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 1
    w = torch.zeros(n * (1 if up is None else 2), 8, device="cuda", dtype=torch.bfloat16)
    w[:n, 0] = values.cuda()
    if up is not None:
        w[n:, 0] = up
    y = torch.empty(M, n, device="cuda", dtype=torch.bfloat16)
    gdn.gdn_linear_ex(x, w, [(0, n, y, act)], gated=up is not None)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    return y.cpu().double()


# 2^-8 of the value is twice the bf16 rounding; the argument of erfc, up to 9 here, is off by 2^-23 of
# itself, which the tail turns into 2 * 81 * 2^-23 < 2^-15 of the value, and erfcf by 2^-21; sigmoid
# and SiLU have an exponential with 2 + 1.2 |x| steps of 2^-23, < 2^-16.  Results below the
# smallest normal number of fp32, over bf16's or the exponential's, may be 0.
@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("up", [None, 1024.0])
@pytest.mark.parametrize("act", ["gelu", "silu", "sigmoid", "none"])
def test_activation_tails(act, M, up):
    lo = -12.5 if act == "gelu" else -80.0
    v = torch.cat([torch.linspace(lo, 12.5, 2001), torch.tensor([-6.0, -5.0, -4.0, -3.0, 0.0, 1e-30, -1e-30, 3e38])]).bfloat16()
    x = v.double()
    want = {"gelu": 0.5 * x * torch.erfc(-x / math.sqrt(2.0)), "silu": x * torch.sigmoid(x), "sigmoid": torch.sigmoid(x),
            "none": x}[act]
    if up is not None:
        v, want = v[:-1], want[:-1] * up  # 3e38 times up overflows
    err = (activated(v, act, M, up) - want).abs()
    bound = (2.0 ** -8 + 2.0 ** -15) * want.abs() + 2.0 ** -126 * (up or 1.0)
    assert bool((err <= bound).all()), "x = %s" % v[(err > bound).any(0)][:8].tolist()
