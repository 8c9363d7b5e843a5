"""Calls of gdn_attn that its documentation allows."""
import math

import pytest
import torch

import attn_reference as R
from gated_deltanet_mixer_gb300 import gdn
from test_gpu_attn_cache import BF, F32, _lib, offsets, ok, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 4, 40, 150])
@pytest.mark.parametrize("ws", [True, False])
def test_o_beside_q_in_one_buffer(dt, D, n, ws):
    """q and o column blocks of one buffer, packed and of fixed length: as apart, and nothing else of the buffer moves."""
    Hq, Hk, B = 8, 2, 2
    cache = R.Cache([n + 300, n + 5], Hk, D, 16, device="cuda").fill()
    g = torch.Generator(device="cuda").manual_seed(n)
    buf = torch.randn(B, n, 3 * Hq * D, device="cuda", generator=g).to(dt)
    for q_at, o_at in ((0, 2), (1, 0)):
        for packed in (True, False):
            one = buf.clone()
            kw = dict(Hq=Hq, cu_seqlens=offsets([n] * B)) if packed else dict(Hq=Hq)
            flat = (lambda x: x.flatten(0, 1)) if packed else (lambda x: x)
            q, o = (flat(one)[..., at * Hq * D:(at + 1) * Hq * D] for at in (q_at, o_at))
            apart = torch.full(o.shape, math.nan, device="cuda", dtype=dt)
            if ws:
                kw["workspace"] = workspace(B, B * n if packed else n, Hq, Hk, D, dt, packed=packed)
            gdn.gdn_attn(q.clone(), apart, *cache.args(), **kw)
            gdn.gdn_attn(q, o, *cache.args(), **kw)
            ok()
            assert torch.equal(o, apart)
            keep = [i for i in range(3) if i != o_at]
            assert all(torch.equal(one[..., i * Hq * D:(i + 1) * Hq * D], buf[..., i * Hq * D:(i + 1) * Hq * D]) for i in keep)
