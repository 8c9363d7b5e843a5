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


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hk,r", [(1, 1), (2, 8), (1, 24)])
@pytest.mark.parametrize("packed", [True, False])
def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(dt, D, Hk, r, packed):
    """Sized once: fewer sequences, fewer tokens, shorter tables.  (What a call uses rises and falls with them.)"""
    B, n, kv = 4, 1500 // max(1, r // 2), 6000
    cache = R.Cache([kv] * B, Hk, D, 128, device="cuda").fill()
    Hq = Hk * r
    io = dict(io_dtype=gdn.GDN_BF16 if dt == BF else gdn.GDN_F32, packed=packed)
    w = torch.empty(gdn.gdn_attn_workspace_bytes(B, B * n if packed else n, Hq, Hk, D, max_new=n, max_kv=kv, **io), dtype=torch.uint8,
                    device="cuda")
    assert w.numel() > 0
    q = torch.randn(B, n, Hq * D, device="cuda").to(dt)
    for b in (B, 1, 2):
        small = R.Cache([kv] * b, Hk, D, 128, device="cuda")
        small.table, args = cache.table[:b].contiguous(), cache.args()[2:]
        for m in sorted({n, n - 1, n // 2, n // 3, n // 5, n // 16 or 1, 40, 17, 5, 2, 1}):
            for top in (kv, 3000, 700, 128):
                if m > top:
                    continue
                x = q[:b, :m].reshape(b * m, -1) if packed else q[:b, :m].contiguous()
                o = torch.full_like(x, math.nan)
                kw = dict(cu_seqlens=offsets([m] * b), max_new=m) if packed else {}
                gdn.gdn_attn(x, o, torch.full((b,), top, dtype=torch.int32, device="cuda"), small.table, *args, Hq=Hq, max_kv=top,
                             workspace=w, **kw)
                assert not bool(o.isnan().any())
                assert gdn.gdn_attn_workspace_bytes(b, b * m if packed else m, Hq, Hk, D, max_new=m if packed else 0, max_kv=top, **io) <= w.numel()
    ok()
