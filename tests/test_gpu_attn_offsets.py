"""Offsets that are out of order or range: each way gdn_attn and gdn_kv_append look for their sequences skips all of them,
writes nothing and records it."""
import math

import pytest
import torch

import attn_reference as R
from gated_deltanet_mixer_gb300 import gdn
from test_gpu_attn_cache import BF, F32, _lib, ok, refused, workspace  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS, FEW, TILE = 0, 1, 2


def broken(B, n):
    """Offsets of B sequences of n tokens with one that cannot be: (offsets, tokens of the call)."""
    cu = [n * b for b in range(B + 1)]
    for at in sorted({0, B // 2, B}):
        for value in (-1, -(1 << 31), cu[-1] + 1, (1 << 31) - 1):
            yield cu[:at] + [value] + cu[at + 1:]
        if 0 < at:
            yield cu[:at] + [cu[at - 1] - 1] + cu[at + 1:]
        if at < B:
            yield cu[:at] + [cu[at + 1] + 1] + cu[at + 1:]


@pytest.mark.parametrize("kernel,dt,n", [(FEW, BF, 1), (FEW, BF, 3), (TILE, BF, 40), (ROWS, F32, 1), (ROWS, F32, 20)])
@pytest.mark.parametrize("B", [1, 3, 32, 33, 128, 129, 300])
@pytest.mark.parametrize("ws", [True, False])
def test_attn(kernel, dt, n, B, ws):
    Hq, Hk, D, kv = 4, 1, 64, 2000 if B < 4 else 200
    cache = R.Cache([kv] * min(B, 3), Hk, D, 16, device="cuda").fill()
    cache.table, cache.kv = cache.table[:1].repeat(B, 1), cache.kv[:1].repeat(B)
    T = n * B
    bf = gdn.GDN_BF16 if dt == BF else gdn.GDN_F32
    form = gdn.gdn_selftest_attn_form(B, T, Hq, Hk, D, max_new=n, max_kv=kv, workspace=ws, io_dtype=bf)
    assert form.kernel == kernel
    if B < 4 and ws and kernel != FEW:
        assert form.parts > 1  # the join looks for its sequences too
    q = torch.randn(T, Hq * D, device="cuda").to(dt)
    o = torch.full_like(q, math.nan)
    w = workspace(B, T, Hq, Hk, D, dt, max_new=n, max_kv=kv) if ws else None
    for cu in broken(B, n):
        gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, cu_seqlens=torch.tensor(cu, device="cuda").to(torch.int32), max_new=n, max_kv=kv,
                     workspace=w)
        refused()
        assert bool(o.isnan().all()), cu
    gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, cu_seqlens=torch.arange(0, T + 1, n, device="cuda").to(torch.int32), max_new=n, max_kv=kv,
                 workspace=w)
    ok()
    assert not bool(o.isnan().any())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B", [1, 3, 129, 300])
def test_append(dt, B):
    n = 3
    cache = R.Cache([n + 20] * B, 1, 64, 16, device="cuda").fill()
    before = [t.clone() for t in cache.args()]
    kv = torch.randn(n * B, 128, device="cuda").to(dt)
    for cu in broken(B, n):
        gdn.gdn_kv_append(kv[:, :64], kv[:, 64:], *cache.args(), cu_seqlens=torch.tensor(cu, device="cuda").to(torch.int32), max_new=n)
        refused()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, cache.args())), cu
