"""Every way gdn_attn runs: each kernel, each tile of rows, tokens whole and cut into parts, with the form asked for by
name (gdn_selftest_attn_form), against the 64-bit form."""
import math

import pytest
import torch

import attn_reference as R
from gated_deltanet_mixer_gb300 import gdn
from test_gpu_attn_cache import BF, F32, _lib, attend, check, check_rows, offsets, ok, workspace  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS, FEW, TILE = 0, 1, 2


def form(new, Hq, Hk, D, dt, max_kv, ws=True):
    return gdn.gdn_selftest_attn_form(len(new), sum(new), Hq, Hk, D, max_new=max(new), max_kv=max_kv, workspace=ws,
                                      io_dtype=gdn.GDN_BF16 if dt == BF else gdn.GDN_F32)


@pytest.mark.parametrize("D,r,n,rows", [(256, 1, 1, 8), (256, 6, 1, 8), (256, 8, 1, 8), (256, 6, 2, 16), (256, 16, 1, 16),
                                        (128, 8, 1, 8), (128, 8, 2, 16), (128, 3, 5, 16), (64, 8, 1, 8), (64, 5, 3, 16), (64, 8, 4, 32), (64, 32, 1, 32)])
def test_few_rows(D, r, n, rows):
    """Units that lie in one block's range, in two and in many; more units than blocks."""
    for lens in ([3000 + n], [n, 700, 64 + n, 2048, 17 + n], [40 + n] * 180):
        new = [n] * len(lens)
        f = form(new, 2 * r, 2, D, BF, max(lens))
        assert (f.kernel, f.rows) == (FEW, rows)
        check(R.Cache(lens, 2, D, 16, device="cuda").fill(), new, 2 * r, BF, max_kv=max(lens))


def test_few_rows_of_some():
    """Fewer new tokens than max_new says in some sequences, none in others, with many sequences (their lengths are
    scanned several to a thread)."""
    lens = [(37 * i) % 300 for i in range(700)]
    new = [min(n, i % 4) for i, n in enumerate(lens)]
    assert form(new, 4, 2, 64, BF, 300).kernel == FEW
    check(R.Cache(lens, 2, 64, 32, device="cuda", extra=0).fill(), new, 4, BF, max_kv=300)


@pytest.mark.parametrize("D,r,n", [(256, 6, 3), (256, 8, 30), (128, 8, 4), (128, 32, 1), (128, 1, 100), (64, 8, 9), (64, 2, 70)])
@pytest.mark.parametrize("kv", [300, 5000])
def test_tiles_in_parts(D, r, n, kv):
    """Few tiles over many tokens: cut into parts, whose join also sees parts without tokens (a short sequence)."""
    lens = [kv, n + 5]
    f = form([n, n], r, 1, D, BF, kv)
    assert f.kernel == TILE and f.rows == 128 and (f.parts > 1) == (kv > 1000)
    assert form([n, n], r, 1, D, BF, kv, ws=False).parts == 1
    cache = R.Cache(lens, 1, D, 16, device="cuda").fill()
    check(cache, [n, n], r, BF, max_kv=kv)
    check(cache, [n, n], r, BF, max_kv=kv, ws=False)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tiles_whole(D):
    """More tiles than the GPU has SMs."""
    lens, new = [700, 1500, 90], [600, 1500, 90]
    f = form(new, 16, 2, D, BF, 1500)
    assert (f.kernel, f.parts) == (TILE, 1)
    check(R.Cache(lens, 2, D, 64, device="cuda").fill(), new, 16, BF, max_kv=1500)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 20])
def test_fp32_in_parts(D, n):
    f = form([n], 4, 2, D, F32, 3000)
    assert f.kernel == ROWS and f.parts > 1
    check(R.Cache([3000], 2, D, 16, device="cuda").fill(), [n], 4, F32, max_kv=3000)


@pytest.mark.parametrize("n,r", [(1, 4), (60, 4)])
def test_nan_pages_in_parts(n, r):
    """A NaN scale in a page of one part reaches every row that sees the page, and no earlier row."""
    kv, D = 4000, 128
    for scale in ("sk", "sv"):
        cache = R.Cache([kv], 1, D, 16, device="cuda").fill()
        q, want = attend(cache, [n], r, BF, max_kv=kv)
        getattr(cache, scale)[int(cache.table[0, (kv - 20) // 16])] = math.nan
        _, got = attend(cache, [n], r, BF, q=q, max_kv=kv)
        ok()
        sees = torch.arange(kv - n, kv, device="cuda") >= (kv - 20) // 16 * 16
        assert bool(got[sees].isnan().all()) and torch.equal(got[~sees], want[~sees])


def test_a_workspace_that_is_too_small_is_refused():
    for n in (1, 20):
        cache = R.Cache([5000], 1, 128, 16, device="cuda").fill()
        q = torch.randn(n, 8 * 128, device="cuda").bfloat16()
        ws = workspace(1, n, 8, 1, 128, BF, max_new=n, max_kv=5000)
        assert ws.numel() > 0
        with pytest.raises(gdn.GdnError):
            gdn.gdn_attn(q, torch.empty_like(q), *cache.args(), Hq=8, cu_seqlens=offsets([n]), max_new=n, max_kv=5000,
                         workspace=ws[:256])


def test_the_workspace_does_for_shorter_tables():
    """gdn_attn_workspace_bytes without max_kv: enough for any table."""
    for n, r in ((1, 8), (10, 8), (200, 8)):
        ws = workspace(1, n, r, 1, 128, BF, max_new=n)
        for kv in (n + 50, 3000, 9000, 20000):
            cache = R.Cache([kv], 1, 128, 128, device="cuda").fill()
            q = torch.randn(n, r * 128, device="cuda").bfloat16()
            o = torch.empty_like(q)
            gdn.gdn_attn(q, o, *cache.args(), Hq=r, cu_seqlens=offsets([n]), max_new=n, workspace=ws)
            ok()
            check_rows(o, q, cache, 0, n, kv, r, True, 128 ** -0.5, BF)


def test_two_calls_at_once():
    """Two streams, a workspace each: as one after the other, bit for bit."""
    for n in (1, 40):
        D, r, kv = 128, 8, 3000
        caches = [R.Cache([kv], 1, D, 16, seed=i, device="cuda").fill(seed=i + 5) for i in range(2)]
        q = [torch.randn(n, r * D, device="cuda").bfloat16() for _ in range(2)]
        kw = dict(Hq=r, cu_seqlens=offsets([n]), max_new=n, max_kv=kv)
        want = [torch.empty_like(x) for x in q]
        for i in range(2):
            gdn.gdn_attn(q[i], want[i], *caches[i].args(), workspace=workspace(1, n, r, 1, D, BF, max_new=n, max_kv=kv), **kw)
        torch.cuda.synchronize()
        got = [torch.full_like(x, math.nan) for x in q]
        streams = [torch.cuda.Stream() for _ in range(2)]
        ws = [workspace(1, n, r, 1, D, BF, max_new=n, max_kv=kv) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                gdn.gdn_attn(q[i], got[i], *caches[i].args(), workspace=ws[i], stream=streams[i], **kw)
        ok()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_page_in_two_places():
    """A page shared by two sequences, and one that stands twice in a table, read as what they are."""
    cache = R.Cache([64, 64], 1, 64, 16, device="cuda").fill()
    cache.table[1, :2] = cache.table[0, :2]
    cache.table[1, 3] = cache.table[1, 2]
    for n in (1, 40):
        check(cache, [n, n], 4, BF)
