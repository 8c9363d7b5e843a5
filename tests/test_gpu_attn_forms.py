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
@pytest.mark.parametrize("causal", [True, False])
def test_last_tiles_in_parts(D, causal):
    """Two tiles more than the GPU takes at once: those in parts, of a packed sequence and of fixed lengths; and fewer new
    tokens than the call says, so that other tiles, or none, are the last."""
    slots = torch.cuda.get_device_properties(0).multi_processor_count * (1 if D == 256 else 2)
    tokens = 16 * (slots // 2 + 1)  # of two tiles of 128 rows each, with 8 query heads to each of 2 key heads
    n, kv = tokens - 5, tokens + 700
    f = form([n], 16, 2, D, BF, kv)
    assert f.kernel == TILE and f.parts > 1 and form([n], 16, 2, D, BF, kv, ws=False).parts == 1
    cache = R.Cache([kv], 2, D, 16, device="cuda").fill()
    q, o = attend(cache, [n], 16, BF, causal=causal, max_kv=kv)
    ok()
    for at in (0, 16, n - 40):  # the first rows are the last tiles
        if causal:
            k, v = cache.rows(0, kv - n + at + 40)
            check_rows(o[at:at + 40], q[at:at + 40], cache, 0, 40, kv - n + at + 40, 16, True, D ** -0.5, BF, k=k, v=v)
        else:
            check_rows(o[at:at + 40], q[at:at + 40], cache, 0, 40, kv, 16, False, D ** -0.5, BF)
    _, whole = attend(cache, [n], 16, BF, causal=causal, max_kv=kv, q=q, ws=False)
    assert float((whole.float() - o.float()).abs().max()) <= 2 * 2.0 ** -8 * float(whole.float().abs().max())
    both = R.Cache([kv, kv - 3], 1, D, 16, device="cuda").fill()
    q2 = q[:n, :8 * D].repeat(2, 1).reshape(2, n, 8 * D).contiguous()
    kw = dict(causal=causal, max_kv=kv)
    o2 = torch.full_like(q2, math.nan)
    w = workspace(2, n, 8, 1, D, BF, packed=False, max_kv=kv)
    assert w.numel() > 0
    gdn.gdn_attn(q2, o2, *both.args(), Hq=8, workspace=w, **kw)
    ok()
    o3 = torch.full_like(q2, math.nan)
    gdn.gdn_attn(q2, o3, *both.args(), Hq=8, **kw)
    ok()
    assert float((o2.float() - o3.float()).abs().max()) <= 2 * 2.0 ** -8 * float(o3.float().abs().max())
    for fewer in (1, 300, n - 200):
        w = workspace(1, n, 16, 2, D, BF, max_new=n, max_kv=kv)
        o4 = torch.full((n, 16 * D), math.nan, device="cuda", dtype=BF)
        gdn.gdn_attn(q[:n].contiguous(), o4, *cache.args(), Hq=16, cu_seqlens=offsets([fewer]), max_new=n, workspace=w, **kw)
        ok()
        assert bool(o4[fewer:].isnan().all())
        top = min(fewer, 40)
        if causal:
            k, v = cache.rows(0, kv - fewer + top)
            check_rows(o4[:top], q[:top], cache, 0, top, kv - fewer + top, 16, True, D ** -0.5, BF, k=k, v=v)
        else:
            check_rows(o4[:top], q[:top], cache, 0, top, kv, 16, False, D ** -0.5, BF)


@pytest.mark.parametrize("B", [1, 31, 33, 128, 129, 300])
@pytest.mark.parametrize("ws", [True, False])
def test_many_sequences_of_tiles(B, ws):
    """Tiles are taken by their size over all sequences, up to some number of them; ties, sequences without new tokens,
    one that the call's bounds skip."""
    new = [(29 * i) % 90 for i in range(B)]
    new[0] = 61
    lens = [n + (131 * i) % 400 for i, n in enumerate(new)]
    cache = R.Cache(lens, 1, 64, 16, device="cuda").fill()
    check(cache, new, 8, BF, ws=ws, max_kv=max(lens))
    if B > 1:
        q, o = attend(cache, new, 8, BF, ws=ws, max_new=max(new) - 1, max_kv=max(lens))
        torch.cuda.synchronize()
        assert gdn.gdn_device_status(reset=True) == gdn.GDN_ERR_INVALID_ARG
        at = 0
        for b, n in enumerate(new):
            if n == max(new):
                assert bool(o[at:at + n].isnan().all())
            elif n:
                check_rows(o[at:at + n], q[at:at + n], cache, b, n, lens[b], 8, True, 64 ** -0.5, BF)
            at += n


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
