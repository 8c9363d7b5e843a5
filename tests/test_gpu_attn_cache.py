"""Attention over the paged 8-bit cache, appending to it, rotary positions and
page tables on the GPU against 64-bit forms of their formulas.

Tolerances.  A rounding to type t is off by at most half a step, h(t) = eps(t) / 2
of the value.  gdn_attn: p is rounded once to 16 bits (h = 2^-8 of bf16 at most) in
bf16 io, not in fp32; a score is a sum of D products in fp32, off by at most
(D + 8) 2^-24 of the sum of their sizes A, and enters p as a factor e^error; the
sum over L tokens is off by (L + 8) 2^-24 of itself, numerator and denominator; the
output is rounded once.  With S = sum_j p_j |v_j|:
    |error| <= (h_p + 4 (D + 8) 2^-24 A + 2 (L + 8) 2^-24) S + h(t) |o|
(4: the factors on a token and on the sum, twice for the higher orders)."""
import math

import pytest
import torch

import attn_reference as R
from gated_deltanet_mixer_gb300 import gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
H = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert torch.cuda.is_available()
    assert gdn.gdn_device_status(reset=True) == 0


def ok():
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0


def refused():
    """The calls so far left an invalid-argument record; takes it away."""
    torch.cuda.synchronize()
    assert gdn.gdn_device_status(reset=True) == gdn.GDN_ERR_INVALID_ARG


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def rows(n, width, dt, g, pad=0, size=1.0):
    """[n, width] with rows `pad` elements further apart than they are wide."""
    return (size * torch.randn(n, width + pad, device="cuda", generator=g)).to(dt)[:, :width]


def workspace(B, T, Hq, Hk, D, dt, packed=True, **kw):
    n = gdn.gdn_attn_workspace_bytes(B, T, Hq, Hk, D, packed=packed, io_dtype=gdn.GDN_BF16 if dt == BF else gdn.GDN_F32, **kw)
    return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN, whatever it is read as


def check_rows(got, q, cache, b, n, kv, Hq, causal, scale, dt, k=None, v=None):
    if k is None:
        k, v = cache.rows(b, kv)
    D = cache.D
    want, S, A = R.attend(q.reshape(n, Hq, D), k, v, n, causal, scale)
    hp = H[BF] if dt == BF else 0.0
    tol = (hp + 4 * (D + 8) * 2.0 ** -24 * A[:, :, None] + 2 * (kv + 8) * 2.0 ** -24) * S + H[dt] * want.abs()
    if dt == BF:
        tol = tol + R.least(cache, b, n, kv, Hq, causal)
    err = (got.reshape(n, Hq, D).double() - want).abs()
    assert bool((err <= tol + 1e-37).all()), "off by %.3g of the tolerance" % float((err / (tol + 1e-37)).max())


def attend(cache, new, Hq, dt, causal=True, scale=0.0, seed=3, ws=True, pad=8, q=None, max_new=None, max_kv=0):
    """A packed call, max_new as the lengths have it; o [tokens, Hq * D], NaN where nothing was written."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, width = max(1, sum(new)), Hq * cache.D
    max_new = max(new) if max_new is None else max_new
    if q is None:
        q = rows(T, width, dt, g, pad)
    buf = torch.full((T, width + 2 * pad), math.nan, device="cuda", dtype=dt)
    o = buf[:, :width]
    w = workspace(len(new), T, Hq, cache.Hk, cache.D, dt, max_new=max_new, max_kv=max_kv) if ws else None
    gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, cu_seqlens=offsets(new), causal=causal, scale=scale, workspace=w, max_new=max_new,
                 max_kv=max_kv)
    torch.cuda.synchronize()
    assert bool(buf[:, width:].isnan().all())  # between the rows
    return q, o


def check(cache, new, Hq, dt, causal=True, scale=0.0, **kw):
    q, o = attend(cache, new, Hq, dt, causal, scale, **kw)
    ok()
    at = 0
    for b, n in enumerate(new):
        if n:
            check_rows(o[at:at + n], q[at:at + n], cache, b, n, cache.lens[b], Hq, causal, scale or cache.D ** -0.5, dt)
        at += n


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,Hk,r,page", [(64, 2, 1, 16), (128, 1, 3, 32), (256, 2, 6, 16), (128, 2, 8, 64), (256, 1, 2, 128),
                                         (64, 3, 16, 16), (256, 1, 12, 16), (128, 1, 64, 16)])
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("said", [True, False])
def test_single_tokens(dt, D, Hk, r, page, ws, said):
    """Decoding: one token each, lengths around tile and page borders, from one on."""
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 300, 1000]
    check(R.Cache(lens, Hk, D, page, device="cuda").fill(), [1] * len(lens), Hk * r, dt, ws=ws,
          max_new=None if said else 0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,Hk,r,page", [(64, 2, 4, 16), (128, 2, 1, 32), (256, 2, 6, 16), (128, 1, 8, 128), (256, 1, 5, 64)])
def test_ragged_prompts(dt, D, Hk, r, page):
    """Prompts of odd lengths with and without a cached prefix, none among them, rows that fill tiles or not."""
    new = [1, 0, 130, 7, 64, 21, 33, 257]
    lens = [1, 5, 130, 200, 64, 22, 500, 300]
    check(R.Cache(lens, Hk, D, page, device="cuda").fill(), new, Hk * r, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n", [2, 3, 4, 5, 8, 13, 16, 40])
def test_few_tokens(dt, n):
    """Drafted tokens verified."""
    lens = [n, n + 1, 70, 129, 515]
    check(R.Cache(lens, 2, 128, 16, device="cuda").fill(), [n] * len(lens), 8, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [(1, 5000), (4, 3001), (300, 2500), (1, 70000)])
def test_long(dt, D, new, kv):
    check(R.Cache([kv, 100 + new], 1, D, 64, device="cuda").fill(), [new, new], 4, dt, max_kv=kv, max_new=new)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 9, 150])
def test_not_causal(dt, D, new):
    """Every row sees the whole cache, which may be shorter than the rows are many, or empty (gives 0)."""
    cache = R.Cache([1, 77, 200, 0, 5], 2, D, 16, device="cuda").fill()
    check(cache, [new] * 5, 6, dt, causal=False)


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_that_see_nothing(dt):
    """Causal rows before the first cached token give 0."""
    cache = R.Cache([3, 0, 20], 2, 128, 16, device="cuda").fill()
    check(cache, [5, 4, 150], 4, dt)
    check(R.Cache([3, 0, 1, 70], 2, 128, 16, device="cuda").fill(), [5, 4, 3, 5], 2, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n", [1, 4, 100])
def test_fixed_length_and_strides(dt, n):
    """[B, T, ..] views of a fused buffer without cu_seqlens, as packed."""
    B, Hq, D = 3, 8, 128
    cache = R.Cache([n, n + 40, n + 300], 2, D, 16, device="cuda").fill()
    g = torch.Generator(device="cuda").manual_seed(5)
    fused = torch.randn(B, n, (Hq + 4) * D, device="cuda", generator=g).to(dt)
    q = fused[..., 2 * D:2 * D + Hq * D]
    o = torch.empty(B, n, Hq * D, device="cuda", dtype=dt)
    gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, workspace=workspace(B, n, Hq, 2, D, dt, packed=False))
    ok()
    for b in range(B):
        check_rows(o[b], q[b], cache, b, n, cache.lens[b], Hq, True, D ** -0.5, dt)
    _, packed = attend(cache, [n] * B, Hq, dt, q=q.reshape(B * n, Hq * D))
    assert torch.equal(packed.reshape(B, n, -1), o)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 40, 200])
@pytest.mark.parametrize("scale", [1e-6, 0.3, 2.0, -0.1])
def test_scales_of_the_scores(dt, new, scale):
    """Nearly uniform weights, and nearly one-hot ones."""
    check(R.Cache([new + 300], 1, 128, 16, device="cuda").fill(), [new], 4, dt, scale=scale)


@pytest.mark.parametrize("new", [1, 5, 200])
def test_a_sink_and_a_long_tail(new):
    """One token far above thousands whose weights are each some 2^-15 of it and together as much."""
    D, kv = 128, 30000
    cache = R.Cache([kv], 1, D, 16, device="cuda").fill(mean=0.0)
    p0 = int(cache.table[0, 0])
    cache.sk.fill_(2.0 ** -7)
    k = torch.full((D,), 1.0, device="cuda") * 1.0
    cache.k8[p0, :, 0] = (k / cache.sk[p0, 0]).to(torch.float8_e4m3fn).view(torch.uint8)
    for j in range(-(-kv // 16)):
        cache.k8[int(cache.table[0, j]), :, (1 if j == 0 else 0):] = 0x08  # 2^-6 2^-7: next to nothing
    q = torch.full((new, 2 * D), 10.4 / D ** 0.5, device="cuda").bfloat16()
    check(cache, [new], 2, BF, q=q)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 6, 140])
def test_value_scales_far_apart(dt, new):
    """Pages whose values differ by 2^40 in size, zeros among them."""
    cache = R.Cache([new + 400], 2, 128, 16, device="cuda").fill()
    for j, e in enumerate((-20, 7, -33, 0, -10, -2, 5)):
        cache.sv[int(cache.table[0, 2 * j])] = 2.0 ** e
    cache.v8[int(cache.table[0, 3])] = 0
    cache.sv[int(cache.table[0, 3])] = 2.0 ** -120
    check(cache, [new], 4, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,kv,steps", [(2, 49, (0, 0, 0, 60)), (2, 17, (0, 60)), (7, 70, (0, 0, 0, 40, 80)), (20, 33, (0, 50, 100)),
                                          (140, 160, tuple(range(0, 120, 12)))])
def test_larger_values_of_later_tokens_do_not_reach_a_row(dt, D, new, kv, steps):
    """The value scales grow from page to page, up to 2^60 times, right behind what a row sees."""
    cache = R.Cache([kv], 2, D, 16, device="cuda").fill()
    for j, e in enumerate(steps):
        cache.sv[int(cache.table[0, j])] = 2.0 ** (e - 100)
    check(cache, [new], 8, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [2, 30, 140])
def test_weights_far_below_the_largest(dt, new):
    """Dimensions whose value is zero at the token with nearly all the weight: what is left of the others'."""
    cache = R.Cache([new + 60], 2, 128, 16, device="cuda").fill(mean=0.0)
    cache.v8[int(cache.table[0, 0]), :, 3] = 0
    cache.sk[cache.table[0].long()] = 2.0 ** -6
    cache.k8[int(cache.table[0, 0]), :, 3] = torch.full((128,), 60.0).to(torch.float8_e4m3fn).view(torch.uint8).to("cuda")
    for size in (16.0, 20.0, 24.0, 28.0):  # weights of e^-size next to it, about
        q = torch.full((new, 4 * 128), size * 64 / 60 / 128 ** 0.5, device="cuda").to(dt)
        check(cache, [new], 4, dt, q=q)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 6, 140])
@pytest.mark.parametrize("least", [2.0 ** -120, 2.0 ** -99, 0.0])
def test_least_scales(dt, new, least):
    """Values (or keys) that are all zeros, as of padding, or as small as they go."""
    for what in ("v", "k"):
        for zero in (True, False):
            cache = R.Cache([new + 90], 2, 128, 16, device="cuda").fill()
            getattr(cache, "s" + what)[cache.table[0].long()] = least
            if zero:
                getattr(cache, what + "8")[cache.table[0].long()] = 0
            check(cache, [new], 4, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 6, 140])
def test_sizes_of_q(dt, new):
    """Heads of q that differ by 2^40 in size."""
    cache = R.Cache([new + 200], 1, 128, 16, device="cuda").fill()
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(new, 4, 128, device="cuda", generator=g)
    q *= torch.tensor([2.0 ** -30, 1.0, 2.0 ** 10, 2.0 ** -8], device="cuda")[None, :, None]
    q[0, 1, :64] *= 2.0 ** -20
    check(cache, [new], 4, dt, q=q.reshape(new, -1).to(dt), scale=1e-3)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 4, 40, 150])
def test_what_lies_behind_a_token_does_not_reach_it(dt, new):
    """NaN bytes behind the end (the fill of the cache), NaN keys and values in later pages: rows before are as without them."""
    Hq, D, n = 4, 128, new
    lens = [n + 160]
    clean = R.Cache(lens, 2, D, 16, device="cuda").fill()
    q, want = attend(clean, [n], Hq, dt)
    dirty = R.Cache(lens, 2, D, 16, device="cuda").fill()
    last = (lens[0] - 1) // 16 * 16     # the page of the last token
    p = int(dirty.table[0, last // 16])
    dirty.sk[p, 0] = math.nan
    dirty.sv[p, 1] = math.nan
    _, got = attend(dirty, [n], Hq, dt, q=q)
    sees = torch.arange(lens[0] - n, lens[0], device="cuda") >= last
    assert bool(got[sees].isnan().all())
    assert torch.equal(got[~sees], want[~sees])
    ok()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 30, 150])
def test_nan_and_infinity_in_q(dt, new):
    """A NaN or infinity in a head of q makes that row and head NaN and reaches no other."""
    Hq, D = 4, 64
    cache = R.Cache([new + 100], 2, D, 16, device="cuda").fill()
    q, want = attend(cache, [new], Hq, dt)
    bad = q.clone()
    bad[new // 2, D + 3] = math.nan
    bad[0, 2 * D + 5] = math.inf
    _, got = attend(cache, [new], Hq, dt, q=bad)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[new // 2, D:2 * D] = True
    hit[0, 2 * D:3 * D] = True
    assert bool(got[hit].isnan().all())
    assert torch.equal(got[~hit], want[~hit])
    ok()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 50, 150])
def test_lengths_and_pages_that_cannot_be(dt, new):
    """Sequences with impossible lengths are skipped, pages that are none left out; the rest is computed."""
    Hq = 4
    lens = [new + 100, new + 60, new + 30, new + 90]
    cache = R.Cache(lens, 2, 64, 16, device="cuda").fill()
    q, want = attend(cache, [new] * 4, Hq, dt)
    ok()
    cache.kv[1] = -3
    cache.kv[2] = 100000
    gone = int(cache.table[3, 1])
    cache.table[3, 1] = cache.k8.shape[0]
    _, got = attend(cache, [new] * 4, Hq, dt, q=q)
    refused()
    assert bool(got[new:3 * new].isnan().all())
    assert torch.equal(got[:new], want[:new])
    cache.table[3, 1] = gone
    k, v = cache.rows(3, lens[3])
    keep = torch.ones(lens[3], dtype=torch.bool, device="cuda")
    keep[16:32] = False
    check_rows(got[3 * new:], q[3 * new:], cache, 3, new, lens[3], Hq, True, 64 ** -0.5, dt, k=k[keep], v=v[keep])


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-1, 5, 6, 9], [0, 5, 6, 10]])
def test_offsets_that_cannot_be(cu):
    cache = R.Cache([40, 40, 40], 1, 64, 16, device="cuda").fill()
    before = [t.clone() for t in cache.args()]
    q = torch.randn(9, 2 * 64, device="cuda").bfloat16()
    o = torch.full_like(q, math.nan)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gdn.gdn_attn(q, o, *cache.args(), Hq=2, cu_seqlens=cu)
    refused()
    assert bool(o.isnan().all())
    gdn.gdn_kv_append(q[:, :64], q[:, 64:], *cache.args(), cu_seqlens=cu)
    refused()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, cache.args()))


def test_more_new_tokens_than_said():
    cache = R.Cache([40, 40], 1, 64, 16, device="cuda").fill()
    q, o = attend(cache, [5, 4], 2, BF, max_new=4)
    refused()
    assert bool(o[:5].isnan().all()) and not bool(o[5:].isnan().any())
    q, o = attend(cache, [5, 4], 2, BF, max_kv=39)
    refused()
    assert bool(o.isnan().all())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 40])
def test_rows_behind_the_last_sequence_stay(dt, new):
    cache = R.Cache([100, 50], 1, 64, 16, device="cuda").fill()
    T, Hq = 2 * new + 7, 4
    q = torch.randn(T, Hq * 64, device="cuda").to(dt)
    o = torch.full_like(q, math.nan)
    gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, cu_seqlens=offsets([new, new]), workspace=workspace(2, T, Hq, 1, 64, dt))
    ok()
    assert bool(o[2 * new:].isnan().all()) and not bool(o[:2 * new].isnan().any())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 3, 40, 140])
def test_a_graph_replays_with_other_lengths(dt, new):
    """Captured once; lengths, tables and inputs change between replays, on a stream of its own; results repeat exactly."""
    Hq, Hk, D = 8, 2, 128
    lens = [new + 10, new + 400]
    cache = R.Cache(lens, Hk, D, 16, device="cuda", blocks=64).fill()
    q = torch.randn(2 * new, Hq * D, device="cuda").to(dt)
    o = torch.empty_like(q)
    ws = workspace(2, 2 * new, Hq, Hk, D, dt)
    cu = offsets([new, new])

    def call():
        gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, cu_seqlens=cu, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    first = o.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    o.fill_(math.nan)
    graph.replay()
    ok()
    assert torch.equal(o, first)
    cache.lens = [new + 400, new + 3]
    cache.table.copy_(cache.table.flip(0))
    cache.kv.copy_(torch.tensor(cache.lens, dtype=torch.int32))
    q.copy_(torch.randn_like(q))
    graph.replay()
    ok()
    for b in range(2):
        s = slice(b * new, (b + 1) * new)
        check_rows(o[s], q[s], cache, b, new, cache.lens[b], Hq, True, D ** -0.5, dt)


def test_a_cache_past_32_bits():
    """Pages whose bytes lie beyond 4 GB."""
    Hk, D, page = 8, 256, 128
    P = (5 << 30) // (Hk * D * page)
    k8 = torch.zeros(P, Hk, page, D, dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    sk, sv = torch.full((P, Hk), 2.0 ** -6, device="cuda"), torch.full((P, Hk), 2.0 ** -6, device="cuda")
    for new in (1, 30):
        small = R.Cache([300], Hk, D, page, device="cuda").fill()
        table = torch.tensor([[P - 1, 3, P - 7]], dtype=torch.int32, device="cuda")
        kv = torch.tensor([300 - new], dtype=torch.int32, device="cuda")
        for j in range(3):
            p = int(small.table[0, j])
            for a, b in ((k8, small.k8), (v8, small.v8), (sk, small.sk), (sv, small.sv)):
                a[table[0, j]] = b[p]
        x = torch.randn(1, new, 2 * Hk * D, device="cuda").bfloat16()
        k, v = x[..., :Hk * D], x[..., Hk * D:]
        kv += new
        gdn.gdn_kv_append(k, v, kv, table, k8, v8, sk, sv)
        gdn.gdn_kv_append(k, v, *small.args())
        q = torch.randn(1, new, Hk * D, device="cuda").bfloat16()
        o, o2 = torch.empty_like(q), torch.empty_like(q)
        gdn.gdn_attn(q, o, kv, table, k8, v8, sk, sv, Hq=Hk)
        gdn.gdn_attn(q, o2, *small.args(), Hq=Hk)
        ok()
        assert torch.equal(o, o2)
        check_rows(o[0], q[0], small, 0, new, 300, Hk, True, D ** -0.5, BF)


# ------------------------------------------------------------------ appending
def append_both(lens, new, Hk, D, page, dt, seed=0, size=1.0, edit=None, cache=None, filled=True):
    """The library's cache and the formula's behind the same tokens."""
    a = cache or R.Cache(lens, Hk, D, page, seed=seed, device="cuda", fill=0x35)
    if cache is None:
        before = [kv - n for kv, n in zip(lens, new)]
        a.lens = before
        a.fill()
    a.lens = list(lens)
    a.kv.copy_(torch.tensor(lens, dtype=torch.int32))
    b = R.Cache(lens, Hk, D, page, seed=seed, device="cuda")
    for n in ("table", "k8", "v8", "sk", "sv"):
        setattr(b, n, getattr(a, n).clone())
    g = torch.Generator(device="cuda").manual_seed(seed + 9)
    T = max(1, sum(new))
    kv = rows(T, 2 * Hk * D, dt, g, pad=8, size=size)
    if edit:
        edit(kv)
    k, v = kv[:, :Hk * D], kv[:, Hk * D:]
    gdn.gdn_kv_append(k, v, *a.args(), cu_seqlens=offsets(new))
    ok()
    cut = [x.reshape(T, Hk, D).split(list(new) + ([1] if sum(new) == 0 else [])) for x in (k, v)]
    R.append(cut[0], cut[1], b, lens, new)
    return a, b


def same(a, b):
    for n in ("sk", "sv"):
        assert torch.equal(getattr(a, n).view(torch.int32) & 0x7fffffff, getattr(b, n).view(torch.int32) & 0x7fffffff) or \
            torch.equal(torch.nan_to_num(getattr(a, n), nan=-5.0), torch.nan_to_num(getattr(b, n), nan=-5.0)), n
    for n in ("k8", "v8"):
        x, y = getattr(a, n), getattr(b, n)
        # -0 and 0 are one value: rounding in 64 bits keeps the sign as well
        assert torch.equal(x, y), "%s: %d bytes differ" % (n, int((x != y).sum()))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,Hk,page", [(64, 1, 16), (128, 3, 32), (256, 4, 16), (128, 2, 64), (256, 2, 128)])
def test_append(dt, D, Hk, page):
    """Bytes and scales equal the formula's: single tokens, ragged prompts, none; at and around page borders."""
    lens = [1, 16, 17, 40, 300, 129, 128, 64, 5]
    new = [1, 1, 1, 7, 211, 129, 2, 64, 0]
    same(*append_both(lens, new, Hk, D, page, dt))


@pytest.mark.parametrize("dt", [BF, F32])
def test_append_grows_a_scale(dt):
    """Larger tokens behind smaller ones in a half-filled page, and smaller behind larger ones."""
    for size in (2.0 ** -20, 0.01, 30.0, 1000.0, 2.0 ** 16):
        same(*append_both([20, 30, 47, 33], [1, 3, 10, 1], 2, 64, 16, dt, size=size))


@pytest.mark.parametrize("dt", [BF, F32])
def test_append_ties_borders_and_zeros(dt):
    """448 times a power of two and its neighbours as a page's largest value, halves of steps, zeros, saturation, the smallest."""
    step = {BF: 2.0 ** -8, F32: 2.0 ** -23}[dt]

    def edit(kv):
        kv.mul_(0.0)
        for i, top in enumerate((7.0, 7.0 * (1 + 2 * step), 448.0, 57344.0, 60000.0, 1e6, 2.0 ** -118, 2.0 ** -125, 0.0)):
            kv[16 * i:16 * i + 16] = torch.linspace(-1, 1, kv.shape[1], device="cuda").to(kv.dtype) * top
            kv[16 * i + 3, 5] = top
            kv[16 * i + 3, 5 + 64] = -top
            kv[16 * i + 4, :8] = torch.tensor([1.0625, 1.1875, -1.0625, 0.0009765625, 0.0029296875, 2.5, 17.0, 19.0],
                                              device="cuda") * top / 448

    same(*append_both([144], [144], 1, 64, 16, dt, edit=edit))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_what_is_not_finite(dt, bad):
    """The page and head of it get a NaN scale, no other; no NaN byte is written; and the scale stays NaN."""
    def edit(kv):
        kv[2, 3] = bad          # k, head 0
        kv[9, 2 * 64 + 64 + 1] = bad  # v, head 1

    a, b = append_both([30, 40], [10, 3], 2, 64, 16, dt, edit=edit)
    same(a, b)
    assert int(a.sk.isnan().sum()) > 0
    a2, b2 = append_both([31, 41], [1, 1], 2, 64, 16, dt, cache=a, seed=0)
    same(a2, b2)


def test_append_token_by_token_is_append_at_once():
    """Where scales do not grow past what is subnormal, the same bytes."""
    lens, D, Hk = [45], 64, 2
    whole, _ = append_both(lens, lens, Hk, D, 16, BF)
    g = torch.Generator(device="cuda").manual_seed(9)
    kv = rows(45, 2 * Hk * D, BF, g, pad=8)
    c = R.Cache(lens, Hk, D, 16, device="cuda", fill=0x35)
    for t in range(45):
        c.kv.fill_(t + 1)
        gdn.gdn_kv_append(kv[None, t:t + 1, :Hk * D], kv[None, t:t + 1, Hk * D:], *c.args())
    ok()
    p = c.table[0].long()
    for n in ("sk", "sv"):
        assert torch.equal(getattr(c, n)[p], getattr(whole, n)[p])
    x, y = (t.k8[p].view(torch.float8_e4m3fn).float() for t in (c, whole))
    assert float((x - y).abs().max()) <= 2.0 ** -10  # half a step of the subnormals


def test_append_refuses_what_cannot_be():
    c = R.Cache([40, 40, 40], 1, 64, 16, device="cuda", fill=0x35).fill()
    before = c.k8.clone(), c.sk.clone()
    kv = torch.randn(3, 4, 128, device="cuda")
    c.kv[0] = 3            # fewer than the call's
    c.kv[1] = 4000
    c.table[2, 2] = 99999
    gdn.gdn_kv_append(kv[..., :64], kv[..., 64:], *c.args())
    refused()
    written = c.k8 != before[0]
    assert bool((written.sum() == 0)) or set(written.flatten(1).any(1).nonzero().flatten().tolist()) <= {int(c.table[2, 2 - 0])}
    assert torch.equal(torch.nan_to_num(c.sk), torch.nan_to_num(before[1]))


# ------------------------------------------------------------- rotary positions
def rope_tol(want, x, dt, m):
    """cos and sin are off by 2 2^-24 plus the rounding of the angle, 2^-24 pi; two products and a sum in fp32, one rounding
    to the type: with |pair| the size of both, (2^-24 (2 + pi + 4)) m |pair| + h(t) |y|."""
    return 10 * 2.0 ** -24 * m * 2 ** 0.5 * x.abs().amax() + H[dt] * want.abs()


SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0),
            dict(kind="parts", factor=16.0, original=4096, fast=32.0, slow=1.0)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(256, 64), (128, 128), (64, 16), (64, 2), (80, 20), (256, 256), (7, 6), (24, 24)])
@pytest.mark.parametrize("tokens", [1, 5, 77])
def test_rope(dt, layout, D, rot, tokens):
    """Near and far positions, negative ones too, in place and not, odd head widths."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (tokens,), generator=g, device="cuda").to(torch.int32)
    pos[: tokens // 2] = torch.arange(tokens // 2, dtype=torch.int32)
    for scaling in SCALINGS:
        if rot == 2 and scaling and scaling["kind"] == "ntk":
            continue
        plan = gdn.gdn_rope_plan(rot, base=1e4, layout=layout, scaling=scaling)
        f, m = R.frequencies(rot, 1e4, scaling)
        # the plan's frequencies are doubles: 2^-53 of a turn's part per position and their own rounding
        slack = 4 * 2.0 ** 31 * 2.0 ** -52
        fused = torch.randn(tokens, 6 * D, generator=g, device="cuda").to(dt)
        q, k = fused[:, :3 * D], fused[:, 3 * D:5 * D]
        qo, ko = torch.full((tokens, 3 * D), math.nan, device="cuda", dtype=dt), torch.full((tokens, 2 * D), math.nan, device="cuda", dtype=dt)
        want = [R.rope(x, pos, rot, D, f, m, layout) for x in (q, k)]
        keep = fused.clone()
        gdn.gdn_rope(plan, pos, [(q, qo), (k, ko)], D=D)
        ok()
        assert torch.equal(fused, keep)
        for x, y, w in ((q, qo, want[0]), (k, ko, want[1])):
            assert bool(((y.double() - w).abs() <= rope_tol(w, x, dt, m) + slack * m * x.abs().amax()).all())
            assert torch.equal(y.unflatten(1, (-1, D))[..., rot:], x.unflatten(1, (-1, D))[..., rot:])
        gdn.gdn_rope(plan, pos, [(q, q), (k, k)], D=D)
        ok()
        assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(fused[:, 5 * D:], keep[:, 5 * D:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(layout):
    """<u, rope(x)> = <rope^T(u), x>, and turning back undoes the turn but for m^2."""
    g = torch.Generator(device="cuda").manual_seed(1)
    plan = gdn.gdn_rope_plan(64, layout=layout, scaling=SCALINGS[3])
    pos = torch.arange(1000, 1050, dtype=torch.int32, device="cuda")
    x, u = (torch.randn(50, 4 * 128, generator=g, device="cuda") for _ in range(2))
    y, w, back = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_rope(plan, pos, [(x, y)], D=128)
    gdn.gdn_rope(plan, pos, [(u, w)], D=128, inverse=True)
    gdn.gdn_rope(plan, pos, [(y, back)], D=128, inverse=True)
    ok()
    n = x.numel()
    assert abs(float((u.double() * y.double()).sum() - (w.double() * x.double()).sum())) <= 20 * 2.0 ** -24 * 1.6 * n ** 0.5 * 16
    r, z = back.unflatten(1, (4, 128))[..., :64], x.unflatten(1, (4, 128))[..., :64]
    assert float((r - z * plan.m ** 2).abs().max()) <= 40 * 2.0 ** -24 * 2 * float(x.abs().max())
    assert torch.equal(back.unflatten(1, (4, 128))[..., 64:], x.unflatten(1, (4, 128))[..., 64:])


def test_rope_many_tokens_and_odd_addresses():
    g = torch.Generator(device="cuda").manual_seed(2)
    plan = gdn.gdn_rope_plan(64)
    f, m = R.frequencies(64, 1e4)
    pos = torch.arange(5001, dtype=torch.int32, device="cuda")
    for pad, cut in ((0, 0), (3, 1), (8, 8)):
        x = torch.randn(5001, 2 * 128 + pad + cut, generator=g, device="cuda").bfloat16()[:, cut:cut + 256]
        y = torch.empty(5001, 256 + pad, device="cuda", dtype=BF)[:, :256]
        gdn.gdn_rope(plan, pos, [(x, y)], D=128)
        ok()
        w = R.rope(x, pos, 64, 128, f, m, "half")
        assert bool(((y.double() - w).abs() <= rope_tol(w, x, BF, m) + 1e-6).all())


# ------------------------------------------------------------------ page tables
def pages_by_hand(kv, new, free, used, table, page):
    table, slots, pos, cu = table.clone(), [], [], [0]
    for b, (k, n) in enumerate(zip(kv, new)):
        for t in range(k, k + n):
            if t % page == 0:
                table[b, t // page] = free[used]
                used += 1
            slots.append(int(table[b, t // page]) * page + t % page)
            pos.append(t)
        cu.append(cu[-1] + n)
    return table, slots, pos, cu, used


@pytest.mark.parametrize("B,top,most,page", [(1, 0, 1, 16), (1, 0, 5000, 16), (5, 40, 3, 16), (64, 100, 1, 32), (300, 30, 9, 64),
                                             (1024, 10, 4, 16), (1500, 20, 20, 128), (3000, 0, 2, 16), (16384, 5, 1, 16)])
@pytest.mark.parametrize("in_place", [True, False])
def test_pages(B, top, most, page, in_place):
    g = torch.Generator().manual_seed(B)
    kv = torch.randint(0, top + 1, (B,), generator=g)
    new = torch.randint(0, most + 1, (B,), generator=g)
    new[0] = most
    width = max(1, int(((kv + new + page - 1) // page).max()))
    table = torch.full((B, width + 2), -7, dtype=torch.int32)
    nfree = int(((kv + new + page - 1) // page - (kv + page - 1) // page).sum()) + 4
    free = torch.randperm(nfree + 50, generator=g)[:nfree].to(torch.int32)
    for b in range(B):
        have = -(-int(kv[b]) // page)
        table[b, :have] = torch.randint(0, 1000, (have,), generator=g).to(torch.int32)
    want = pages_by_hand(kv.tolist(), new.tolist(), free.tolist(), 3, table, page)
    total = want[3][-1]
    d = [t.to(torch.int32).cuda() for t in (kv, new, free)]
    used, tab = torch.tensor([3], dtype=torch.int32, device="cuda"), table.cuda()
    kv_out, used_out = (d[0], used) if in_place else (torch.empty_like(d[0]), torch.empty_like(used))
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.full((total + 5,), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((total + 5,), 77, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_pages(d[0], d[1], d[2], used, tab[:, :width], kv_out, used_out, cu, slots, pos, page=page)
    ok()
    assert torch.equal(tab.cpu(), want[0])
    assert slots.tolist() == want[1] + [-1] * 5 and pos.tolist() == want[2] + [0] * 5
    assert cu.tolist() == want[3] and kv_out.tolist() == (kv + new).tolist() and int(used_out) == want[4]


@pytest.mark.parametrize("what", ["negative", "table", "pages", "tokens", "used", "cached"])
def test_pages_all_or_nothing(what):
    kv, new = torch.tensor([5, 16, 0]), torch.tensor([20, 1, 3])
    free, used, n = torch.arange(10), 2, 24
    if what == "negative":
        new[1] = -1
    if what == "table":
        kv[2] = 60
    if what == "pages":
        free = free[:4]
    if what == "tokens":
        n = 23
    if what == "used":
        used = -1
    if what == "cached":
        kv[0] = -5
    i32 = [t.to(torch.int32).cuda() for t in (kv, new, free)]
    table = torch.full((3, 3), 99, dtype=torch.int32, device="cuda")
    u = torch.tensor([used], dtype=torch.int32, device="cuda")
    cu = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    slots = torch.full((n,), 5, dtype=torch.int64, device="cuda")
    pos = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    before = i32[0].clone()
    gdn.gdn_kv_pages(i32[0], i32[1], i32[2], u, table, i32[0], u, cu, slots, pos, page=16)
    refused()
    assert bool((table == 99).all()) and int(u) == used and torch.equal(i32[0], before)
    assert bool((cu == 0).all()) and bool((slots == -1).all()) and bool((pos == 0).all())


# ------------------------------------------------------------------ all together
@pytest.mark.parametrize("dt", [BF, F32])
def test_a_layer_over_its_steps(dt):
    """Pages, rotary positions, appending and attention as a server runs them: a batch of prompts, then single tokens in a
    captured graph whose page tables, lengths and offsets stay on the GPU; every step against the formulas on what the
    cache then holds, and the cache against the turned keys within the bytes' rounding."""
    B, Hq, Hk, D, rot, page, steps = 3, 6, 2, 64, 32, 16, 20
    prompts = [37, 1, 120]
    g = torch.Generator(device="cuda").manual_seed(0)
    c = R.Cache([0] * B, Hk, D, page, device="cuda", extra=40, blocks=12)
    free = torch.randperm(40, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = gdn.gdn_rope_plan(rot)
    f, m = R.frequencies(rot, 1e4)
    i32 = dict(dtype=torch.int32, device="cuda")

    class Step:
        def __init__(self, new):
            self.n = sum(new)
            self.new = torch.tensor(new, **i32)
            self.cu, self.pos = torch.zeros(B + 1, **i32), torch.zeros(self.n, **i32)
            self.slots = torch.zeros(self.n, dtype=torch.int64, device="cuda")
            self.x = torch.zeros(self.n, (Hq + 2 * Hk) * D, device="cuda", dtype=dt)
            self.o = torch.zeros(self.n, Hq * D, device="cuda", dtype=dt)
            self.max_new = max(new)
            self.ws = workspace(B, self.n, Hq, Hk, D, dt, max_new=self.max_new)

        def run(self):
            q, k, v = self.x.split([Hq * D, Hk * D, Hk * D], 1)
            gdn.gdn_kv_pages(c.kv, self.new, free, used, c.table, c.kv, used, self.cu, self.slots, self.pos, page=page)
            gdn.gdn_rope(plan, self.pos, [(q, q), (k, k)], D=D)
            gdn.gdn_kv_append(k, v, *c.args(), cu_seqlens=self.cu, max_new=self.max_new)
            gdn.gdn_attn(q, self.o, *c.args(), Hq=Hq, cu_seqlens=self.cu, max_new=self.max_new, workspace=self.ws)

    history = [[] for _ in range(B)]

    def verify(step, raw, new):
        ok()
        at = 0
        for b, n in enumerate(new):
            kv = int(c.kv[b])
            c.lens[b] = kv
            k = raw[at:at + n, Hq * D:(Hq + Hk) * D]
            history[b].append(R.rope(k, torch.arange(kv - n, kv, device="cuda"), rot, D, f, m, "half"))
            turned = torch.cat(history[b]).view(kv, Hk, D)
            held = c.rows(b, kv)[0]
            # a rounding of x, and one to e4m3 (2^-4 of the value, 2^-10 of the scale, which is above amax / 448 by 2 at most),
            # twice where a scale has grown
            top = turned.abs().max()
            assert bool(((held - turned).abs() <= 2 * (2.0 ** -4 * turned.abs() + 2.0 ** -9 / 448 * 2 * top) + 2.0 ** -7 * turned.abs()).all())
            check_rows(step.o[at:at + n], step.x[at:at + n, :Hq * D], c, b, n, kv, Hq, True, D ** -0.5, dt)
            at += n

    p = Step(prompts)
    p.x.copy_(torch.randn(p.x.shape, device="cuda", generator=g))
    raw = p.x.clone()
    p.run()
    verify(p, raw, prompts)
    s = Step([1] * B)
    raw = torch.randn(s.x.shape, device="cuda", generator=g).to(dt)
    s.x.copy_(raw)
    s.run()  # once as it is: kernels load
    verify(s, raw, [1] * B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(steps):
        raw = torch.randn(s.x.shape, device="cuda", generator=g).to(dt)
        s.x.copy_(raw)
        graph.replay()
        verify(s, raw, [1] * B)
