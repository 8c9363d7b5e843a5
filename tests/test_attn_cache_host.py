"""Host-side checks of gdn_kv_append, gdn_attn, gdn_rope and gdn_kv_pages that
need no GPU: bad arguments are refused before the device is touched (addresses
are never dereferenced); the frequencies of a plan; the 64-bit forms that the
GPU tests compare with, against hand-made values and each other."""
import ctypes
import math

import pytest
import torch

import attn_reference as R
from gated_deltanet_mixer_gb300 import build as gdn_build
from gated_deltanet_mixer_gb300 import gdn

BASE, STEP = 0x7F0000000000, 1 << 36
OK_ON_HOST = (5, 7)  # every check passed; then no device (or not this one)


def fake(i, offset=0):
    return BASE + i * STEP + offset


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


def shape(**over):
    a = dict(B=2, T=8, Hq=8, Hk=2, D=128, io_dtype=gdn.GDN_BF16, max_new=0, max_kv=0)
    a.update({k: v for k, v in over.items() if k in a})
    return gdn.gdn_attn_shape(**a)


def cache(**over):
    a = dict(k=fake(0), v=fake(1), k_scale=fake(2), v_scale=fake(3), n_pages=64, page=16, block_table=fake(4), table_ld=8,
             max_blocks=8, kv_lens=fake(5))
    a.update({k: v for k, v in over.items() if k in a})
    return gdn.gdn_kv_cache(**a)


CACHE = ("page", "n_pages", "k_scale", "v_scale", "block_table", "table_ld", "max_blocks", "kv_lens")


def attn(L, **over):
    a = dict(q=fake(8), o=fake(9), ldq=1024, ldo=1024, cu_seqlens=None, causal=1, scale=0.0, workspace=None, workspace_bytes=0)
    a.update({k: v for k, v in over.items() if k in a})
    c = {k: v for k, v in over.items() if k in CACHE}
    c.update(over.get("cache", {}))
    return L.gdn_attn(ctypes.byref(shape(**over)), ctypes.byref(gdn.gdn_attn_io(cache=cache(**c), **a)), None)


def append(L, **over):
    a = dict(k=fake(8), v=fake(9), ldk=256, ldv=256, cu_seqlens=None)
    a.update({k: v for k, v in over.items() if k in a})
    c = {k: v for k, v in over.items() if k in CACHE}
    c.update(over.get("cache", {}))
    return L.gdn_kv_append(ctypes.byref(shape(**over)), ctypes.byref(gdn.gdn_kv_append_io(cache=cache(**c), **a)), None)


CACHE_CASES = [(1, dict(B=0)), (1, dict(T=0)), (1, dict(Hk=0)), (1, dict(D=0)), (1, dict(io_dtype=3)), (1, dict(max_new=-1)),
               (1, dict(max_kv=-1)), (1, dict(cache=dict(k=None))), (1, dict(cache=dict(v=None))), (1, dict(k_scale=None)),
               (1, dict(v_scale=None)), (1, dict(block_table=None)), (1, dict(kv_lens=None)), (1, dict(n_pages=0)),
               (1, dict(max_blocks=0)), (1, dict(table_ld=7)), (2, dict(D=96)), (2, dict(D=512)), (2, dict(page=8)),
               (2, dict(page=24)), (2, dict(page=256)), (2, dict(table_ld=1 << 33)), (2, dict(n_pages=1 << 28)),
               (2, dict(B=65537)), (2, dict(T=1 << 25)), (2, dict(max_blocks=1 << 27, table_ld=1 << 27)),
               (3, dict(cache=dict(k=fake(0, 8)))), (3, dict(cache=dict(v=fake(1, 1)))), (3, dict(k_scale=fake(2, 2))),
               (3, dict(block_table=fake(4, 2))), (3, dict(kv_lens=fake(5, 1))), (3, dict(cu_seqlens=fake(6, 2)))]


@pytest.mark.parametrize("status,bad", CACHE_CASES)
def test_cache_arguments(L, status, bad):
    assert attn(L, **bad) == status
    assert append(L, **bad) == status


def test_attn_arguments(L):
    assert L.gdn_attn(None, None, None) == 1
    assert attn(L) in OK_ON_HOST
    assert attn(L, cu_seqlens=fake(6), max_new=3, max_kv=100) in OK_ON_HOST
    for bad in (dict(q=None), dict(o=None), dict(ldq=1023), dict(ldo=8), dict(Hq=0), dict(scale=math.nan), dict(scale=math.inf)):
        assert attn(L, **bad) == 1, bad
    for bad in (dict(Hq=7), dict(Hq=130, Hk=2, ldq=130 * 128, ldo=130 * 128), dict(ldq=1 << 33)):
        assert attn(L, **bad) == 2, bad
    for bad in (dict(q=fake(8, 8)), dict(o=fake(9, 2)), dict(ldq=1028), dict(ldo=1025), dict(workspace=fake(10, 16), workspace_bytes=64)):
        assert attn(L, **bad) == 3, bad
    for bad in (dict(o=fake(8)), dict(o=fake(8, 512)), dict(o=fake(0, 1024)), dict(o=fake(3)), dict(o=fake(4)), dict(o=fake(5)),
                dict(workspace=fake(9), workspace_bytes=256), dict(workspace=fake(0), workspace_bytes=256)):
        assert attn(L, **bad) == 4, bad


def test_append_arguments(L):
    assert L.gdn_kv_append(None, None, None) == 1
    assert append(L) in OK_ON_HOST
    assert append(L, Hq=0) in OK_ON_HOST   # not used
    for bad in (dict(k=None), dict(v=None), dict(ldk=255), dict(ldv=0)):
        assert append(L, **bad) == 1, bad
    for bad in (dict(k=fake(8, 8)), dict(ldv=260)):
        assert append(L, **bad) == 3, bad
    for bad in (dict(k=fake(0)), dict(v=fake(1, 256)), dict(k=fake(2)), dict(cache=dict(v=fake(0))), dict(v_scale=fake(2)),
                dict(v_scale=fake(0)), dict(block_table=fake(3)), dict(kv_lens=fake(1))):
        assert append(L, **bad) == 4, bad


def rope(L, tokens=4, D=128, io=gdn.GDN_BF16, plan=None, positions=fake(7), xs=None, inverse=0, n=None):
    plan = plan or gdn.gdn_rope_plan(64)
    xs = xs or [(fake(0), fake(1), 512, 512, 4), (fake(2), fake(2), 256, 256, 2)]
    arr = (gdn.gdn_rope_x * max(1, len(xs)))(*[gdn.gdn_rope_x(*x) for x in xs])
    return L.gdn_rope(tokens, D, io, ctypes.byref(plan), positions, len(xs) if n is None else n, arr, inverse, None)


def test_rope_arguments(L):
    assert rope(L) in OK_ON_HOST
    broken = [gdn.gdn_rope_plan(64) for _ in range(4)]
    broken[0].rot, broken[1].rot, broken[2].layout, broken[3].m = 0, 130, 2, math.nan
    for bad in [dict(tokens=0), dict(D=0), dict(io=2), dict(positions=None), dict(n=0), dict(n=5), dict(D=32)] + [dict(plan=p) for p in broken]:
        assert rope(L, **bad) == 1, bad
    for x in ((None, fake(1), 512, 512, 4), (fake(0), None, 512, 512, 4), (fake(0), fake(1), 511, 512, 4), (fake(0), fake(1), 512, 1, 4),
              (fake(0), fake(1), 512, 512, 0)):
        assert rope(L, xs=[x]) == 1, x
    for bad in (dict(tokens=1 << 25), dict(D=2048, xs=[(fake(0), fake(1), 2048, 2048, 1)]), dict(xs=[(fake(0), fake(1), 1 << 33, 512, 4)])):
        assert rope(L, **bad) == 2, bad
    for bad in (dict(positions=fake(7, 2)), dict(xs=[(fake(0, 1), fake(1), 512, 512, 4)]), dict(io=gdn.GDN_F32, xs=[(fake(0, 2), fake(1), 512, 512, 4)])):
        assert rope(L, **bad) == 3, bad
    for xs in ([(fake(0), fake(0, 2), 512, 512, 4)], [(fake(0), fake(0), 512, 520, 4)], [(fake(0), fake(1), 512, 512, 4), (fake(2), fake(1), 512, 512, 4)],
               [(fake(0), fake(7), 512, 512, 4)], [(fake(0), fake(1), 512, 512, 4), (fake(1), fake(2), 512, 512, 4)]):
        assert rope(L, xs=xs) == 4, xs
    # q and k turned in place in one fused buffer; out into column blocks of one buffer
    assert rope(L, xs=[(fake(0), fake(0), 1024, 1024, 4), (fake(0, 1024), fake(0, 1024), 1024, 1024, 2)]) in OK_ON_HOST
    assert rope(L, xs=[(fake(0), fake(1), 1024, 768, 4), (fake(0, 1024), fake(1, 1024), 1024, 768, 2)]) in OK_ON_HOST
    assert rope(L, xs=[(fake(0, 2), fake(1, 6), 513, 515, 4)]) in OK_ON_HOST  # elements' own alignment


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0),
                                     dict(kind="parts", factor=16.0, original=4096), dict(kind="parts", factor=1.0, original=100, fast=2.0, slow=0.5)])
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_plans(rot, scaling, base):
    if rot == 2 and scaling and scaling["kind"] == "ntk":
        with pytest.raises(gdn.GdnError):
            gdn.gdn_rope_plan(rot, base=base, scaling=scaling)
        return
    p = gdn.gdn_rope_plan(rot, base=base, scaling=scaling, layout="interleaved")
    f, m = R.frequencies(rot, base, scaling)
    assert p.rot == rot and p.layout == 1 and abs(p.m - m) <= 2.0 ** -23 * m
    for i in range(rot // 2):  # a few roundings of 2^-53 in the powers
        want = float(f[i]) / (2 * math.pi)
        assert abs(p.turns[i] / 2.0 ** 64 - want) <= 64 * 2.0 ** -53 * want + 2.0 ** -64, i
    assert all(t == 0 for t in p.turns[rot // 2:])


def test_plans_refuse():
    for bad in (dict(rot=0), dict(rot=3), dict(rot=-2), dict(rot=258), dict(rot=64, base=1.0), dict(rot=64, base=math.nan),
                dict(rot=64, base=math.inf), dict(rot=64, scaling=dict(kind="linear", factor=0.5)),
                dict(rot=64, scaling=dict(kind="linear", factor=math.nan)), dict(rot=64, scaling=dict(kind="parts", factor=2.0)),
                dict(rot=64, scaling=dict(kind="parts", factor=2.0, original=100, fast=1.0, slow=1.0)),
                dict(rot=64, scaling=dict(kind="parts", factor=2.0, original=100, slow=0.0))):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_rope_plan(**bad)
    with pytest.raises(ValueError):
        gdn.gdn_rope_plan(64, scaling=dict(kind="linear", factor=2.0, other=1))
    with pytest.raises(KeyError):
        gdn.gdn_rope_plan(64, layout="both")


def pages(L, **over):
    a = dict(B=3, page=16, max_blocks=8, n_free=10, table_ld=8, max_tokens=20, kv_lens=fake(0), new_tokens=fake(1), free_pages=fake(2),
             free_used=fake(3), block_table=fake(4), kv_lens_out=fake(5), free_used_out=fake(6), cu_seqlens=fake(7), slots=fake(8),
             positions=fake(9))
    a.update(over)
    return L.gdn_kv_pages(ctypes.byref(gdn.gdn_kv_pages_io(**a)), None)


def test_pages_arguments(L):
    assert L.gdn_kv_pages(None, None) == 1
    assert pages(L) in OK_ON_HOST
    assert pages(L, kv_lens_out=fake(0), free_used_out=fake(3)) in OK_ON_HOST   # in place
    assert pages(L, slots=None, positions=None) in OK_ON_HOST
    assert pages(L, n_free=0, free_pages=None) in OK_ON_HOST
    for bad in [dict(B=0), dict(max_blocks=0), dict(n_free=-1), dict(max_tokens=-1), dict(table_ld=7)] + \
            [{n: None} for n in ("kv_lens", "new_tokens", "free_pages", "free_used", "block_table", "kv_lens_out", "free_used_out", "cu_seqlens")]:
        assert pages(L, **bad) == 1, bad
    for bad in (dict(page=0), dict(page=48), dict(B=16385), dict(table_ld=1 << 33), dict(max_tokens=1 << 31), dict(max_blocks=1 << 27, table_ld=1 << 27)):
        assert pages(L, **bad) == 2, bad
    for bad in (dict(kv_lens=fake(0, 2)), dict(slots=fake(8, 4)), dict(positions=fake(9, 1)), dict(cu_seqlens=fake(7, 2))):
        assert pages(L, **bad) == 3, bad
    for bad in (dict(kv_lens_out=fake(0, 4)), dict(kv_lens_out=fake(1)), dict(cu_seqlens=fake(0)), dict(block_table=fake(2)),
                dict(slots=fake(4)), dict(positions=fake(7)), dict(free_used_out=fake(0, 8))):
        assert pages(L, **bad) == 4, bad


def test_the_binding_refuses_other_tensors():
    c = R.Cache([20, 5], 2, 64, 16).fill()
    x = torch.zeros(4, 128).bfloat16()
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    call = dict(cu_seqlens=cu)
    for bad, kw in (((x, x), {}), ((x.view(2, 2, 128), x.view(2, 2, 128)), call), ((x, x[:3]), call), ((x, x[:, :64]), call),
                    ((x, x), dict(cu_seqlens=cu.long())), ((x, x), dict(cu_seqlens=cu[:2]))):
        with pytest.raises(ValueError):
            gdn.gdn_kv_append(*bad, *c.args(), **kw)
        with pytest.raises(ValueError):
            gdn.gdn_attn(*bad, *c.args(), Hq=2, **kw)
    for bad in ((x, x.float()), (x.half(), x.half())):
        with pytest.raises(TypeError):
            gdn.gdn_kv_append(*bad, *c.args(), **call)
        with pytest.raises(TypeError):
            gdn.gdn_attn(*bad, *c.args(), Hq=2, **call)
    kv, table, k8, v8, sk, sv = c.args()
    for args in ((kv.long(), table, k8, v8, sk, sv), (kv, table[:1], k8, v8, sk, sv), (kv, table.long(), k8, v8, sk, sv),
                 (kv, table, k8, v8[:2], sk, sv), (kv, table, k8.int(), v8, sk, sv), (kv, table, k8, v8, sk[:1], sv),
                 (kv, table, k8, v8, sk, sv.double()), (kv, table, k8.transpose(1, 2), v8.transpose(1, 2), sk, sv)):
        with pytest.raises(ValueError):
            gdn.gdn_attn(x, x, *args, Hq=2, **call)
    plan, pos = gdn.gdn_rope_plan(64), torch.zeros(4, dtype=torch.int32)
    for p, t in ((pos.long(), [(x, x)]), (pos[:3], [(x, x)]), (pos, [(x, x[:, :64])]), (pos, [(x[:, :96], x[:, :96])])):
        with pytest.raises(ValueError):
            gdn.gdn_rope(plan, p, t, D=64)
    with pytest.raises(TypeError):
        gdn.gdn_rope(plan, pos, [(x, x.float())], D=64)


# ------------------------------------------------- the forms the GPU is held to
def test_e4m3_form():
    x = torch.cat([torch.linspace(-500, 500, 4001), torch.linspace(-0.03, 0.03, 4001), torch.tensor([464.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    assert torch.equal(R.e4m3(x).float(), x.clamp(-448, 448).to(torch.float8_e4m3fn).float())
    assert R.e4m3(torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]


def test_scale_form():
    a = torch.tensor([448.0, 449.0, 7.0, 7.0001, 57344.0, 1e9, 0.0, math.inf, 2.0 ** -118], dtype=torch.float64)
    s = R.scale_for(a)
    assert s[:7].tolist() == [1.0, 2.0, 2.0 ** -6, 2.0 ** -5, 128.0, 128.0, 2.0 ** -120] and s[7].isnan() and s[8] == 2.0 ** -120


def test_attention_form_by_hand():
    q = torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]]])
    k = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]], [[1.0, 1.0]]])
    v = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]], [[5.0, 5.0]]])
    o, _, _ = R.attend(q, k, v, 2, True, 1.0)
    e = math.e
    assert torch.allclose(o[0, 0], torch.tensor([e, 1.0], dtype=torch.float64) / (e + 1))
    w = [1.0, e ** 2, e ** 2]
    assert torch.allclose(o[1, 0], torch.tensor([w[0] + 5 * w[2], w[1] + 5 * w[2]], dtype=torch.float64) / sum(w))
    o, _, _ = R.attend(q, k[:1], v[:1], 2, True, 1.0)
    assert o[0].abs().max() == 0 and o[1, 0].tolist() == [1.0, 0.0]


def test_rope_form_by_hand():
    f, m = R.frequencies(4, 100.0)
    assert f.tolist() == [1.0, 0.1] and m == 1.0
    x = torch.tensor([[1.0, 2.0, 3.0, 4.0, 9.0]])
    c, s, c1, s1 = math.cos(3), math.sin(3), math.cos(0.3), math.sin(0.3)
    p = torch.tensor([3])
    assert torch.allclose(R.rope(x, p, 4, 5, f, m, "half")[0], torch.tensor(
        [c - 3 * s, 2 * c1 - 4 * s1, 3 * c + s, 4 * c1 + 2 * s1, 9.0], dtype=torch.float64))
    assert torch.allclose(R.rope(x, p, 4, 5, f, m, "interleaved")[0], torch.tensor(
        [c - 2 * s, 2 * c + s, 3 * c1 - 4 * s1, 4 * c1 + 3 * s1, 9.0], dtype=torch.float64))


def test_append_form():
    """A page filled in two calls: the second's larger token moves the first's bytes by whole exponents."""
    c = R.Cache([3], 1, 64, 16)
    c.lens = [3]
    k = torch.zeros(4, 1, 64)
    k[:, 0, 0] = torch.tensor([1.0, -0.5, 0.25, 8.0])
    R.append([k[:3]], [k[:3]], c, [3], [3])
    p = int(c.table[0, 0])
    assert c.sk[p, 0] == 2.0 ** -8 and c.k8.view(torch.float8_e4m3fn)[p, 0, :3, 0].float().tolist() == [256.0, -128.0, 64.0]
    R.append([k[3:]], [k[3:]], c, [4], [1])
    assert c.sk[p, 0] == 2.0 ** -5
    assert (c.k8.view(torch.float8_e4m3fn)[p, 0, :4, 0].float() * c.sk[p, 0]).tolist() == [1.0, -0.5, 0.25, 8.0]
