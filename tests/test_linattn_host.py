"""Host-side checks of gdn_linattn_* and gdn_linear_ex that need no GPU: bad
arguments are refused before the device is touched (addresses are never
dereferenced)."""
import ctypes

import pytest
import torch

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


def call(L, entry="gdn_linattn_prefill", B=2, T=8, Hk=2, Hv=4, D=128, io=gdn.GDN_BF16, q_scale=0.0, **over):
    sh = gdn.make_shape(B, T, Hk, Hv, D, io, q_scale=q_scale)
    a = dict(q=fake(0), k=fake(1), v=fake(2), ldq=Hk * D, ldk=Hk * D, ldv=Hv * D, ldo=Hv * D, g=fake(3), log_decay=None,
             S0=fake(4), o=fake(5), S_T=fake(6), cu_seqlens=None, workspace=None, workspace_bytes=0)
    if entry == "gdn_linattn_decode":
        a["S0"] = None
    a.update(over)
    return getattr(L, entry)(ctypes.byref(sh), ctypes.byref(gdn.gdn_linattn_io(**a)), None)


def test_linattn_arguments(L):
    sh = gdn.make_shape(1, 1, 1, 1, 128, gdn.GDN_BF16)
    assert L.gdn_linattn_prefill(None, None, None) == 1
    assert L.gdn_linattn_decode(ctypes.byref(sh), None, None) == 1
    for bad in (dict(B=0), dict(T=0), dict(io=5), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(S_T=None),
                dict(g=None), dict(log_decay=fake(7)), dict(ldq=255), dict(ldk=128), dict(ldv=500), dict(ldo=0),
                dict(q_scale=float("inf"))):
        assert call(L, **bad) == 1, bad
    for bad in (dict(D=64, ldq=256, ldk=256, ldv=512, ldo=512), dict(Hk=3, Hv=4), dict(ldq=1 << 33), dict(T=1 << 30)):
        assert call(L, **bad) == 2, bad
    for bad in (dict(q=fake(0, 8)), dict(ldq=260), dict(ldo=516), dict(S_T=fake(6, 4)), dict(g=fake(3, 2)),
                dict(workspace=fake(8, 16), workspace_bytes=1 << 20)):
        assert call(L, **bad) == 3, bad
    assert call(L, io=gdn.GDN_F32, ldq=260, ldk=260) in OK_ON_HOST  # 16-byte rows in fp32
    assert call(L) in OK_ON_HOST
    assert call(L, S_T=fake(4)) in OK_ON_HOST                       # in place
    assert call(L, S0=None, g=None, log_decay=fake(3, 4)) in OK_ON_HOST


def test_linattn_aliases(L):
    for bad in (dict(o=fake(2)), dict(o=fake(0, 64)), dict(S_T=fake(4, 4096)), dict(S_T=fake(1)), dict(o=fake(6)),
                dict(workspace=fake(4), workspace_bytes=4096), dict(workspace=fake(5), workspace_bytes=4096)):
        assert call(L, **bad) == 4, bad
    # views of one buffer: o between v's rows still overlaps v's extent
    assert call(L, ldv=1024, o=fake(2, 1024), ldo=1024) == 4


def test_linattn_decode_takes_the_state_in_place(L):
    d = "gdn_linattn_decode"
    assert call(L, d) in OK_ON_HOST
    for bad in (dict(S0=fake(4)), dict(cu_seqlens=fake(7)), dict(workspace=fake(8), workspace_bytes=4096)):
        assert call(L, d, **bad) == 1, bad
    assert call(L, d, o=fake(6)) == 4


def test_workspace_of_nothing_to_run(L):
    assert L.gdn_linattn_workspace_bytes(None, 0) == 0
    assert gdn.gdn_linattn_workspace_bytes(1, 4096, 1, 1, io_dtype=gdn.GDN_F32) == 0
    assert gdn.gdn_linattn_workspace_bytes(0, 4096, 1, 1) == 0


def linear(L, M=4, N=16, K=64, gated=0, x=fake(0), ldx=64, w=fake(1), ldw=64, bias=None, outs=None):
    outs = outs if outs is not None else [(0, 8, fake(2), 8, 0, None, 0), (8, 16, fake(3), 8, 1, fake(4), 8)]
    arr = (gdn.gdn_linear_ex_out * max(1, len(outs)))(*[gdn.gdn_linear_ex_out(*o) for o in outs])
    return L.gdn_linear_ex(M, N, K, gated, x, ldx, w, ldw, bias, len(outs), arr, None)


def test_linear_ex_arguments(L):
    assert linear(L) in OK_ON_HOST
    assert linear(L, gated=1, bias=fake(5)) in OK_ON_HOST
    for bad in (dict(M=0), dict(N=0), dict(K=0), dict(x=None), dict(w=None), dict(ldx=56), dict(outs=[]),
                dict(outs=[(0, 17, fake(2), 32, 0, None, 0)]), dict(outs=[(4, 4, fake(2), 8, 0, None, 0)]),
                dict(outs=[(0, 8, None, 8, 0, None, 0)]), dict(outs=[(0, 8, fake(2), 7, 0, None, 0)]),
                dict(outs=[(0, 8, fake(2), 8, 4, None, 0)]), dict(outs=[(0, 8, fake(2), 8, -1, None, 0)]),
                dict(outs=[(0, 8, fake(2), 8, 0, fake(3), 7)]),
                dict(outs=[(0, 8, fake(2), 8, 0, None, 0), (7, 16, fake(3), 16, 0, None, 0)]),
                dict(outs=[(2 * i, 2 * i + 2, fake(2 + i), 8, 0, None, 0) for i in range(5)])):
        assert linear(L, **bad) == 1, bad
    assert linear(L, ldx=1 << 33) == 2
    assert linear(L, M=1 << 30, N=1 << 28) == 2                  # more tiles than 31 bits count
    for bad in (dict(x=fake(0, 8)), dict(ldw=68), dict(bias=fake(5, 2)), dict(outs=[(0, 8, fake(2, 1), 8, 0, None, 0)]),
                dict(outs=[(0, 8, fake(2), 8, 0, fake(3, 1), 8)])):
        assert linear(L, **bad) == 3, bad
    for bad in (dict(outs=[(0, 8, fake(0, 64), 8, 0, None, 0)]), dict(outs=[(0, 8, fake(1), 8, 0, None, 0)]),
                dict(bias=fake(2), outs=[(0, 8, fake(2), 8, 0, None, 0)]),
                dict(outs=[(0, 8, fake(2), 8, 0, None, 0), (8, 16, fake(2, 16), 16, 0, None, 0)]),
                dict(outs=[(0, 8, fake(2), 8, 0, fake(2), 16)]),     # in place, but another stride
                dict(outs=[(0, 8, fake(2), 8, 0, None, 0), (8, 16, fake(3), 8, 0, fake(2), 8)])):
        assert linear(L, **bad) == 4, bad
    assert linear(L, outs=[(0, 8, fake(2), 8, 0, fake(2), 8)]) in OK_ON_HOST  # added in place
    # gated: the up rows of w count
    assert linear(L, gated=1, outs=[(0, 8, fake(1, 20 * 128), 8, 0, None, 0)]) == 4


def test_binding_refuses_what_it_can_see():
    bf = torch.bfloat16
    q, v = torch.zeros(2, 3, 256, dtype=bf), torch.zeros(2, 3, 512, dtype=bf)
    S, g = torch.zeros(2, 4, 128, 128), torch.zeros(2, 3, 4)
    ok = dict(q=q, k=q.clone(), v=v, S=S, o=torch.zeros_like(v), Hk=2, Hv=4, g=g)

    def bad(err, **kw):
        a = dict(ok, **kw)
        with pytest.raises(err):
            gdn.gdn_linattn_decode(a["q"], a["k"], a["v"], a["S"], a["o"], Hk=a["Hk"], Hv=a["Hv"], g=a["g"])

    bad(TypeError, k=q.float())
    bad(TypeError, q=q.half(), k=q.half(), v=v.half(), o=v.half())
    bad(ValueError, k=q[:, :2])
    bad(ValueError, o=v[:1])
    bad(ValueError, S=S[:1])
    bad(ValueError, S=S.double())
    bad(ValueError, g=g[:, :2])
    bad(ValueError, q=torch.zeros(2, 3, 512, dtype=bf)[..., ::2])
    bad(ValueError, q=torch.zeros(2, 4, 256, dtype=bf)[:, :3])  # a gap between the sequences
    x, w, y = torch.zeros(2, 16, dtype=bf), torch.zeros(6, 16, dtype=bf), torch.zeros(2, 6, dtype=bf)
    for kw, err in ((dict(w=w[:, :8]), ValueError), (dict(w=w[:5], gated=True), ValueError),
                    (dict(bias=torch.zeros(5, dtype=bf)), ValueError), (dict(y=y.float()), TypeError),
                    (dict(y=y[:, :5]), ValueError), (dict(y=y[:1]), ValueError), (dict(act="tanh"), KeyError)):
        with pytest.raises(err):
            gdn.gdn_linear_ex(x, kw.get("w", w), [(0, 6, kw.get("y", y), kw.get("act", "none"))], bias=kw.get("bias"),
                              gated=kw.get("gated", False))


def test_packed_layouts_are_the_structures():
    """What the binding packs by hand lies where the C structures have it."""
    for fmt, cls in ((gdn._PACK_SHAPE, gdn.gdn_shape), (gdn._PACK_LINATTN, gdn.gdn_linattn_io),
                     (gdn._PACK_LINEAR_OUT, gdn.gdn_linear_ex_out)):
        assert fmt.size == ctypes.sizeof(cls)
        vals = [float(i) if t is ctypes.c_float else i for i, (_, t) in enumerate(cls._fields_, 1)]
        got = cls.from_buffer_copy(fmt.pack(*vals))
        assert [getattr(got, f) for f, _ in cls._fields_] == vals


def test_linear_ex_outputs_may_be_column_blocks_of_one_buffer(L):
    def two(off, wa=8, wb=8, ld=24, ld2=None):
        return [(0, wa, fake(2), ld, 0, None, 0), (16 - wb, 16, fake(2, off), ld2 or ld, 0, None, 0)]
    assert linear(L, outs=two(16)) in OK_ON_HOST                  # right behind the first block
    assert linear(L, outs=two(32)) in OK_ON_HOST                  # the last 8 of 24 columns
    assert linear(L, outs=two(48 * 3 + 16)) in OK_ON_HOST         # the same block, three rows further down
    assert linear(L, outs=two(14)) == 4                           # one column shared
    assert linear(L, outs=two(34)) == 4                           # the last column is the next row's first
    assert linear(L, outs=two(16, ld2=32)) == 4                   # another stride
    # the earlier block behind the later one, and a residual next to an output
    assert linear(L, outs=[(8, 16, fake(2, 16), 24, 0, None, 0), (0, 8, fake(2), 24, 0, None, 0)]) in OK_ON_HOST
    assert linear(L, outs=[(0, 8, fake(2), 24, 0, fake(2, 16), 24)]) in OK_ON_HOST
    assert linear(L, outs=[(0, 8, fake(2), 24, 0, fake(2, 8), 24)]) == 4
