"""GPU parity of linear attention with decay (gdn_linattn_prefill, _decode)
against the token loop in 64 bits.

Tolerances, from the formulas (A: the same sums over absolute values):
  o, bf16 io     2^-8 |o| for the stored rounding (half a step) plus 2^-14 A:
                 operands in two bf16 pieces are off by 2^-17 each, the decay
                 ratios by 2^-18, at most 64 truncating sums by 2^-23 each.
  S_T, bf16 io   2^-18 A: three pieces 2^-24, twelve truncating sums per
                 chunk 2^-19.4, the decays and one fp32 sum per chunk.
  fp32 io        (2 T + 160) 2^-24 A: one fused multiply-add and one product
                 per token, a 128-term sum.
Decode runs the fp32 arithmetic whatever the io type."""
import math

import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn
from linattn_reference import D, Guarded, recur

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert torch.cuda.is_available()
    assert gdn.gdn_device_status(reset=True) == 0


def gates(n, Hv, kind, rng):
    if kind == "head":
        return None, -torch.exp2(-8.0 * torch.arange(1, Hv + 1) / Hv)
    mu = {"token": 3.0, "fast": -2.0}[kind]
    return -torch.nn.functional.softplus(-(mu + torch.randn(n, Hv, generator=rng))), None


class Case:
    """Inputs on the host (exact values of the io type) and the 64-bit results per sequence."""

    def __init__(self, lens, Hk, Hv, io, kind="token", s0=True, seed=1, edit=None, scale=0.0):
        rng = torch.Generator().manual_seed(seed)
        n = sum(lens)
        self.lens, self.Hk, self.Hv, self.scale = lens, Hk, Hv, scale
        self.dt = torch.bfloat16 if io == "bf16" else torch.float32
        self.q, self.k = (torch.nn.functional.silu(torch.randn(n, Hk * D, generator=rng)).to(self.dt) for _ in range(2))
        self.v = torch.randn(n, Hv * D, generator=rng).to(self.dt)
        self.g, self.ld = gates(n, Hv, kind, rng)
        self.S0 = 0.1 * torch.randn(len(lens), Hv, D, D, generator=rng) if s0 else None
        if edit:
            edit(self)

    def reference(self, b):
        at, n = sum(self.lens[:b]), self.lens[b]
        g = self.g[at:at + n].double() if self.g is not None else self.ld.double().expand(n, self.Hv)
        f = lambda x, H: x[at:at + n].double().view(n, H, D)  # noqa: E731
        return recur(f(self.q, self.Hk), f(self.k, self.Hk), f(self.v, self.Hv), g,
                     None if self.S0 is None else self.S0[b].double(), self.scale or None)

    def check(self, o, S, decode=False, skip=()):
        o, S = o.cpu().double().view(-1, self.Hv, D), S.cpu().double()
        for b, n in enumerate(self.lens):
            if b in skip:
                continue
            at = sum(self.lens[:b])
            ro, rS, Ao, AS = self.reference(b)
            fp32 = decode or self.dt == torch.float32
            eS = (2 * n + 160) * 2.0 ** -24 * AS if fp32 else 2.0 ** -18 * AS
            eo = (2 * n + 160) * 2.0 ** -24 * Ao if fp32 else 2.0 ** -14 * Ao
            eo = eo + (2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24) * ro.abs()
            dS, do = (S[b] - rS).abs(), (o[at:at + n] - ro).abs()
            assert bool((dS <= eS + 1e-30).all()), "S of sequence %d: %.3g of the bound" % (b, (dS / (eS + 1e-30)).max())
            assert bool((do <= eo + 1e-30).all()), "o of sequence %d: %.3g of the bound" % (b, (do / (eo + 1e-30)).max())


def fused(c, pad=0):
    """q, k, v as views of one wider buffer (rows `pad` elements apart beyond their width)."""
    w = (2 * c.Hk + c.Hv) * D
    buf = torch.full((c.q.shape[0], w + pad), 5.0, dtype=c.dt, device="cuda")
    buf[:, :c.Hk * D], buf[:, c.Hk * D:2 * c.Hk * D], buf[:, 2 * c.Hk * D:w] = c.q.cuda(), c.k.cuda(), c.v.cuda()
    return buf[:, :c.Hk * D], buf[:, c.Hk * D:2 * c.Hk * D], buf[:, 2 * c.Hk * D:w]


def cuda(t):
    return None if t is None else t.cuda()


def prefill(c, packed=False, workspace=True, in_place=False, pad=0, stream=None):
    B, n = len(c.lens), sum(c.lens)
    q, k, v = fused(c, pad)
    o = Guarded((n, c.Hv * D), c.dt, ld=c.Hv * D + pad)
    S = Guarded((B, c.Hv, D, D), torch.float32)
    S0, ot = cuda(c.S0), o.t
    if in_place:
        S.t.copy_(S0)
        S0 = S.t
    cu = None
    if packed:
        at = [0]
        for x in c.lens:
            at.append(at[-1] + x)
        cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    else:
        T = c.lens[0]
        q, k, v, ot = (x.unflatten(0, (B, T)) for x in (q, k, v, ot))
    need = gdn.gdn_linattn_workspace_bytes(B, n if packed else c.lens[0], c.Hk, c.Hv, packed=packed,
                                           io_dtype=gdn.GDN_BF16 if c.dt == torch.bfloat16 else gdn.GDN_F32)
    ws = Guarded((need,), torch.uint8) if workspace and need else None
    gdn.gdn_linattn_prefill(q, k, v, S0, ot, S.t, Hk=c.Hk, Hv=c.Hv, g=cuda(c.g), log_decay=cuda(c.ld), cu_seqlens=cu,
                            workspace=None if ws is None else ws.t, scale=c.scale, stream=stream)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    assert o.intact() and S.intact() and (ws is None or ws.intact())
    return o.t, S.t


@pytest.mark.parametrize("T", [1, 2, 16, 63, 64, 65, 127, 128, 200, 321])
@pytest.mark.parametrize("kind", ["token", "head"])
def test_prefill_lengths(T, kind):
    c = Case([T, T], 1, 2, "bf16", kind, seed=T)
    c.check(*prefill(c))


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 2), (2, 6), (4, 4)])
def test_prefill_heads(Hk, Hv):
    c = Case([150], Hk, Hv, "bf16", s0=False, seed=Hv)
    c.check(*prefill(c, pad=64))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_fast_decay_resets_and_scale(io):
    """Decays that underflow within a chunk, resets anywhere in it, an odd scale."""
    def edit(c):
        c.g[[0, 5, 63, 64, 100], 0] = -math.inf
        c.g[70, 1] = -1e4
        c.g[10:20, 1] = -60.0
        c.g[20:30, 1] = 0.0
    c = Case([140], 1, 2, io, "fast", edit=edit, scale=-0.37)
    c.check(*prefill(c))


def test_prefill_one_head_scaled_far_from_one():
    """Values of 1e-18 and 1e15: the pieces keep bf16's range."""
    def edit(c):
        c.k[:] = (c.k.float() * 1e-18).bfloat16()
        c.v[:] = (c.v.float() * 1e15).bfloat16()
        c.S0 *= 1e-3
    c = Case([100], 1, 1, "bf16", edit=edit)
    c.check(*prefill(c))


@pytest.mark.parametrize("T", [1, 7, 8, 9, 65])
def test_prefill_fp32(T):
    c = Case([T, T], 2, 4, "f32", seed=20 + T)
    c.check(*prefill(c, pad=4))


@pytest.mark.parametrize("kind", ["token", "head"])
def test_prefill_in_segments(kind):
    """Few units and a long prompt: several segments, with and without S0 in place."""
    c = Case([2000], 1, 2, "bf16", kind, seed=31)
    need = gdn.gdn_linattn_workspace_bytes(1, 2000, 1, 2)
    assert need > 0
    o1, S1 = prefill(c)
    c.check(o1, S1)
    o2, S2 = prefill(c, in_place=True)
    assert torch.equal(o1, o2) and torch.equal(S1, S2)
    c.check(*prefill(c, workspace=False))
    c = Case([1025], 1, 1, "bf16", kind, s0=False, seed=32)
    c.check(*prefill(c))


def test_prefill_packed_ragged_with_empty_sequences():
    c = Case([70, 0, 64, 1, 129, 0, 33], 1, 2, "bf16", seed=40)
    c.check(*prefill(c, packed=True))
    c = Case([5, 0, 17], 1, 2, "f32", seed=41)
    c.check(*prefill(c, packed=True))
    # segments of very unequal sequences, one of them shorter than a segment
    c = Case([1800, 0, 30], 1, 1, "bf16", seed=42)
    assert gdn.gdn_linattn_workspace_bytes(3, 1830, 1, 1, packed=True) > 0
    c.check(*prefill(c, packed=True))


def test_nothing_flows_between_packed_sequences():
    """NaN and infinities in one sequence's q, k, v leave its neighbours alone,
    although their last chunks end inside its rows' tiles."""
    def edit(c):
        c.q[40:80], c.k[40:80] = math.nan, math.inf
        c.v[40:80] = math.nan
    c = Case([40, 40, 50], 1, 2, "bf16", seed=43, edit=edit)
    o, S = prefill(c, packed=True)
    c.check(o, S, skip=(1,))
    assert bool(o[40:80].isnan().any())


def test_packed_offsets_out_of_range_are_reported_and_skipped():
    c = Case([64, 64], 1, 1, "bf16", seed=44)
    q, k, v = fused(c)
    for cu in ([0, 100, 64], [0, 64, 129], [-1, 64, 128]):
        o, S = Guarded((128, D), c.dt), Guarded((2, 1, D, D), torch.float32)
        S.t.fill_(3.0)
        gdn.gdn_linattn_prefill(q, k, v, None, o.t, S.t, Hk=1, Hv=1, g=c.g.cuda(),
                                cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert gdn.gdn_device_status(reset=True) == gdn.GDN_ERR_INVALID_ARG
        assert o.intact() and S.intact()
        bad = 0 if cu[0] < 0 else 1
        assert bool((S.t[bad] == 3.0).all())
    assert gdn.gdn_device_status() == 0


def test_prefill_continues_and_repeats_bit_for_bit():
    c = Case([300], 2, 4, "bf16", seed=50)
    o, S = prefill(c)
    o2, S2 = prefill(c)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    # the same prompt in two calls, the state carried
    a, b = Case([300], 2, 4, "bf16", seed=50), Case([300], 2, 4, "bf16", seed=50)
    for x, sl in ((a, slice(0, 171)), (b, slice(171, 300))):
        x.q, x.k, x.v, x.g, x.lens = x.q[sl], x.k[sl], x.v[sl], x.g[sl], [sl.stop - sl.start]
    oa, Sa = prefill(a)
    b.S0 = Sa.cpu()
    ob, Sb = prefill(b)
    c.check(torch.cat([oa, ob]), Sb)


def decode(c, pad=0):
    B, T = len(c.lens), c.lens[0]
    q, k, v = (x.unflatten(0, (B, T)) for x in fused(c, pad))
    o = Guarded((B, T, c.Hv * D), c.dt, ld=c.Hv * D + pad)
    S = Guarded((B, c.Hv, D, D), torch.float32)
    S.t.copy_(c.S0)
    gdn.gdn_linattn_decode(q, k, v, S.t, o.t, Hk=c.Hk, Hv=c.Hv, g=cuda(c.g), log_decay=cuda(c.ld), scale=c.scale)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0 and o.intact() and S.intact()
    return o.t.reshape(B * T, -1), S.t


@pytest.mark.parametrize("B,T,Hk,Hv", [(1, 1, 1, 1), (1, 1, 16, 16), (3, 1, 2, 6), (50, 1, 1, 2), (160, 1, 1, 1),
                                       (2, 4, 2, 4), (1, 8, 1, 1), (40, 9, 2, 4), (2, 17, 1, 3)])
@pytest.mark.parametrize("io,kind", [("bf16", "token"), ("bf16", "head"), ("f32", "token")])
def test_decode(B, T, Hk, Hv, io, kind):
    c = Case([T] * B, Hk, Hv, io, kind, seed=B + T)
    c.check(*decode(c, pad=8), decode=True)


def test_decode_reset_and_prompt_then_tokens():
    def edit(c):
        c.g[1] = -math.inf
    c = Case([3, 3], 1, 2, "bf16", edit=edit, seed=60)
    c.check(*decode(c), decode=True)


def test_side_stream_and_graph():
    c = Case([2000], 1, 2, "bf16", seed=70)
    want = prefill(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = prefill(c, stream=s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    q, k, v = (x.unsqueeze(0) for x in fused(c))
    o, S, S0, g = torch.empty_like(v.contiguous()), torch.empty(1, 2, D, D, device="cuda"), c.S0.cuda(), c.g.cuda()
    ws = torch.empty(gdn.gdn_linattn_workspace_bytes(1, 2000, 1, 2), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_linattn_prefill(q, k, v, S0, o, S, Hk=1, Hv=2, g=g, workspace=ws)
        gdn.gdn_linattn_decode(q[:, :1], k[:, :1], v[:, :1], S, o[:, :1], Hk=1, Hv=2, g=g[:1])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    assert torch.equal(o[0, 1:], want[0][1:])


@pytest.mark.parametrize("io,T", [("bf16", 4096), ("bf16", 90), ("f32", 512)])
def test_very_slow_constant_decay(io, T):
    """A half-life of 100,000 tokens, q = v = 0: the state is S0 e^{T g}, up to
    two roundings of the state per application of a decay (2^-24 each, worst
    case all one way: a constant decay takes the same step every time)."""
    g = -6.9e-6
    q = torch.zeros(1, T, D, dtype=torch.bfloat16 if io == "bf16" else torch.float32, device="cuda")
    S0 = torch.rand(1, 1, D, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) + 0.5
    S, o = torch.empty_like(S0), torch.empty_like(q)
    for ws in (False, True):
        n = gdn.gdn_linattn_workspace_bytes(1, T, 1, 1) if io == "bf16" else 0
        gdn.gdn_linattn_prefill(q, q, q, S0, o, S, Hk=1, Hv=1, log_decay=torch.tensor([g], device="cuda"),
                                workspace=torch.empty(n, dtype=torch.uint8, device="cuda") if ws and n else None)
        torch.cuda.synchronize()
        ratio = (S.double() / S0.double()) / math.exp(T * float(torch.tensor(g)))
        assert (ratio - 1).abs().max().item() < 2 * T * 2.0 ** -24


# Units below and above the number of SMs, tokens short of, at and past the groups' and blocks' ends.
@pytest.mark.parametrize("B,Hk,Hv", [(3, 1, 2), (40, 2, 4)])
@pytest.mark.parametrize("T", [3, 4, 5, 8, 12, 23])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decode_several_tokens(B, Hk, Hv, T, io):
    c = Case([T] * B, Hk, Hv, io, seed=90 + T)
    c.check(*decode(c, pad=8), decode=True)


@pytest.mark.parametrize("lens", [[1, 0, 2, 1, 1], [0, 37, 3, 4, 12, 1], [2] * 40 + [9, 0, 30] + [5] * 40])
def test_prefill_fp32_packed(lens):
    c = Case(lens, 1, 2, "f32", seed=120 + len(lens))
    c.check(*prefill(c, packed=True))
