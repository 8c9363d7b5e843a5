"""Linear attention at unusual decays: NaN, strong ones in front of slow ones,
resets of a large state.  Tolerances as in test_gpu_linattn.py."""
import math

import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn
from linattn_reference import D
from test_gpu_linattn import Case, decode, prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert gdn.gdn_device_status(reset=True) == 0


def check_with_nan(c, o, S, token_loop):
    """NaN exactly where the 64-bit loop has it, the rest within the tolerances."""
    o, S = o.cpu().double().view(-1, c.Hv, D), S.cpu().double()
    for b, n in enumerate(c.lens):
        at = sum(c.lens[:b])
        ro, rS, Ao, AS = c.reference(b)
        e = (2 * n + 160) * 2.0 ** -24
        half = 2.0 ** -8 if c.dt == torch.bfloat16 else 2.0 ** -24
        for got, ref, bound in ((S[b], rS, (e if token_loop else 2.0 ** -18) * AS),
                                (o[at:at + n], ro, (e if token_loop else 2.0 ** -14) * Ao + half * ro.abs())):
            assert torch.equal(got.isnan(), ref.isnan())
            ok = ~ref.isnan()
            assert bool(((got - ref).abs()[ok] <= bound[ok] + 1e-30).all())


@pytest.mark.parametrize("io,T", [("bf16", 20), ("bf16", 200), ("bf16", 2000), ("f32", 70)])
@pytest.mark.parametrize("where", [0, 17, -1])
def test_nan_decay_reaches_everything_behind_it(io, T, where):
    """From its token on, in its head: outputs and the state; nothing else.  20 tokens run token
    by token, 200 in chunks, 2000 in segments."""
    def edit(c):
        c.g[where, 0] = math.nan
    c = Case([T], 1, 2, io, seed=200 + T, edit=edit)
    check_with_nan(c, *prefill(c), io == "f32" or T == 20)


def test_nan_decay_of_a_token_from_the_cache_and_of_a_head():
    def edit(c):
        c.g[1, 1] = math.nan
    c = Case([3], 1, 2, "bf16", seed=210, edit=edit)
    check_with_nan(c, *decode(c), True)

    def head(c):
        c.ld[0] = math.nan
    c = Case([150], 1, 2, "bf16", "head", seed=211, edit=head)
    check_with_nan(c, *prefill(c), False)


def test_nan_decay_stays_in_its_sequence():
    def edit(c):
        c.g[100, 0] = math.nan
    c = Case([70, 40, 129], 1, 2, "bf16", seed=212, edit=edit)
    check_with_nan(c, *prefill(c, packed=True), False)


@pytest.mark.parametrize("strong", [-1.0, -5.0, -10.0, -20.0, -40.0, -80.0, -math.inf])
@pytest.mark.parametrize("first", [0, 20])
def test_slow_decays_behind_strong_ones(strong, first):
    """40 strong decays, then pairs of tokens that cancel: v of the second is minus the first's after its
    decay, so that o is what the rounding of v leaves and an error of the ratio of their decays shows."""
    def edit(c):
        c.g[:] = -0.3 * torch.rand(c.g.shape, generator=torch.Generator().manual_seed(1))
        c.g[first:first + 40] = strong
        for t in range(first + 40, 128, 2):
            c.k[t + 1] = c.k[t]
            for h in range(c.Hv):
                cols = slice(h * D, (h + 1) * D)
                c.v[t + 1, cols] = -(c.v[t, cols].double() * math.exp(c.g[t + 1, h])).to(c.dt)
    c = Case([128], 1, 2, "bf16", seed=220, edit=edit)
    c.check(*prefill(c))


def test_reset_of_a_large_state():
    """Behind a reset inside a chunk an output still sees 2^-58 of the state at the chunk's start, and
    the state e^-80 of what it was; both count in the bound, nothing else does."""
    def edit(c):
        c.S0 *= 1e9
        c.g[[5, 90]] = -math.inf
    c = Case([130], 1, 2, "bf16", seed=230, edit=edit)
    o, S = (x.cpu().double() for x in prefill(c))
    ro, rS, Ao, AS = c.reference(0)
    q = c.q.double().abs().view(-1, 1, 1, D)
    left = 2.0 ** -58 / math.sqrt(D) * (c.S0[0].double().abs() * q).sum(-1)  # [T, Hv, D]
    bound = 2.0 ** -14 * Ao + 2.0 ** -8 * ro.abs() + 1.01 * left
    assert bool(((o.view(-1, 2, D) - ro).abs() <= bound).all())
    assert bool(((S[0] - rS).abs() <= 2.0 ** -18 * AS + math.exp(-80) * c.S0[0].double().abs()).all())


def test_large_outputs_behind_a_reset():
    """Sums behind strong decays carry a factor of 2^58: outputs around 2^52 come out whole."""
    def edit(c):
        c.g[10] = -math.inf
        c.v[:] = (c.v.float() * 2.0 ** 50).bfloat16()
        c.S0 *= 2.0 ** 50
    c = Case([130], 1, 2, "bf16", seed=231, edit=edit)
    c.check(*prefill(c))
