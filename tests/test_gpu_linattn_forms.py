"""The ways a bf16 prompt runs (chunks, segments, parts of segments, many units)
against the token loop in 64 bits.  Each test asks first how its call runs, so
that it fails when the rule for that moves.  Tolerances as in test_gpu_linattn.py."""
import random

import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn
from linattn_reference import D, recur
from test_gpu_linattn import Case, prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert gdn.gdn_device_status(reset=True) == 0


def form(c, packed=False):
    f = gdn.gdn_selftest_linattn_form(len(c.lens), sum(c.lens) if packed else c.lens[0], c.Hk, c.Hv, packed)
    return bool(f.chunked), f.segments, f.parts


def check_some(c, o, S, sequences, heads):
    """Those sequences and heads of the result."""
    o, S = o.cpu().double().view(-1, c.Hv, D), S.cpu().double()
    kh = [h // (c.Hv // c.Hk) for h in heads]
    for b in sequences:
        n, at = c.lens[b], sum(c.lens[:b])
        f = lambda x, H, pick: x[at:at + n].double().view(n, H, D)[:, pick]  # noqa: E731
        g = c.g[at:at + n].double() if c.g is not None else c.ld.double().expand(n, c.Hv)
        ro, rS, Ao, AS = recur(f(c.q, c.Hk, kh), f(c.k, c.Hk, kh), f(c.v, c.Hv, heads), g[:, heads],
                               None if c.S0 is None else c.S0[b, heads].double())
        dS, do = (S[b, heads] - rS).abs(), (o[at:at + n, heads] - ro).abs()
        assert bool((dS <= 2.0 ** -18 * AS + 1e-30).all()), "S of %d: %.3g of the bound" % (b, (dS / (2.0 ** -18 * AS)).max())
        eo = 2.0 ** -14 * Ao + 2.0 ** -8 * ro.abs() + 1e-30
        assert bool((do <= eo).all()), "o of %d: %.3g of the bound" % (b, (do / eo).max())


@pytest.mark.parametrize("T", [25, 33, 47, 63, 64, 65])
def test_prompts_of_one_chunk_or_less(T):
    """With many heads these run in chunks, the only one of a call short or just full."""
    c = Case([T] * 64, 2, 8, "bf16", seed=300 + T)
    assert form(c) == (True, 1, 1)
    check_some(c, *prefill(c, pad=8), sequences=(0, 1, 30, 63), heads=[0, 3, 7])


@pytest.mark.parametrize("T,kind", [(200, "token"), (321, "head")])
def test_more_units_than_sms(T, kind):
    c = Case([T] * 3, 32, 64, "bf16", kind, seed=310)
    assert form(c) == (True, 1, 1)
    check_some(c, *prefill(c), sequences=(0, 2), heads=[0, 31, 32, 63])


@pytest.mark.parametrize("n", [200, 513, 700])
def test_many_packed_sequences(n):
    """Up to 512 run longest first, more in their order; empty and one-token ones among them."""
    r = random.Random(n)
    c = Case([r.choice((0, 1, 2, 3, 5, 9, 17, 64, 65, 100)) for _ in range(n)], 1, 1, "bf16", seed=320)
    assert form(c, packed=True)[0]
    c.check(*prefill(c, packed=True))


def test_segments_in_parts():
    """As many units as a third of the SMs: segments whose states come from three parts each."""
    c = Case([6000], 16, 48, "bf16", "head", seed=330)
    assert form(c) == (True, 3, 3)
    check_some(c, *prefill(c, in_place=True), sequences=(0,), heads=[0, 20, 47])


def test_packed_segments_in_parts():
    c = Case([4700, 300], 8, 24, "bf16", seed=331)
    assert form(c, packed=True) == (True, 3, 3)
    check_some(c, *prefill(c, packed=True), sequences=(0, 1), heads=[0, 11, 23])


def test_which_prompts_run_token_by_token():
    def chunked(*a, **kw):
        return gdn.gdn_selftest_linattn_form(*a, **kw).chunked
    assert not chunked(1, 64, 1, 2) and chunked(1, 200, 1, 2)
    assert not chunked(64, 24, 2, 8) and chunked(64, 64, 2, 8)
    assert not chunked(1, 4096, 1, 2, io_dtype=gdn.GDN_F32)
    assert chunked(8, 160, 1, 16, packed=True)  # one of the eight may have them all
    f = gdn.gdn_selftest_linattn_form(1, 2000, 1, 2, workspace=False)
    assert (f.chunked, f.segments, f.parts) == (1, 1, 1)
    assert gdn.gdn_selftest_linattn_form(1, 2000, 1, 2).segments > 1
