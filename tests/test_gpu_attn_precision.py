"""What gdn_attn promises of its weights in bf16 io: 11 bits of each weight with its page's value scale, down to 2^-25 of the
largest such product that the row has seen, and 2^-36 of it below; for tiles of rows the queries' bits.  The CPU tests
show that the bounds tell fewer bits, and a reference that is not the largest product, from these."""
import math

import pytest
import torch

import attn_precision as P
import attn_reference as R
from gated_deltanet_mixer_gb300 import gdn

BF = torch.bfloat16
FEW, TILE = 1, 2


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert gdn.gdn_device_status(reset=True) == 0


def run(cache, q, n, Hq, kernel, causal=True, scale=0.0, ws=True, parts=None):
    kv, D = cache.lens[0], cache.D
    f = gdn.gdn_selftest_attn_form(1, n, Hq, cache.Hk, D, max_new=n, max_kv=kv, workspace=ws)
    assert f.kernel == kernel and (parts is None or (f.parts > 1) == parts)
    w = None
    if ws:
        w = torch.full((max(256, gdn.gdn_attn_workspace_bytes(1, n, Hq, cache.Hk, D, max_new=n, max_kv=kv)),), 0xff, dtype=torch.uint8,
                       device="cuda")
    o = torch.full((n, Hq * D), math.nan, device="cuda", dtype=BF)
    gdn.gdn_attn(q, o, *cache.args(), Hq=Hq, cu_seqlens=torch.tensor([0, n], dtype=torch.int32, device="cuda"), causal=causal,
                 scale=scale, workspace=w, max_new=n, max_kv=kv)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    want, tol = P.attend(q.reshape(n, Hq, D), *P.parts(cache, 0, kv), n, causal, scale or D ** -0.5, kernel == TILE)
    err = (o.reshape(n, Hq, D).double() - want).abs()
    assert bool((err <= tol + 2.0 ** -133).all()), "off by %.3g of the tolerance" % float((err / (tol + 2.0 ** -133)).max())


FORMS = [(1, FEW), (3, FEW), (40, TILE), (150, TILE)]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kernel", FORMS)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("late", [True, False])
@pytest.mark.parametrize("lead,drop", [(30, 60), (36, 60), (40, 100), (110, 115), (20, 25), (3, 40)])
def test_large_values_that_hardly_count(lib, D, n, kernel, ws, late, lead, drop):
    """A page of value scale 1 with weights of 2^-drop, in front of or behind the page with the weight and scale 2^-lead."""
    if n == 40 and D == 64:
        n = 41
    c, q, scale = P.weights_against_scales(n, D, lead, drop, "cuda", late=late)
    run(c, q.repeat(1, 2), n, 8, kernel, scale=scale, ws=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("n,kernel", FORMS)
@pytest.mark.parametrize("lead,drop", [(36, 60), (20, 40)])
def test_large_values_that_hardly_count_in_parts(lib, n, kernel, lead, drop):
    c, q, scale = P.weights_against_scales(n, 128, lead, drop, "cuda", kv=6000)
    run(c, q.repeat(1, 2), n, 8, kernel, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("n,kernel", FORMS)
@pytest.mark.parametrize("least", [2.0 ** -120, 2.0 ** -110, 2.0 ** -101])
def test_the_least_value_scales(lib, n, kernel, least):
    c = R.Cache([n + 90], 2, 128, 16, device="cuda").fill()
    c.sv[c.table[0].long()] = least
    g = torch.Generator(device="cuda").manual_seed(1)
    run(c, torch.randn(n, 8 * 128, device="cuda", generator=g).to(BF), n, 8, kernel)


@pytest.mark.gpu
@pytest.mark.parametrize("n,kernel", FORMS)
@pytest.mark.parametrize("least", [2.0 ** -120, 2.0 ** -110, 2.0 ** -90, 1.0])
@pytest.mark.parametrize("drop", [12, 20])
def test_small_weights_alone_have_values(lib, n, kernel, least, drop):
    """The token with nearly all the weight has values of 0, and the scales are as small as they go: what is left is the
    others', of weight 2^-drop."""
    D = 128
    c = R.Cache([n + 50], 2, D, 16, device="cuda").fill(mean=0.0)
    t, g = c.table[0].long(), torch.Generator().manual_seed(drop)
    c.k8[t] = (0.125 * torch.randint(-1, 2, (t.numel(), 2, 16, D), generator=g)).to(torch.float8_e4m3fn).view(torch.uint8).to("cuda")
    c.k8[t[0], :, 0], c.v8[t[0], :, 0] = 0x38, 0
    c.sk[t], c.sv[t] = 1.0, least
    q = torch.ones(n, 8 * D, device="cuda").to(BF)
    run(c, q, n, 8, kernel, scale=drop * math.log(2.0) / D)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kernel", FORMS)
@pytest.mark.parametrize("kv", [5, 20, 300, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("spread", [0, 30, 100])
def test_weights(lib, D, n, kernel, kv, causal, spread):
    """Random keys, values and queries; value scales of pages up to 2^spread apart."""
    if n == 40 and D == 64:
        n = 41
    c = R.Cache([kv + n], 2, D, 16, device="cuda").fill(seed=kv + n)
    g = torch.Generator().manual_seed(spread)
    t = c.table[0].long()
    c.sv[t] = (2.0 ** -torch.randint(0, spread + 1, (t.numel(), 2), generator=g).float()).to("cuda")
    q = torch.randn(n, 8 * D, generator=g).to("cuda")
    run(c, q.to(BF), n, 8, kernel, causal=causal, scale=1.7 * D ** -0.5)


def few_tokens(n, D, device="cpu"):
    """Few tokens whose values cancel: what is left shows how the weights were rounded."""
    c = R.Cache([n + 3], 2, D, 16, device=device).fill(seed=5)
    p = c.table[0].long()
    sign = torch.where(torch.arange(16) % 2 == 0, 0x38, 0xb8).to(torch.uint8).to(device)  # 1, -1
    c.v8[p[0]] = sign[None, :, None]
    c.sv[p] = 1.0
    g = torch.Generator().manual_seed(9)
    return c, torch.randn(n, 8 * D, generator=g).to(BF).to(device)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kernel", [(1, FEW), (3, FEW), (60, TILE)])
def test_values_that_cancel(lib, D, n, kernel):
    c, q = few_tokens(n, D, "cuda")
    run(c, q, n, 8, kernel)


def ratio(got, want, tol):
    return float(((got - want).abs() / (tol + 2.0 ** -133)).max())


def fp16(p, s):
    """Through fp16, times 2^11 over the largest product."""
    w = p * s
    ref = w.amax(-1, keepdim=True)
    return (w / ref * 2.0 ** 11).half().double() * ref * 2.0 ** -11


def test_the_bound_tells_8_bits_from_11():
    n, D = 60, 64
    c, q = few_tokens(n, D)
    q, args = q.reshape(n, 8, D), P.parts(c, 0, n + 3)
    want, tol = P.attend(q, *args, n, True, D ** -0.5, False)
    tol = tol - 2.0 ** -8 * want.abs()  # no rounding of the output here
    assert ratio(P.rounded(q, *args, n, D ** -0.5, lambda p, s: p * s), want, tol) < 1e-3
    assert ratio(P.rounded(q, *args, n, D ** -0.5, fp16), want, tol) <= 1
    assert ratio(P.rounded(q, *args, n, D ** -0.5, lambda p, s: p.bfloat16().double() * s), want, tol + 2.0 ** -8 * want.abs()) > 1


@pytest.mark.parametrize("lead,drop", [(30, 60), (36, 60), (40, 100)])
def test_the_bound_tells_the_largest_product_from_the_largest_factors(lead, drop):
    c, q, scale = P.weights_against_scales(3, 64, lead, drop)
    q, args = q.reshape(3, 4, 64), P.parts(c, 0, 51)
    want, tol = P.attend(q, *args, 3, True, scale, True)
    assert ratio(P.rounded(q, *args, 3, scale, fp16), want, tol) <= 1
    apart = P.rounded(q, *args, 3, scale, lambda p, s: (p * s / s.amax(-1, keepdim=True) * 2.0 ** 11).half().double() *
                      s.amax(-1, keepdim=True) * 2.0 ** -11)
    assert ratio(apart, want, tol) > 1
