"""Rotary positions in fp32 held to what the angle's 32 bits leave: the reference turns by the plan's own integers, at near
and far positions alike, and the bound goes with each pair."""
import math

import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn

BF, F32 = torch.bfloat16, torch.float32


def turned(x, pos, plan, D, inverse=False, bits=None):
    """(y, bound) of x [tokens, heads * D] in 64 bits.  The angle is p * turns modulo 2^64, of a turn; beyond the nearest
    quarter, at most 2^-3 of a turn, as fp32 it is off by 2^-28: pi 2^-27.  Its sine and cosine are off by 2 steps of 2^-24,
    m times them by half a step; two products and a sum round by half a step of the pair's size h at most, each: with
    |a| + |b| <= sqrt(2) h,
        (pi / 8 + 2 sqrt(2) + sqrt(2) / 2 + 1) 2^-24 m h < 5 2^-24 m h,  6 with the higher orders,
    and one rounding to the type.  bits: an angle of so many bits instead, for the bound's own test."""
    n = plan.rot // 2
    f = torch.tensor([plan.turns[i] - (1 << 64 if plan.turns[i] >> 63 else 0) for i in range(n)], dtype=torch.int64, device=x.device)
    angle = pos.long()[:, None] * f  # wraps
    if bits:
        angle = (angle >> (64 - bits)) << (64 - bits)
    a = angle.double() * 2.0 ** -64 * 2 * math.pi
    c, s = (plan.m * torch.cos(a))[:, None], ((-1 if inverse else 1) * plan.m * torch.sin(a))[:, None]
    y = x.double().unflatten(-1, (-1, D)).clone()
    ia = torch.arange(n) if plan.layout == 0 else torch.arange(0, 2 * n, 2)
    ib = ia + (n if plan.layout == 0 else 1)
    u, w = y[..., ia], y[..., ib]
    h = 6 * 2.0 ** -24 * plan.m * torch.hypot(u, w)
    y[..., ia], y[..., ib] = u * c - w * s, w * c + u * s
    bound = torch.zeros_like(y)
    bound[..., ia], bound[..., ib] = h, h
    half = {BF: 2.0 ** -8, F32: 0.0}[x.dtype]
    return y.flatten(-2), (bound + half * y.abs()).flatten(-2)


def problem(dt, far, device="cpu", D=128, tokens=257):
    g = torch.Generator().manual_seed(far % 1000)
    pos = torch.randint(-far, far, (tokens,), generator=g).to(torch.int32)
    return torch.randn(tokens, 3 * D, generator=g).to(dt).to(device), pos.to(device)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 64, 6])
@pytest.mark.parametrize("far", [300, 1 << 17, (1 << 31) - 1])
@pytest.mark.parametrize("scaling", [None, dict(kind="parts", factor=16.0, original=4096)])
@pytest.mark.parametrize("inverse", [False, True])
def test_angles(dt, layout, rot, far, scaling, inverse):
    from gated_deltanet_mixer_gb300 import build
    build.build()
    plan = gdn.gdn_rope_plan(rot, layout=layout, scaling=scaling)
    x, pos = problem(dt, far, "cuda")
    want, bound = turned(x, pos, plan, 128, inverse)
    y = torch.empty_like(x)
    gdn.gdn_rope(plan, pos, [(x, y)], D=128, inverse=inverse)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    err = (y.double() - want).abs()
    assert bool((err <= bound).all()), "off by %.3g of the bound" % float((err / bound.clamp(min=1e-30)).max())


def test_the_bound_tells_an_angle_of_fewer_bits():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    for layout in ("half", "interleaved"):
        plan = gdn.gdn_rope_plan(64, layout=layout)
        for far in (300, (1 << 31) - 1):
            x, pos = problem(F32, far)
            want, bound = turned(x, pos, plan, 128)
            for bits, good in ((32, True), (22, False)):
                got, _ = turned(x, pos, plan, 128, bits=bits)
                assert bool(((got - want).abs() <= bound).all()) == good, (layout, far, bits)
