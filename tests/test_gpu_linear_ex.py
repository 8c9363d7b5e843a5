"""GPU parity of gdn_linear_ex against the formulas in 64 bits.

Tolerance: the sum p is off by at most (K/16 + 8) 2^-23 sum |x w| (one
truncating sum per 16 products, the split's sums) plus the bias' fp32 sum;
that error enters y with the activation's slope (at most 1.13) and, gated, the
other factor; the fast exponential adds 2^-20 of the activation; the stored
rounding is half a step, 2^-8 |y|."""
import math

import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn
from linattn_reference import Guarded, act64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert torch.cuda.is_available()
    assert gdn.gdn_device_status(reset=True) == 0


def rand(*shape, ld=None, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if ld is None:
        return (scale * torch.randn(*shape, device="cuda", generator=g)).bfloat16()
    t = torch.full((shape[0], ld), 9.0, device="cuda", dtype=torch.bfloat16)
    t[:, :shape[1]] = rand(*shape, seed=seed, scale=scale)
    return t[:, :shape[1]]


def check(M, N, K, gated=False, bias=True, ranges=None, residual=False, in_place=False, pad=0, seed=0, odd=0):
    ld = -(-(K + pad) // 8) * 8
    x = rand(M, K, ld=ld, seed=seed)
    w = rand(N * (2 if gated else 1), K, ld=ld, seed=seed + 1, scale=1 / math.sqrt(K))
    bi = rand(w.shape[0], seed=seed + 2) if bias else None
    ranges = ranges or [(0, N, "silu" if gated else "none")]
    outs, guards = [], []
    for i, (b, e, act) in enumerate(ranges):
        g = Guarded((M, e - b), torch.bfloat16, ld=e - b + odd)
        res = rand(M, e - b, ld=e - b + odd, seed=seed + 3 + i) if residual else None
        first = res.clone() if residual else None
        if in_place:
            g.t.copy_(res)
            res = g.t
        outs.append((b, e, g.t, act, res))
        guards.append((g, first))
    gdn.gdn_linear_ex(x, w, outs, bias=bi, gated=gated)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    p = x.double() @ w.double().T
    A = x.double().abs() @ w.double().abs().T
    if bias:
        p, A = p + bi.double(), A + bi.double().abs()
    dp = (K / 16 + 8) * 2.0 ** -23 * A
    for (b, e, _, act, _), (g, first) in zip(outs, guards):
        y = act64(p[:, b:e], act)
        d = 1.13 * dp[:, b:e] + 2.0 ** -20 * y.abs()
        if gated:
            u, du = p[:, N + b:N + e], dp[:, N + b:N + e]
            d = d * (u.abs() + du) + y.abs() * du
            y = y * u
        if residual:
            y = y + first.double()
        d = d + 2.0 ** -23 * y.abs()
        d = d + 2.0 ** -8 * (y.abs() + d)
        err = (g.t.double() - y).abs()
        assert bool((err <= d + 1e-30).all()), "%.3g of the bound" % (err / (d + 1e-30)).max()
        assert g.intact()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("N,K", [(8, 8), (130, 72), (520, 1000), (2048, 2048)])
def test_plain(M, N, K):
    check(M, N, K, seed=M)


@pytest.mark.parametrize("M,N,K", [(1, 16480, 512), (2560, 2050, 200), (1300, 4104, 136)])
def test_whole_waves_and_wide_rows(M, N, K):
    check(M, N, K, bias=False, seed=5, pad=16)
    check(M, N, K, residual=True, seed=6)


@pytest.mark.parametrize("M", [1, 40, 200])
def test_ranges_and_activations(M):
    check(M, 700, 264, ranges=[(0, 96, "silu"), (96, 333, "gelu"), (333, 517, "sigmoid"), (520, 700, "none")], seed=M, odd=5)
    check(M, 700, 264, ranges=[(0, 96, "gelu"), (128, 256, "silu")], residual=True, seed=M + 1)


def test_ranges_on_the_tile_kernel():
    check(2600, 4000, 128, ranges=[(0, 1024, "silu"), (1024, 1111, "gelu"), (1111, 2048, "none"), (2048, 4000, "sigmoid")],
          residual=True, seed=8)


@pytest.mark.parametrize("M", [1, 20, 100])
@pytest.mark.parametrize("N", [1, 63, 64, 200, 1001])
def test_gated(M, N):
    check(M, N, 320, gated=True, seed=N, residual=M > 1)


def test_gated_tile_kernel():
    check(2600, 1111, 200, gated=True, seed=9)
    check(1300, 2048, 136, gated=True, seed=10, ranges=[(0, 1000, "gelu"), (1000, 2048, "none")], bias=False, residual=True)


@pytest.mark.parametrize("M,N", [(3, 512), (2600, 2048)])
def test_residual_in_place_and_odd_strides(M, N):
    check(M, N, 192, residual=True, in_place=True, seed=11)
    check(M, N, 192, residual=True, in_place=True, seed=12, odd=3)


def test_extreme_sums():
    """Activations far out: silu and sigmoid saturate, nothing turns NaN."""
    x = torch.full((2, 8), 30.0, device="cuda", dtype=torch.bfloat16)
    x[1] = -30.0
    w = torch.ones(16, 8, device="cuda", dtype=torch.bfloat16)
    y = [torch.empty(2, 4, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    gdn.gdn_linear_ex(x, w, [(4 * i, 4 * i + 4, y[i], a) for i, a in enumerate(("none", "silu", "gelu", "sigmoid"))])
    torch.cuda.synchronize()
    for i, (hi, lo) in enumerate(((240.0, -240.0), (240.0, 0.0), (240.0, 0.0), (1.0, 0.0))):
        assert bool((y[i][0] == hi).all()) and bool(((y[i][1] - lo).abs() < 1e-30).all())


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph():
    x, w = rand(5, 1024, seed=1), rand(512, 1024, seed=2)
    y = [torch.empty(5, 512, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    gdn.gdn_linear_ex(x, w, [(0, 512, y[0], "gelu")])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_linear_ex(x, w, [(0, 512, y[1], "gelu")], stream=s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_linear_ex(x, w, [(0, 512, y[2], "gelu")])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 320), (2049, 5000, 1000), (8192, 2056, 64)])
def test_pairs_of_ctas(M, N, K):
    check(M, N, K, seed=20, residual=True)
    check(M, N, K, gated=True, seed=21, bias=K != 64)


@pytest.mark.parametrize("M", [3, 30, 64])
def test_few_tokens_in_several_waves_of_smaller_tiles(M):
    check(M, 24600, 1024, seed=M, pad=8)
    check(M, 24599, 1000, seed=M + 1, odd=3, residual=True,
          ranges=[(0, 8200, "silu"), (8200, 16001, "none"), (16001, 24599, "sigmoid")])
    check(M, 12300, 1024, gated=True, seed=M + 2, residual=M > 3)
    check(M, 12299, 1000, gated=True, seed=M + 3, bias=False, odd=1)


@pytest.mark.parametrize("M,N,K", [(219, 421, 1640), (526, 62, 1136), (130, 129, 2048), (1100, 40, 520)])
def test_few_columns_in_several_tiles_of_tokens(M, N, K):
    check(M, N, K, seed=M, residual=True, odd=1)
    check(M, N, K, seed=M + 1, gated=True, ranges=[(0, 33, "silu"), (33, N, "sigmoid")])
