"""Every kernel of gdn_linear_ex against the formulas in 64 bits, on ragged sizes.

The choice among them is a cost model, so each test first asks which kernel the
call takes: when the model moves, the test fails instead of quietly running
something else.  Tolerances as in test_gpu_linear_ex.py."""
import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn
from test_gpu_linear_ex import check, rand

pytestmark = pytest.mark.gpu

PAIR, TILE, FEW = range(3)

# Few tokens or columns: (tokens of a tile, tiles of fewer than 128 rows of w, a cluster of several CTAs), gated, M, N, K
FEW_CASES = [
    ((16, False, False), False, 1, 9, 3),
    ((16, False, True), False, 1, 9, 194),
    ((16, True, False), False, 2033, 11, 217),
    ((16, True, True), False, 1141, 13, 260),
    ((32, False, False), False, 1228, 129, 3),
    ((32, False, True), False, 751, 9, 586),
    ((32, True, False), False, 17, 8115, 194),
    ((32, True, True), False, 1013, 9, 718),
    ((64, False, False), False, 33, 7687, 3),
    ((64, False, True), False, 34, 1987, 667),
    ((64, True, False), False, 33, 6907, 195),
    ((64, True, True), False, 1548, 9, 1298),
    ((128, False, False), False, 65, 6913, 3),
    ((128, False, True), False, 65, 1783, 1478),
    ((256, False, True), False, 132, 2427, 2633),
    ((16, False, False), True, 1, 9, 3),
    ((16, False, True), True, 1, 9, 194),
    ((16, True, False), True, 2021, 9, 194),
    ((16, True, True), True, 446, 9, 764),
    ((32, False, False), True, 17, 4871, 3),
    ((32, False, True), True, 1266, 9, 323),
    ((32, True, True), True, 651, 9, 1089),
    ((64, False, False), True, 33, 4917, 4),
    ((64, False, True), True, 34, 1685, 327),
    ((64, True, True), True, 1483, 9, 1266),
    ((128, False, True), True, 71, 3259, 195),
    ((256, False, True), True, 135, 1387, 1773),
]
# One CTA's tiles: (their columns, more of them than SMs), gated, M, N, K
TILE_CASES = [
    ((64, False), False, 2181, 11, 132),
    ((64, True), False, 200, 5015, 137),
    ((128, False), False, 134, 5499, 771),
    ((128, True), False, 391, 7651, 580),
    ((256, False), False, 1551, 2619, 2454),
    ((256, True), False, 1815, 4885, 1286),
    ((64, False), True, 2203, 11, 135),
    ((64, True), True, 137, 5035, 130),
    ((128, False), True, 282, 4903, 1191),
    ((128, True), True, 594, 7075, 622),
]
# Pairs of CTAs: (more tiles than pairs), gated, M, N, K
PAIR_CASES = [
    ((False,), False, 296, 6837, 1730),
    ((True,), False, 920, 7861, 965),
    ((False,), True, 139, 4965, 875),
    ((True,), True, 667, 5011, 466),
]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert gdn.gdn_device_status(reset=True) == 0


def form(M, N, K, gated, residual):
    f = gdn.gdn_selftest_linear_ex_form(M, N, K, gated, residual)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if f.kernel == FEW:
        return FEW, (f.tile, f.rows_w < 128, f.split > 1)
    return f.kernel, (f.tile, f.tiles > sms) if f.kernel == TILE else (f.tiles > sms // 2,)


def ranges(N):
    """Four ranges with an activation each, the first two on whole 16-byte rows where N is large, and
    columns that none of them covers."""
    a, b, c = (N * i // 4 for i in (1, 2, 3))
    if N > 64:
        a, b = a // 8 * 8, b // 8 * 8
    return [(0, a, "silu"), (a, b, "none"), (b, c, "gelu"), (c + 1, N, "sigmoid")]


@pytest.mark.parametrize("kernel,want,gated,M,N,K",
                         [(k, *c) for k, cases in ((FEW, FEW_CASES), (TILE, TILE_CASES), (PAIR, PAIR_CASES)) for c in cases])
def test_every_form(kernel, want, gated, M, N, K):
    for residual in (False, True):
        assert form(M, N, K, gated, residual) == (kernel, want)
    check(M, N, K, gated=gated, seed=1, pad=8)
    check(M, N, K, gated=gated, seed=2, ranges=ranges(N))
    check(M, N, K, gated=gated, seed=3, ranges=ranges(N), residual=True, odd=3, bias=False)
    check(M, N, K, gated=gated, seed=4, residual=True, in_place=True, odd=1)


@pytest.mark.parametrize("kernel,want,gated,M,N,K", [(FEW, *FEW_CASES[4]), (TILE, *TILE_CASES[3]), (PAIR, *PAIR_CASES[1]),
                                                     (PAIR, *PAIR_CASES[3])])
def test_a_form_repeats_itself_bit_for_bit(kernel, want, gated, M, N, K):
    assert form(M, N, K, gated, False) == (kernel, want)
    ld = -(-K // 8) * 8
    x, w = rand(M, K, ld=ld, seed=1), rand(N * (2 if gated else 1), K, ld=ld, seed=2, scale=K ** -0.5)
    y = [torch.empty(M, N, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    for t in y:
        gdn.gdn_linear_ex(x, w, [(0, N, t, "silu")], gated=gated)
    torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_every_kernel_is_in_the_list():
    """As many forms as the library instantiates."""
    assert {(c[0][0], c[1]) for c in FEW_CASES} == {(n, g) for n in (16, 32, 64, 128, 256) for g in (False, True)}
    assert {(c[0][0], c[1]) for c in TILE_CASES} == {(64, False), (128, False), (256, False), (64, True), (128, True)}
    assert {c[1] for c in PAIR_CASES} == {False, True}
