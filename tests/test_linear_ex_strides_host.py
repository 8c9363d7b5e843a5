"""Output and residual strides of gdn_linear_ex that no buffer can have are
refused on the host: their extents would wrap around and pass the checks."""
import pytest

from gated_deltanet_mixer_gb300 import build as gdn_build
from gated_deltanet_mixer_gb300 import gdn
from test_linattn_host import OK_ON_HOST, fake, linear


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


@pytest.mark.parametrize("ld", [(1 << 32) + 8, 1 << 61, 1 << 62])
def test_strides_beyond_any_buffer(L, ld):
    assert linear(L, outs=[(0, 8, fake(2), ld, 0, None, 0)]) == 2
    assert linear(L, outs=[(0, 8, fake(2), 8, 0, fake(3), ld)]) == 2
    assert linear(L, M=1, outs=[(0, 8, fake(2), 8, 0, None, ld)]) in OK_ON_HOST  # no residual: its stride is not looked at
    assert linear(L, M=1, outs=[(0, 8, fake(2), 1 << 32, 0, None, 0)]) in OK_ON_HOST
