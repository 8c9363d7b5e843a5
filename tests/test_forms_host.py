"""Host-side checks of the entry points that say which kernel a call takes."""
import ctypes

import pytest

from gated_deltanet_mixer_gb300 import build as gdn_build
from gated_deltanet_mixer_gb300 import gdn

OK_ON_HOST = (5, 7)  # every check passed; then no device (or not this one)


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


def test_linear_ex_form_arguments(L):
    f = gdn.gdn_linear_ex_form()
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, 0)):
        assert L.gdn_selftest_linear_ex_form(*bad, 0, 0, ctypes.byref(f)) == 1
    assert L.gdn_selftest_linear_ex_form(8, 8, 8, 0, 0, None) == 1
    assert L.gdn_selftest_linear_ex_form(1 << 30, 1 << 28, 8, 0, 0, ctypes.byref(f)) == 2
    assert L.gdn_selftest_linear_ex_form(8, 8, 8, 0, 0, ctypes.byref(f)) in OK_ON_HOST


def test_linattn_form_arguments(L):
    f = gdn.gdn_linattn_form()
    sh = gdn.make_shape(2, 100, 2, 4, 128, gdn.GDN_BF16)
    assert L.gdn_selftest_linattn_form(None, 0, 0, ctypes.byref(f)) == 1
    assert L.gdn_selftest_linattn_form(ctypes.byref(sh), 0, 0, None) == 1
    assert L.gdn_selftest_linattn_form(ctypes.byref(gdn.make_shape(2, 0, 2, 4, 128, gdn.GDN_BF16)), 0, 0, ctypes.byref(f)) == 1
    assert L.gdn_selftest_linattn_form(ctypes.byref(gdn.make_shape(2, 9, 3, 4, 128, gdn.GDN_BF16)), 0, 0, ctypes.byref(f)) == 2
    assert L.gdn_selftest_linattn_form(ctypes.byref(sh), 1, 1, ctypes.byref(f)) in OK_ON_HOST
