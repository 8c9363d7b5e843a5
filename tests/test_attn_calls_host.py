"""Calls of gdn_attn that its documentation allows, checked without a GPU (addresses are never dereferenced)."""
import pytest

from test_attn_cache_host import L, OK_ON_HOST, attn, fake  # noqa: F401

ALIAS = 4  # gdn_status
W = 8 * 128 * 2  # bytes of a row of q or o


@pytest.mark.parametrize("cu", [None, fake(6)])
def test_o_beside_q_in_one_buffer(L, cu):  # noqa: F811
    """Disjoint column blocks of one buffer, either in front; not where they touch, or the strides differ."""
    kw = dict(ldq=4096, ldo=4096, cu_seqlens=cu)
    for q, o in ((0, W), (W, 0), (0, 4 * W - W), (0, 5 * W), (256, W + 256)):
        assert attn(L, q=fake(8, q), o=fake(8, o), **kw) in OK_ON_HOST, (q, o)
    for q, o in ((0, 0), (0, 512), (0, W - 16), (W, 16), (0, 4 * W - 16), (0, 4 * W)):
        assert attn(L, q=fake(8, q), o=fake(8, o), **kw) == ALIAS, (q, o)
    assert attn(L, q=fake(8), o=fake(8, W), ldq=4096, ldo=4104, cu_seqlens=cu) == ALIAS
    assert attn(L, q=fake(8), o=fake(8, W), workspace=fake(8, 2 * W), workspace_bytes=256, **kw) == ALIAS
