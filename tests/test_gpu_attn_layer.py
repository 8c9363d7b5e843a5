"""The attention layer on the library's operators: run as a program (prompts, then single tokens from a captured graph,
against one prompt), and a padded step whose last rows belong to no request."""
import sys

import pytest
import torch

from gated_deltanet_mixer_gb300 import attn_layer, gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_mixer_gb300 import build
    build.build()
    gdn.lib()
    assert gdn.gdn_device_status(reset=True) == 0


@pytest.mark.parametrize("args", ["--hidden 512 --ffn 1024 --Hq 6 --Hk 1 --D 256 --rot 64 --T 150 --new 3",
                                  "--hidden 1024 --ffn 512 --Hq 8 --Hk 8 --D 64 --rot 64 --B 5 --T 37 --new 20",
                                  "--hidden 512 --ffn 1024 --Hq 16 --Hk 2 --D 128 --rot 32 --B 1 --T 700 --new 2"])
def test_runs_as_a_program(args, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["attn_layer"] + args.split())
    attn_layer.main()
    assert "outputs differ" in capsys.readouterr().out


def test_a_padded_step_and_one_that_does_not_fit():
    """Buffers for 8 tokens, 5 given: the requests' rows as without padding, the cache as well; then pages run out, and
    nothing moves."""
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.randn(8, 256, device="cuda").bfloat16()
    outs, layers = [], []
    for rows in (5, 8):
        layer = attn_layer.AttnLayer(256, 256, 4, 2, 64, 64, attn_layer.PagedCache(2, 2, 64, 3, max_blocks=2))
        y = x[:rows].clone()
        layer.forward(y, torch.tensor([4, 1], **i32), layer.step(rows, 4))
        torch.cuda.synchronize()
        assert gdn.gdn_device_status() == 0
        outs.append(y)
        layers.append(layer)
    assert torch.equal(outs[0], outs[1][:5])
    a, b = (l.cache for l in layers)
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.kv_lens, b.kv_lens) and int(b.used) == 2
    layer, before = layers[1], [t.clone() for t in (b.kv_lens, b.table, b.used, b.sk)]
    y = torch.randn(40, 256, device="cuda").bfloat16()
    layer.forward(y, torch.tensor([20, 20], **i32), layer.step(40, 20))
    torch.cuda.synchronize()
    assert gdn.gdn_device_status(reset=True) == gdn.GDN_ERR_INVALID_ARG
    assert all(torch.equal(u, v) for u, v in zip(before, (b.kv_lens, b.table, b.used, b.sk)))
