"""gdn_kv_pages on both sides of the sizes where it takes other numbers of threads and CTAs."""
import pytest
import torch

from gated_deltanet_mixer_gb300 import gdn
from test_gpu_attn_cache import _lib, ok, pages_by_hand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,room", [(256, 256), (257, 256), (256, 257), (4096, 20480), (4097, 20480), (4096, 20481), (1, 256), (1, 257),
                                    (1, 20481), (1, 70000)])
def test_borders(B, room):
    g = torch.Generator().manual_seed(B + room)
    page = 16
    kv = torch.randint(0, 50, (B,), generator=g)
    new = torch.zeros(B, dtype=torch.long)
    new[torch.randperm(B, generator=g)[:room]] = 1
    new[0] += room - int(new.sum()) - (3 if room > B else 0)  # a few slots stay free
    new.clamp_(min=0)
    width = int(((kv + new + page - 1) // page).max())
    table = torch.full((B, width), -7, dtype=torch.int32)
    for b in range(B):
        table[b, :-(-int(kv[b]) // page)] = b
    free = torch.randperm(B + room, generator=g).to(torch.int32)
    want = pages_by_hand(kv.tolist(), new.tolist(), free.tolist(), 0, table, page)
    d = [t.to(torch.int32).cuda() for t in (kv, new, free)]
    used, tab = torch.zeros(1, dtype=torch.int32, device="cuda"), table.cuda()
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.full((room,), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((room,), 77, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_pages(d[0], d[1], d[2], used, tab, d[0], used, cu, slots, pos, page=page)
    ok()
    total, spare = want[3][-1], room - want[3][-1]
    assert 0 <= spare <= room and total > 0
    assert torch.equal(tab.cpu(), want[0]) and cu.tolist() == want[3] and int(used) == want[4]
    assert slots.tolist() == want[1] + [-1] * spare and pos.tolist() == want[2] + [0] * spare
    assert d[0].tolist() == (kv + new).tolist()
