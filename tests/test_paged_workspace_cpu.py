"""Workspaces of caches that weigh pages, on a machine without a GPU."""
import pytest
import torch

from bwd_tile_mean_gb300 import vsa

BF = torch.bfloat16


def sizes():
    c = vsa.PagedCache("bshd", BF, 2, 4, 2, 128, 16, 4, 3, device="cpu", weigh=True)
    L, d = vsa.lib(), vsa.C.byref(c.desc)
    return int(L.vsa_paged_workspace_size(d)), int(L.vsa_paged_weigh_workspace_size(d))


@pytest.mark.parametrize("what", ["page_table", "seq_lens", "k_mean"])
def test_the_weights_part_of_the_workspace_is_the_calls_own(what):
    """A workspace as large as page weights need, whose last part is also a
    tensor of the cache: the plain calls leave that part alone, the weighing
    one would write it."""
    plain, large = sizes()
    buf = torch.zeros(large + 16384, dtype=torch.uint8)
    at = -buf.data_ptr() % 256
    tail = buf[at + plain:]
    kinds = dict(page_table=((2, 3), torch.int32), seq_lens=((2,), torch.int32), k_mean=((4, 2, 128), torch.float32))
    shape, kind = kinds[what]
    n = torch.Size(shape).numel() * 4
    given = {what: tail[:n].view(kind).view(shape)}
    c = vsa.PagedCache("bshd", BF, 2, 4, 2, 128, 16, 4, 3, device="cpu", workspace=buf[at:], **given)
    q, w = torch.zeros(2, 4, 128, dtype=BF), torch.zeros(2, 2, 3)
    with pytest.raises(ValueError, match="workspace.*shares memory|shares memory.*workspace"):
        c.attend(q, page_weight=w)
    with pytest.raises(ValueError, match="GPU only"):
        c.attend(q)
