"""Block scales to and from page-locked host memory, as they go with swapped-out blocks."""

import pytest
import torch

from paged_kv_cache_418_b200 import ops

pytestmark = pytest.mark.gpu


def test_scales_to_page_locked_memory_and_back():
    g = torch.Generator().manual_seed(1)
    dev = [torch.rand(9, 5, generator=g).cuda() for _ in range(2)]
    host = [torch.zeros(20, 5).pin_memory() for _ in range(2)]
    back = [torch.zeros(9, 5, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.tensor([[3, 17], [8, 0], [0, 4]])
    # the pairs in device memory, then in page-locked host memory
    ops.pa_copy_scales(*host, *dev, out.cuda(), err)
    torch.cuda.synchronize()
    for h, d in zip(host, dev):
        assert torch.equal(h[out[:, 1]], d.cpu()[out[:, 0]]) and int((h != 0).any(dim=1).sum()) == 3
    ops.pa_copy_scales(*back, *host, out.flip(1).contiguous().pin_memory(), err)
    torch.cuda.synchronize()
    for b, d in zip(back, dev):
        assert torch.equal(b.cpu()[out[:, 0]], d.cpu()[out[:, 0]]) and int((b != 0).any(dim=1).sum()) == 3
    assert int(err.item()) == 0
    # a pair out of range is skipped and flagged
    ops.pa_copy_scales(*back, *host, torch.tensor([[20, 1], [0, 9], [4, 1]]).cuda(), err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.PA_DEV_BAD_PAIR
    assert torch.equal(back[0][1].cpu(), host[0][4])


def test_ordinary_host_memory_is_refused():
    dev = [torch.ones(4, 5, device="cuda") for _ in range(2)]
    host = [torch.zeros(4, 5) for _ in range(2)]
    pairs = torch.zeros(1, 2, dtype=torch.int64)
    for args in ((*host, *dev, pairs.cuda()), (*dev, *host, pairs.cuda()), (*dev, *dev, pairs), (*host, *host, pairs)):
        with pytest.raises(ops.PAError) as e:
            ops.pa_copy_scales(*args)
        assert e.value.status == 2
