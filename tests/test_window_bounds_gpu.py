"""The smallest and largest bounds that the windowed and block-scaled calls take."""

import pytest
import torch

from paged_kv_cache_418_b200 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16", "blk8"])
def test_a_batch_of_empty_sequences_with_its_true_bound(kind):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "blk8": torch.uint8}[kind]
    c = torch.zeros(2, 16, 2, 64, dtype=dt, device="cuda")
    s = torch.ones(2, 2, device="cuda")
    q = torch.randn(5, 8, 64, device="cuda").to(torch.float32 if kind == "f32" else torch.bfloat16)
    out = torch.full(q.shape, float("nan"), device="cuda")
    bt = torch.full((5, 1), -1, dtype=torch.int32, device="cuda")
    cl = torch.zeros(5, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = ops.window_workspace_for(q, c, 0, 3, 1)
    if kind == "blk8":
        ops.pa_decode_blk8(out, q, c, c, s, s, bt, cl, 0.1, 0, 3, 1, ws, err)
    else:
        ops.pa_decode_window_kv(out, q, c, c, 1.0, 1.0, bt, cl, 0.1, 3, 1, 0, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, torch.zeros_like(out))
