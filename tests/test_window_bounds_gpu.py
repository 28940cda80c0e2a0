"""The smallest and largest bounds that the windowed and block-scaled calls take."""

import pytest
import torch

from paged_kv_cache_418_b200 import ops
from range_testlib import Cache

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


@pytest.mark.parametrize("blk8", [False, True])
def test_a_loose_bound_of_the_new_tokens(blk8):
    """max_query_len bounds the new tokens of a sequence; a bound far past them changes nothing and costs
    nothing (chunks past a call's last token are not walked)."""
    g = torch.Generator().manual_seed(2)
    seqs = [(torch.randn(n, 2, 128, generator=g), torch.randn(n, 2, 128, generator=g)) for n in (300, 70)]
    t = "fp8" if blk8 else "bf16"
    c = Cache(seqs, 16, t, t, [torch.zeros(-(-n // 16), 2) for n in (300, 70)] if blk8 else None)
    q = torch.randn(110, 8, 128, generator=g).bfloat16().cuda()
    qs = torch.tensor([0, 100, 110], dtype=torch.int32, device="cuda")

    def run(bound):
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        if blk8:
            ops.pa_prefill_blk8(out, q, c.k, c.v, c.ks, c.vsc, c.bt, c.cl, qs, bound, 0.09, 300, 0, 0)
        else:
            ops.pa_prefill_window_kv(out, q, c.k, c.v, 1.0, 1.0, c.bt, c.cl, qs, bound, 0.09, 200, 4, 300)
        b.record()
        torch.cuda.synchronize()
        return out, a.elapsed_time(b)

    run(100)
    exact, _ = run(100)
    for bound in (110, 2 ** 20, 2 ** 31 - 1):
        out, ms = run(bound)
        assert torch.equal(out, exact) and ms < 5, (bound, ms)
