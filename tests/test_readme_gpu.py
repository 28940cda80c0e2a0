"""The README's Python examples run as they stand, on batches of several sequences."""

import os
import re

import pytest
import torch

from paged_kv_cache_418_b200 import ops

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _blocks():
    with open(README) as f:
        return re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)


def _step(T, Hq, Hkv, D, bs, dtype):
    """A decode step of T sequences whose earlier tokens fill two blocks less one slot."""
    g = torch.Generator().manual_seed(1)
    nb = 2 * T + 1
    tables = torch.randperm(nb, generator=g)[:2 * T].view(T, 2)
    dev = "cuda"
    return dict(T=T, Hq=Hq, Hkv=Hkv, D=D, max_context_len=2 * bs, nb=nb, bs=bs, block_tables=tables.int().to(dev),
                context_lens=torch.full((T,), 2 * bs, dtype=torch.int32, device=dev),
                slot_mapping=(tables[:, 1] * bs + bs - 1).to(dev), dtype=dtype,
                err=torch.zeros(1, dtype=torch.int32, device=dev))


def test_the_plain_example():
    s = _step(6, 8, 2, 128, 16, torch.bfloat16)
    shape = (s["nb"], s["bs"], s["Hkv"], s["D"])
    new = lambda *x: torch.randn(*x, device="cuda").to(s["dtype"])
    s.update(k_cache=new(*shape), v_cache=new(*shape), q=new(s["T"], s["Hq"], s["D"]),
             new_k=new(s["T"], s["Hkv"], s["D"]), new_v=new(s["T"], s["Hkv"], s["D"]))
    exec([b for b in _blocks() if "pa_decode(" in b][0], s)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(s["out"]).all())


def test_the_block_scaled_example():
    """Rows of a fused projection into the cache and the attention over them, against dense attention."""
    s = _step(6, 8, 2, 128, 16, torch.bfloat16)
    T, Hq, Hkv, D, bs = (s[x] for x in ("T", "Hq", "Hkv", "D", "bs"))
    s.update(window=20, sinks=3, positions=torch.full((T,), 2 * bs - 1, dtype=torch.int64, device="cuda"),
             qkv=torch.randn(T, Hq + 2 * Hkv, D, device="cuda").to(s["dtype"]),
             cos_sin=torch.cat([torch.ones(2 * bs, D // 2), torch.zeros(2 * bs, D // 2)], 1).cuda(),     # (no turn)
             k_cache=torch.zeros(s["nb"], bs, Hkv, D, dtype=torch.uint8, device="cuda"))
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    s["k_scales"], s["v_scales"] = (torch.ones(s["nb"], Hkv, device="cuda") for _ in range(2))
    old = torch.randn(2, T * (2 * bs - 1), Hkv, D, device="cuda").to(s["dtype"])
    slots = (s["block_tables"].long()[:, :, None] * bs + torch.arange(bs, device="cuda")).view(T, -1)[:, :-1].reshape(-1)
    ops.pa_rope_and_cache_blk8(None, None, old[0], old[1], None, None, s["k_cache"], s["v_cache"], s["k_scales"],
                               s["v_scales"], slots.contiguous())
    s.update(torch=torch, ops=ops)                 # (of the example above it)
    exec([b for b in _blocks() if "pa_decode_blk8" in b][0], s)
    torch.cuda.synchronize()
    assert int(s["err"].item()) == 0
    assert torch.equal(s["q_rot"], s["qkv"][:, :Hq])
    from range_testlib import E4M3, attend, check, sees
    k, v = ((c.view(E4M3).float() * sc[:, None, :, None])[s["block_tables"].long()].reshape(T, 2 * bs, Hkv, D).cpu().double()
            for c, sc in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])))
    for b in range(T):
        ref, tol = attend(s["q_rot"][b].cpu().double(), k[b], v[b], sees(2 * bs, 2 * bs - 1, 20, 3), D ** -0.5, 2.0 ** -20, 2.0 ** -43)
        check(s["out"][b], ref, tol, f"sequence {b}")
