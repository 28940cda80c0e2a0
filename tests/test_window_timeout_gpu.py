"""The pipeline waits of the windowed and block-scaled kernels are bounded: with a CTA's first load left
out and a limit of 1 ms the launch reports PA_DEV_TIMEOUT and returns, and the next one is right."""

import pytest
import torch

from paged_kv_cache_418_b200 import ops
from range_testlib import Cache, attend, check, decode, prefill, sees

pytestmark = pytest.mark.gpu


def _values(seed, lens, rows, Hq, Hkv, qt):
    g = torch.Generator().manual_seed(seed)
    seqs = [(torch.randn(n, Hkv, 128, generator=g), torch.randn(n, Hkv, 128, generator=g)) for n in lens]
    return torch.randn(rows, Hq, 128, generator=g).to({"f16": torch.float16, "bf16": torch.bfloat16}[qt]), seqs


@pytest.mark.parametrize("kind,Hq,Hkv", [("bf16", 16, 8), ("f16", 4, 1), ("blk8", 8, 8), ("blk8", 6, 3)])
def test_decode_wait_limit_runs_out_and_the_next_launch_is_correct(monkeypatch, kind, Hq, Hkv):
    lens, qt = [900, 17, 2500], "f16" if kind == "f16" else "bf16"
    q, seqs = _values(5, lens, 3, Hq, Hkv, qt)
    c = Cache(seqs, 16, *(["fp8"] * 2 if kind == "blk8" else [qt] * 2),
              [torch.zeros(-(-n // 16), Hkv) for n in lens] if kind == "blk8" else None)
    window, sinks = (0, 0) if kind == "blk8" else (700, 4)
    out = torch.empty(q.shape, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = q.cuda()
    ws = ops.window_workspace_for(qd, c.k, max(lens), window, sinks)
    monkeypatch.setenv("PA_TC_WAIT_NS", "1000000")
    monkeypatch.setenv("PA_TC_TEST_WITHHOLD_Q", "1")
    if kind == "blk8":
        ops.pa_decode_blk8(out, qd, c.k, c.v, c.ks, c.vsc, c.bt, c.cl, 0.09, max(lens), 0, 0, ws, err)
    else:
        ops.pa_decode_window_kv(out, qd, c.k, c.v, 1.0, 1.0, c.bt, c.cl, 0.09, window, sinks, max(lens), ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.PA_DEV_TIMEOUT, "no wait ran out"
    monkeypatch.delenv("PA_TC_WAIT_NS")
    monkeypatch.delenv("PA_TC_TEST_WITHHOLD_Q")
    out = decode(c, q, 0.09, window, sinks)
    for b, n in enumerate(lens):
        ref, tol = attend(q[b].double(), c.k64[b], c.v64[b], sees(n, n - 1, window, sinks), 0.09, 2.0 ** -16, 0.0)
        check(out[b], ref, tol, f"sequence {b}")


@pytest.mark.parametrize("kind,Hq,Hkv", [("bf16", 8, 1), ("f16", 4, 2), ("blk8", 8, 1), ("mixed", 4, 4)])
def test_prefill_wait_limit_runs_out_and_the_next_launch_is_correct(monkeypatch, kind, Hq, Hkv):
    """Units of one query tile and of two, with converters and without."""
    lens, new, qt = [900, 40, 1500], [100, 3, 20], "f16" if kind == "f16" else "bf16"
    q, seqs = _values(6, lens, sum(new), Hq, Hkv, qt)
    kt, vt = {"blk8": ("fp8", "fp8"), "mixed": ("fp8", "bf16")}.get(kind, (qt, qt))
    c = Cache(seqs, 16, kt, vt, [torch.zeros(-(-n // 16), Hkv) for n in lens] if kind == "blk8" else None)
    window, sinks = (0, 0) if kind == "blk8" else (700, 4)
    out = torch.empty(q.shape, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 100, 103, 123], dtype=torch.int32, device="cuda")
    monkeypatch.setenv("PA_TC_WAIT_NS", "1000000")
    monkeypatch.setenv("PA_TC_TEST_WITHHOLD_Q", "1")
    qd = q.cuda()
    if kind == "blk8":
        ops.pa_prefill_blk8(out, qd, c.k, c.v, c.ks, c.vsc, c.bt, c.cl, qs, 100, 0.09, max(lens), 0, 0, err)
    else:
        ops.pa_prefill_window_kv(out, qd, c.k, c.v, 1.0, 1.0, c.bt, c.cl, qs, 100, 0.09, window, sinks, max(lens), err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.PA_DEV_TIMEOUT, "no wait ran out"
    monkeypatch.delenv("PA_TC_WAIT_NS")
    monkeypatch.delenv("PA_TC_TEST_WITHHOLD_Q")
    out = prefill(c, q, new, 0.09, window, sinks)
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            ref, tol = attend(q[at + i].double(), c.k64[b], c.v64[b], sees(n, n - m + i, window, sinks), 0.09,
                              2.0 ** -16, 2.0 ** -34)
            check(out[at + i], ref, tol, f"sequence {b}, token {i}")
        at += m
