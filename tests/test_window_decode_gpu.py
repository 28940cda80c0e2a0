"""Windowed decode and decode over the block-scaled 8-bit cache against 64-bit references:
every type, group size, head size and block size; windows and sinks that end on, before and
behind tile and block edges; empty sequences; NaN in every slot that holds no visible token and
out-of-range table entries for blocks without one; captured, other-stream and shared-workspace
calls."""

import numpy as np
import pytest
import torch

from paged_kv_cache_418_b200 import ops
from window_testlib import DT, Paged, attend, check, visible

pytestmark = pytest.mark.gpu


def _case(seed, ctx, Hq, Hkv, D, bs, qt, kt, vt, window, sinks, blk8=False, spread=0, ks=1.0, vs=1.0):
    keep = [visible(c, c - 1, window, sinks) for c in ctx]
    P = Paged(seed, ctx, Hkv, D, bs, kt, vt, keep, blk8, spread, ks, vs)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(ctx), Hq, D, generator=g).to(DT[qt])
    scale = D ** -0.5
    if kt == "fp8":
        # the codes' values reach 15: keep the scores of a few units
        k_mag = max([1.0] + [float(k.abs().max()) for k in P.k64 if k.numel()])
        scale = scale / k_mag * 4
    ref = torch.zeros(len(ctx), Hq, D, dtype=torch.float64)
    tol = torch.zeros(len(ctx), Hq, 1, dtype=torch.float64)
    for b in range(len(ctx)):
        ref[b], tol[b] = attend(q[b].double(), P.k64[b], P.v64[b], keep[b], scale)
    return P, q, scale, ref, tol


def _run(P, q, scale, window, sinks, ks=1.0, vs=1.0, out_dtype=torch.float32, max_ctx=None, ws=None,
         err=None, stream=None):
    kc, vc, ksc, vsc, bt, cl = P.dev()
    qd = q.cuda()
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    mc = max(P.ctx + [1]) if max_ctx is None else max_ctx
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if err is None else err
    ws = ops.window_workspace_for(qd, kc, mc, window, sinks) if ws is None else ws
    torch.cuda.synchronize()
    if P.blk8:
        ops.pa_decode_blk8(out, qd, kc, vc, ksc, vsc, bt, cl, scale, mc, window, sinks, ws, err, stream)
    else:
        ops.pa_decode_window_kv(out, qd, kc, vc, ks, vs, bt, cl, scale, window, sinks, mc, ws, err, stream)
    torch.cuda.synchronize()
    return out, int(err.item())


CTX = [0, 1, 15, 16, 17, 40, 333, 700]
TYPES = [("f32", "f32", "f32"), ("f16", "f16", "f16"), ("bf16", "bf16", "bf16"),
         ("f32", "fp8", "fp8"), ("f16", "fp8", "fp8"), ("bf16", "fp8", "bf16"), ("f16", "f16", "fp8"),
         ("f16", "fp8", "f16"), ("bf16", "bf16", "fp8")]


@pytest.mark.parametrize("qt,kt,vt", TYPES)
@pytest.mark.parametrize("D,bs,G,Hkv,window,sinks", [
    (128, 16, 8, 2, 100, 4), (64, 32, 1, 3, 33, 17), (128, 32, 16, 1, 16, 0), (64, 16, 4, 2, 1, 1),
    (128, 16, 2, 2, 257, 40), (128, 32, 2, 8, 90, 3), (64, 16, 16, 8, 200, 70), (128, 16, 1, 12, 70, 0)])
def test_window_every_type(qt, kt, vt, D, bs, G, Hkv, window, sinks):
    ks, vs = (0.5, 0.25)
    P, q, scale, ref, tol = _case(D + bs + G + window, CTX, G * Hkv, Hkv, D, bs, qt, kt, vt, window,
                                  sinks, ks=ks, vs=vs)
    out, err = _run(P, q, scale, window, sinks, ks, vs)
    assert err == 0
    check(out, ref, tol, "fp32 output")
    assert torch.equal(out[0], torch.zeros_like(out[0]))            # nothing to attend
    out, err = _run(P, q, scale, window, sinks, ks, vs, out_dtype=DT[qt])
    assert err == 0
    check(out, ref, tol, "query-type output")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (15, 16), (16, 15), (17, 33), (64, 64),
                                          (699, 1), (700, 0), (2 ** 31 - 1, 3), (20, 2 ** 31 - 1)])
def test_window_edges(window, sinks):
    ctx = CTX + [16 * k + d for k in (2, 5, 9) for d in (0, 1, 15)]
    P, q, scale, ref, tol = _case(7, ctx, 8, 2, 128, 32, "bf16", "bf16", "bf16", window, sinks)
    out, err = _run(P, q, scale, window, sinks)
    assert err == 0
    check(out, ref, tol)


@pytest.mark.parametrize("qt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,bs,G,Hkv,window,sinks", [
    (128, 16, 8, 2, 0, 0), (64, 32, 1, 3, 0, 9), (128, 32, 16, 1, 70, 5), (64, 16, 4, 2, 300, 0),
    (128, 16, 1, 4, 0, 0), (128, 16, 8, 8, 0, 0), (64, 32, 2, 16, 150, 20), (128, 32, 16, 8, 0, 0)])
def test_blk8_decode(qt, D, bs, G, Hkv, window, sinks):
    P, q, scale, ref, tol = _case(3 * D + bs + G, CTX, G * Hkv, Hkv, D, bs, qt, "fp8", "fp8", window,
                                  sinks, blk8=True, spread=3)
    for odt in (torch.float32, DT[qt]):
        out, err = _run(P, q, scale, window, sinks, out_dtype=odt)
        assert err == 0
        check(out, ref, tol, str(odt))


def test_blk8_v_scales_far_apart():
    """V scales 2^-66 .. 2^54: the weights are normalised to the largest contribution, so no
    block's part is lost to the 16-bit range of the weights."""
    P, q, scale, ref, tol = _case(11, [300, 64, 17], 16, 2, 128, 16, "bf16", "fp8", "fp8", 0, 0,
                                  blk8=True, spread=60)
    out, err = _run(P, q, scale, 0, 0)
    assert err == 0
    check(out, ref, tol)
    # one block with tiny values holds nearly all the weight: its own magnitude must survive
    P, q, scale, ref, tol = _case(12, [16], 8, 1, 128, 16, "f16", "fp8", "fp8", 0, 0, blk8=True, spread=60)
    out, err = _run(P, q, scale, 0, 0)
    check(out, ref, tol)


def test_peaked_and_rising_scores():
    """Scores that rise by far more than 2^16 along the sequence move the reference maximum."""
    for qt in ("f16", "bf16"):
        P, q, scale, _, _ = _case(21, [900, 130], 8, 1, 128, 16, qt, qt, qt, 800, 4)
        scale = scale * 25
        ref = torch.zeros(2, 8, 128, dtype=torch.float64)
        tol = torch.zeros(2, 8, 1, dtype=torch.float64)
        for b, c in enumerate(P.ctx):
            ref[b], tol[b] = attend(q[b].double(), P.k64[b], P.v64[b], visible(c, c - 1, 800, 4), scale)
        out, err = _run(P, q, scale, 800, 4)
        assert err == 0
        check(out, ref, tol, qt)


def test_bad_lengths_blocks_and_scales_are_flagged_and_left_out():
    ctx = [100, 50, 90]
    P, q, scale, ref, tol = _case(31, ctx, 8, 2, 128, 16, "bf16", "bf16", "bf16", 60, 0)
    # max_context_len below sequence 0's length: zeros and a flag, the others unharmed
    out, err = _run(P, q, scale, 60, 0, max_ctx=95)
    assert err == ops.PA_DEV_BAD_CTX
    assert torch.equal(out[0], torch.zeros_like(out[0]))
    check(out[1:], ref[1:], tol[1:])
    # a bad block inside the window: its tokens are left out
    P.tables[2, 4] = P.pools[0].shape[0]
    keep = visible(90, 89, 60, 0)
    keep[64:80] = False
    r2, t2 = attend(q[2].double(), P.k64[2], P.v64[2], keep, scale)
    out, err = _run(P, q, scale, 60, 0)
    assert err == ops.PA_DEV_BAD_BLOCK_ID
    check(out[2], r2, t2)
    # an invalid block scale: the block is left out for that head
    P, q, scale, ref, tol = _case(32, [80], 8, 2, 128, 16, "bf16", "fp8", "fp8", 0, 0, blk8=True, spread=2)
    ph = int(P.tables[0, 2])
    for bad in (0.0, float("nan"), 3.0, -1.0, float("inf")):
        P.scales[0][ph, 1] = bad
        keep = visible(80, 79, 0, 0)
        keep[32:48] = False
        r1, t1 = attend(q[0].double(), P.k64[0], P.v64[0], keep, scale)
        out, err = _run(P, q, scale, 0, 0)
        assert err == ops.PA_DEV_BAD_SCALE
        check(out[0, 4:], r1[4:], t1[4:], f"scale {bad}")
        check(out[0, :4], ref[0, :4], tol[0, :4], f"scale {bad}: the other head")
    # every block bad: zeros
    P.tables[:] = -1
    out, err = _run(P, q, scale, 0, 0)
    assert err & ops.PA_DEV_BAD_BLOCK_ID and torch.equal(out, torch.zeros_like(out))


def test_nan_in_a_visible_value_reaches_the_output_only_of_its_head():
    P, q, scale, ref, tol = _case(41, [70], 8, 2, 64, 16, "f16", "fp8", "fp8", 0, 0, blk8=True, spread=1)
    P.pools[1][int(P.tables[0, 1]), 3, 0, 5] = 0x7F
    out, err = _run(P, q, scale, 0, 0)
    assert bool(torch.isnan(out[0, :4, 5]).all())
    rest = torch.ones(64, dtype=torch.bool)
    rest[5] = False
    check(out[0, :4][:, rest], ref[0, :4][:, rest], tol[0, :4])
    check(out[0, 4:], ref[0, 4:], tol[0, 4:])


def test_long_context_one_sequence_and_a_large_loose_bound():
    """One sequence split over the whole GPU, with the exact bound and with one far too large."""
    P, q, scale, ref, tol = _case(51, [9001], 4, 1, 128, 32, "bf16", "fp8", "fp8", 0, 0, blk8=True, spread=2)
    for mc in (9001, 200000):
        P.tables = np.pad(P.tables, ((0, 0), (0, -(-mc // 32) - P.tables.shape[1])), constant_values=-1)
        out, err = _run(P, q, scale, 0, 0, max_ctx=mc)
        assert err == 0
        check(out, ref, tol, f"bound {mc}")


def test_two_graphs_share_a_workspace_and_replay():
    A = _case(61, [900, 20, 333], 16, 2, 128, 16, "bf16", "bf16", "bf16", 500, 4)
    B = _case(62, [77, 1200], 16, 2, 128, 16, "bf16", "fp8", "fp8", 0, 0, blk8=True, spread=2)
    n = max(ops.pa_window_workspace_size(3, 16, 2, 128, 900, 500, 4),
            ops.pa_window_workspace_size(2, 16, 2, 128, 1200, 0, 0), 256)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for (P, q, scale, ref, tol), w, s in ((A, 500, 4), (B, 0, 0)):
        t = P.dev()
        qd = q.cuda()
        out = torch.full(q.shape, float("nan"), device="cuda")
        def call(P=P, t=t, qd=qd, out=out, scale=scale, w=w, s=s):
            if P.blk8:
                ops.pa_decode_blk8(out, qd, t[0], t[1], t[2], t[3], t[4], t[5], scale, max(P.ctx), w, s, ws)
            else:
                ops.pa_decode_window_kv(out, qd, t[0], t[1], 1.0, 1.0, t[4], t[5], scale, w, s,
                                        max(P.ctx), ws)
        call()
        torch.cuda.synchronize()
        first = out.clone()
        check(first, ref, tol)
        out.fill_(float("nan"))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append((gr, out, first, call))    # (call keeps the inputs alive)
    for _ in range(3):
        for gr, out, *_ in graphs:
            out.fill_(float("nan"))
            gr.replay()
    torch.cuda.synchronize()
    for _, out, first, _ in graphs:
        assert torch.equal(out, first)              # the same bits, replay after replay


def test_other_stream_and_repeatability():
    P, q, scale, ref, tol = _case(71, [800] * 3, 8, 8, 128, 16, "f16", "f16", "f16", 640, 0)
    s = torch.cuda.Stream()
    first, _ = _run(P, q, scale, 640, 0)
    again, err = _run(P, q, scale, 640, 0, stream=s)
    assert err == 0 and torch.equal(first, again)
    check(first, ref, tol)


def test_blocks_past_4_gib():
    """Physical blocks whose byte offsets pass 32 bits, in the append and in the decode."""
    Hq, Hkv, D, bs = 8, 8, 128, 32
    nb = (1 << 32) // (bs * Hkv * D) + 40                    # 4.3 GB of codes per pool
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    kc = torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(nb, Hkv, device="cuda"), torch.zeros(nb, Hkv, device="cuda")
    g = torch.Generator().manual_seed(5)
    T = 70
    blocks = torch.tensor([nb - 1, 3, nb - 30])
    slots = blocks[torch.arange(T) // bs] * bs + torch.arange(T) % bs
    x = torch.randn(T, 2 * Hkv, D, generator=g).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_rope_and_cache_blk8(None, None, x[:, :Hkv], x[:, Hkv:], None, None, kc, vc, ks, vs, slots.cuda(), False,
                               err)
    from window_testlib import e4m3_values
    val = e4m3_values()
    at = blocks[torch.arange(T) // bs]
    k64, v64 = (val[p.cpu()[at, torch.arange(T) % bs].long()] * s.cpu().double()[at][..., None]
                for p, s in ((kc, ks), (vc, vs)))
    assert float((k64 - x[:, :Hkv].cpu().double()).abs().max()) < 0.5      # rows did land there
    q = torch.randn(1, Hq, D, generator=g).bfloat16()
    ref, tol = attend(q[0].double(), k64, v64, visible(T, T - 1, 0, 0), D ** -0.5)
    out = torch.empty(1, Hq, D, device="cuda")
    ws = ops.window_workspace_for(q, kc, T)
    ws = None if ws is None else ws.cuda()
    ops.pa_decode_blk8(out, q.cuda(), kc, vc, ks, vs, blocks[None].int().cuda(),
                       torch.tensor([T], dtype=torch.int32, device="cuda"), D ** -0.5, T, 0, 0, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(out[0], ref, tol)


@pytest.mark.parametrize("blk8", [True, False])
def test_many_sequences_of_all_lengths(blk8):
    """More units than the GPU has CTAs, empty ones among them: batches of units, cuts inside and
    between sequences."""
    ctx = [(i * i * 7) % 400 if i % 5 else 0 for i in range(300)]
    kt = "fp8" if blk8 else "f16"
    P, q, scale, ref, tol = _case(81, ctx, 24, 12, 64, 16, "f16", kt, kt, 0 if blk8 else 150, 2, blk8=blk8, spread=3)
    out, err = _run(P, q, scale, 0 if blk8 else 150, 2)
    assert err == 0
    check(out, ref, tol)
