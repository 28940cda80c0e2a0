"""Windowed prefill and prefill over the block-scaled 8-bit cache against 64-bit references, and a
serving run of append, prefill and decode together."""

import numpy as np
import pytest
import torch

from paged_kv_cache_418_b200 import ops
from window_testlib import DT, Paged, attend, check, e4m3_values, visible

pytestmark = pytest.mark.gpu


def _w(vt):
    """Error of a weight, relative. Over an 8-bit V pool it is one f16 value: 10 fraction bits, so
    half a step is 2^-11 of a power of two and at most 2^-11 of any value (not 2^-12, which is half
    a step of 11 fraction bits). Each term of a row is then off by up to 2^-11 of itself, and so is
    the row by 2^-11 of the sum of the terms' magnitudes."""
    return 2.0 ** -11 + 2.0 ** -15 if vt == "fp8" else 2.0 ** -15


def _case(seed, prior, new, Hq, Hkv, bs, qt, kt, vt, window, sinks, blk8=False, spread=0, ks=1.0, vs=1.0,
          sharp=1.0):
    ctx = [p + n for p, n in zip(prior, new)]
    keep = []
    for c, n in zip(ctx, new):
        k = torch.zeros(c, dtype=torch.bool)
        for i in range(n):
            k |= visible(c, c - n + i, window, sinks)
        keep.append(k)
    P = Paged(seed, ctx, Hkv, 128, bs, kt, vt, keep, blk8, spread, ks, vs)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(new)
    q = torch.randn(T, Hq, 128, generator=g).to(DT[qt])
    scale = 128 ** -0.5 * sharp
    if kt == "fp8":
        scale = scale / max([1.0] + [float(k.abs().max()) for k in P.k64 if k.numel()]) * 4
    ref = torch.zeros(T, Hq, 128, dtype=torch.float64)
    tol = torch.zeros(T, Hq, 1, dtype=torch.float64)
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in range(n):
            ref[at], tol[at] = attend(q[at].double(), P.k64[b], P.v64[b], visible(c, c - n + i, window, sinks),
                                      scale, _w(vt))
            at += 1
    return P, q, scale, ref, tol, list(new)


def _run(P, q, scale, new, window, sinks, ks=1.0, vs=1.0, out_dtype=torch.float32, max_ctx=None, stream=None):
    kc, vc, ksc, vsc, bt, cl = P.dev()
    qd = q.cuda()
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    qs = torch.tensor(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mc = max(P.ctx) if max_ctx is None else max_ctx
    torch.cuda.synchronize()
    if P.blk8:
        ops.pa_prefill_blk8(out, qd, kc, vc, ksc, vsc, bt, cl, qs, max(new), scale, mc, window, sinks, err,
                            stream)
    else:
        ops.pa_prefill_window_kv(out, qd, kc, vc, ks, vs, bt, cl, qs, max(new), scale, window, sinks, mc, err,
                                 stream)
    torch.cuda.synchronize()
    return out, int(err.item())


TYPES = [("f16", "f16", "f16"), ("bf16", "bf16", "bf16"), ("bf16", "fp8", "fp8"), ("f16", "fp8", "f16"),
         ("bf16", "bf16", "fp8")]
SEQS = ([0, 300, 131, 7, 500, 255], [1, 40, 0, 130, 3, 17])


@pytest.mark.parametrize("qt,kt,vt", TYPES)
@pytest.mark.parametrize("G,Hkv,bs,window,sinks", [(8, 2, 16, 100, 4), (1, 3, 32, 33, 17), (4, 2, 32, 1, 0),
                                                   (16, 1, 16, 257, 150), (2, 2, 16, 128, 128)])
def test_window_prefill(qt, kt, vt, G, Hkv, bs, window, sinks):
    P, q, scale, ref, tol, new = _case(G + bs + window, *SEQS, G * Hkv, Hkv, bs, qt, kt, vt, window, sinks,
                                       ks=0.5, vs=0.25)
    for odt in (torch.float32, DT[qt]):
        out, err = _run(P, q, scale, new, window, sinks, 0.5, 0.25, odt)
        assert err == 0
        check(out, ref, tol, str(odt))


@pytest.mark.parametrize("window,sinks", [(1, 1), (127, 129), (128, 0), (129, 127), (300, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 0)])
def test_window_prefill_edges(window, sinks):
    P, q, scale, ref, tol, new = _case(5, [0, 1000, 640], [200, 65, 128], 4, 1, 16, "bf16", "bf16", "bf16",
                                       window, sinks)
    out, err = _run(P, q, scale, new, window, sinks)
    assert err == 0
    check(out, ref, tol)


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("G,Hkv,bs,window,sinks,spread", [
    (8, 2, 16, 0, 0, 3), (1, 2, 32, 0, 9, 60), (4, 2, 32, 90, 5, 3), (16, 1, 16, 257, 0, 60), (2, 2, 16, 64, 200, 3)])
def test_blk8_prefill(qt, G, Hkv, bs, window, sinks, spread):
    P, q, scale, ref, tol, new = _case(G + bs + 7 * window, *SEQS, G * Hkv, Hkv, bs, qt, "fp8", "fp8", window,
                                       sinks, blk8=True, spread=spread)
    for odt in (torch.float32, DT[qt]):
        if odt == torch.float16 and spread > 10:
            continue                            # the values themselves pass f16's range
        out, err = _run(P, q, scale, new, window, sinks, out_dtype=odt)
        assert err == 0
        check(out, ref, tol, str(odt))


def test_rising_scores():
    for qt in ("f16", "bf16"):
        P, q, scale, ref, tol, new = _case(9, [700, 100], [30, 150], 8, 1, 16, qt, qt, qt, 600, 4, sharp=25.0)
        out, err = _run(P, q, scale, new, 600, 4)
        assert err == 0
        check(out, ref, tol, qt)


def test_bad_lengths_blocks_and_scales():
    P, q, scale, ref, tol, new = _case(13, [80, 30], [20, 10], 8, 2, 16, "bf16", "fp8", "fp8", 0, 0, blk8=True,
                                       spread=2)
    out, err = _run(P, q, scale, new, 0, 0, max_ctx=99)
    assert err == ops.PA_DEV_BAD_CTX                          # sequence 0: not written
    assert bool(torch.isnan(out[:20]).all())
    check(out[20:], ref[20:], tol[20:])
    for what in ("scale", "block"):
        keep = visible(100, 99, 0, 0)
        keep[32:48] = False
        if what == "scale":
            P.scales[1][int(P.tables[0, 2])] = 0.0
        else:
            P.tables[0, 2] = -5
        out, err = _run(P, q, scale, new, 0, 0)
        assert err == (ops.PA_DEV_BAD_SCALE if what == "scale" else ops.PA_DEV_BAD_BLOCK_ID)
        for i in (0, 7, 19):
            r, t = attend(q[i].double(), P.k64[0], P.v64[0], keep & visible(100, 80 + i, 0, 0), scale, _w("fp8"))
            check(out[i], r, t, what)
        check(out[20:], ref[20:], tol[20:], what)


def test_query_starts_past_the_queries_are_flagged_and_nothing_is_written():
    P, q, scale, ref, tol, new = _case(14, [40, 30], [20, 10], 4, 1, 16, "f16", "f16", "f16", 50, 2)
    kc, vc, _, _, bt, cl = P.dev()
    for qs, whole in (([0, 20, 35], 0), ([-3, 20, 30], 1), ([20, 0, 10], 1)):
        out = torch.full((64, 4, 128), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_prefill_window_kv(out[:30], q.cuda(), kc, vc, 1.0, 1.0, bt, cl,
                                 torch.tensor(qs, dtype=torch.int32, device="cuda"), 20, scale, 50, 2, 60, err)
        torch.cuda.synchronize()
        assert int(err.item()) == ops.PA_DEV_BAD_CTX
        assert bool((out[30:] == 7.0).all())


@pytest.mark.parametrize("qt,kt,vt", [("bf16", "bf16", "bf16"), ("bf16", "fp8", "fp8"), ("f16", "f16", "fp8")])
def test_many_short_units(qt, kt, vt):
    """Chunks of one tile and one token, hundreds of units per CTA: every buffer's turn."""
    n = 700
    prior = [(37 * i) % 90 for i in range(n)]
    new = [1 + (i % 3) for i in range(n)]
    P, q, scale, ref, tol, new = _case(15, prior, new, 8, 4, 16, qt, kt, vt, 60, 1)
    out, err = _run(P, q, scale, new, 60, 1)
    assert err == 0
    check(out, ref, tol)


@pytest.mark.parametrize("blk8", [True, False])
def test_serving_run(blk8):
    """A prompt in chunks, then single tokens: append with rotation, prefill, decode, a fork that
    copies a block with its scales; every output against the attention of the rows as cached."""
    Hq, Hkv, D, bs, nb, window, sinks = 8, 2, 128, 16, 40, 70, 3
    g = torch.Generator().manual_seed(77)
    half = 64
    a = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half).double() / half)[None]
    cs = torch.cat([a.cos(), a.sin()], dim=1).float().cuda()
    dt = torch.bfloat16
    pool_dt = torch.uint8 if blk8 else dt
    kc = torch.zeros(nb, bs, Hkv, D, dtype=pool_dt, device="cuda")
    vc = torch.zeros_like(kc)
    ksc = torch.ones(nb, Hkv, device="cuda")
    vsc = torch.ones(nb, Hkv, device="cuda")
    table = torch.randperm(nb, generator=g)[:20].to(torch.int32)
    bt = table[None].cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    vals = e4m3_values()
    ctx, scale = 0, D ** -0.5

    def cached(tab, n):
        at = torch.arange(n)
        ph = tab.cpu().long()[at // bs]
        out = []
        for pool, sc in ((kc, ksc), (vc, vsc)):
            r = pool.cpu()[ph, at % bs]
            out.append(vals[r.long()] * sc.cpu().double()[ph][..., None] if blk8 else r.double())
        return out

    def step(n, tab, bt):
        x = torch.randn(n, Hq + 2 * Hkv, D, generator=g).to(dt).cuda()
        q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
        pos = torch.arange(ctx, ctx + n)
        slots = (tab.cpu().long()[pos // bs] * bs + pos % bs).cuda()
        qo = torch.empty(n, Hq, D, dtype=dt, device="cuda")
        cl = torch.tensor([ctx + n], dtype=torch.int32, device="cuda")
        out = torch.empty(n, Hq, D, device="cuda")
        if blk8:
            ops.pa_rope_and_cache_blk8(qo, q, k, v, pos.cuda(), cs, kc, vc, ksc, vsc, slots, False, err)
        else:
            ops.pa_rope_and_cache_kv(qo, q, k, v, pos.cuda(), cs, kc, vc, 1.0, 1.0, slots, False, err)
        if n > 1:
            qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            if blk8:
                ops.pa_prefill_blk8(out, qo, kc, vc, ksc, vsc, bt, cl, qs, n, scale, ctx + n, window, sinks, err)
            else:
                ops.pa_prefill_window_kv(out, qo, kc, vc, 1.0, 1.0, bt, cl, qs, n, scale, window, sinks,
                                         ctx + n, err)
        else:
            ws = ops.window_workspace_for(qo, kc, ctx + n, window, sinks)
            if blk8:
                ops.pa_decode_blk8(out, qo, kc, vc, ksc, vsc, bt, cl, scale, ctx + n, window, sinks, ws, err)
            else:
                ops.pa_decode_window_kv(out, qo, kc, vc, 1.0, 1.0, bt, cl, scale, window, sinks, ctx + n, ws, err)
        torch.cuda.synchronize()
        k64, v64 = cached(tab, ctx + n)
        for i in range(n):
            ref, tol = attend(qo[i].cpu().double(), k64, v64, visible(ctx + n, ctx + i, window, sinks), scale,
                              _w("fp8") if blk8 and n > 1 else 2.0 ** -15)
            check(out[i], ref, tol, f"token {ctx + i}")

    for n in (50, 1, 1, 37, 1, 64, 1):
        step(n, table, bt)
        ctx += n
    # fork: the last, partly filled block is copied with its scales; both go on
    last = ctx // bs
    free = [b for b in range(nb) if b not in table.tolist()][0]
    pair = torch.tensor([[int(table[last]), free]]).cuda()
    if blk8:
        ops.pa_copy_blocks(kc, vc, pair, err)
        ops.pa_copy_scales(ksc, vsc, ksc, vsc, pair, err)
    else:
        ops.pa_copy_blocks(kc, vc, pair, err)
    fork = table.clone()
    fork[last] = free
    step(1, fork, fork[None].cuda())
    step(1, table, bt)
    assert int(err.item()) == 0


@pytest.mark.parametrize("kind,window,sinks", [("blk8", 0, 0), ("blk8", 200, 30), ("same", 200, 30), ("same", 2 ** 31 - 1, 0)])
def test_units_of_every_kind_in_turn(kind, window, sinks):
    # several hundred units, so that each CTA has some of one query tile and one key tile, of
    # one query tile and several key tiles (which two groups of warps share) and of two query tiles
    rng = np.random.default_rng(7)
    new = [int(x) for x in rng.choice([1, 15, 16, 17, 31, 33, 40, 70], 50)]
    prior = [int(x) for x in rng.choice([0, 1, 60, 130, 280, 400], 50)]
    blk8 = kind == "blk8"
    for qt in ("f16", "bf16"):
        kt = "fp8" if blk8 else qt
        P, q, scale, ref, tol, new = _case(11, prior, new, 64, 8, 16, qt, kt, kt, window, sinks, blk8=blk8,
                                           spread=3 if blk8 else 0, sharp=4.0)
        out, err = _run(P, q, scale, new, window, sinks)
        assert err == 0
        check(out, ref, tol, qt)
