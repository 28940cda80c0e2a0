"""Rotary append on the GPU against 64-bit references: rotated queries, 16-bit, fp32, FP8 and
block-scaled pools; strided projections, partial rotation, padding and bad tokens; blocks that
start, continue and grow their scale."""

import numpy as np
import pytest
import torch

from paged_kv_cache_418_b200 import ops
from window_testlib import DT, e4m3_values, round_e4m3

pytestmark = pytest.mark.gpu


def _table(n, rot):
    half = rot // 2
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64) / half)[None]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _turn(x, cs, il, f=lambda v: v):
    """Rotation of x [T, H, D] by rows cs [T, rot]; f rounds each product and sum."""
    rot = cs.shape[1]
    half = rot // 2
    c, s = cs[:, None, :half], cs[:, None, half:]
    out = x.clone()
    i0 = slice(0, rot, 2) if il else slice(0, half)
    i1 = slice(1, rot, 2) if il else slice(half, rot)
    a, b = x[..., i0], x[..., i1]
    out[..., i0] = f(f(a * c) - f(b * s))
    out[..., i1] = f(f(b * c) + f(a * s))
    return out


def _near(got, exact, terms, what):
    """|got - exact|: three fp32 roundings of terms of size `terms`, then the type's own."""
    g = got.cpu().double()
    half = torch.finfo(got.dtype).eps / 2
    bound = 3 * 2.0 ** -24 * terms * (1 + half) + half * exact.abs() + \
        torch.finfo(got.dtype).smallest_normal * half
    assert bool(((g - exact).abs() <= bound).all()), f"{what}: {float((g - exact).abs().max())}"


def _terms(x, cs, il):
    return _turn(x.abs(), cs.abs(), il).abs() + 2 * x.abs().amax(dim=-1, keepdim=True)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,rot,il,T,fused", [
    (8, 2, 128, 16, 128, False, 37, True), (4, 4, 64, 32, 64, True, 1, False),
    (16, 1, 128, 32, 48, False, 300, True), (1, 1, 64, 16, 16, True, 5, True), (0, 3, 128, 16, 64, False, 9, False)])
def test_rope_kv(dt, Hq, Hkv, D, bs, rot, il, T, fused):
    g = torch.Generator().manual_seed(T + D + rot)
    nb = 40
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(DT[dt])
    pos = torch.randint(0, 500, (T,), generator=g)
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[::4] = -1 if T > 4 else slots[::4]
    cs = _table(500, rot)
    live = slots >= 0
    q64, k64, v64 = x.double().split([Hq, Hkv, Hkv], dim=1)
    c64 = cs.double()[pos]
    for kv in ("same", "fp8", "k8", "v8"):
        if kv in ("k8", "v8") and dt == "f32" and Hq != 8:
            continue
        k8, v8 = kv in ("fp8", "k8"), kv in ("fp8", "v8")
        kp = torch.full((nb, bs, Hkv, D), 77, dtype=torch.uint8 if k8 else DT[dt])
        vp = torch.full((nb, bs, Hkv, D), 77, dtype=torch.uint8 if v8 else DT[dt])
        dk, dv = kp.cuda(), vp.cuda()
        xd = x.cuda()
        q, k, v = xd.split([Hq, Hkv, Hkv], dim=1)
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        qo = torch.full((T, Hq, D), 5.0, dtype=DT[dt], device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_rope_and_cache_kv(qo if Hq else None, q if Hq else None, k, v, pos.cuda(), cs.cuda(), dk, dv,
                                 0.25, 0.5, slots.cuda(), il, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        if Hq:
            _near(qo[live.cuda()], _turn(q64, c64, il)[live], _terms(q64, c64, il)[live], "query")
            assert bool((qo[~live.cuda()] == 5.0).all())            # padding rows are left alone
        want_k, want_v = kp.view(nb * bs, Hkv, D), vp.view(nb * bs, Hkv, D)
        got_k, got_v = dk.cpu().view(nb * bs, Hkv, D), dv.cpu().view(nb * bs, Hkv, D)
        k32 = _turn(x.split([Hq, Hkv, Hkv], dim=1)[1].float(), cs[pos], il)   # fp32, each step rounded
        _near(k32, _turn(k64, c64, il), _terms(k64, c64, il), "the fp32 steps themselves")
        for got, want, q8, rows, sc in ((got_k, want_k, k8, k32, 0.25),
                                        (got_v, want_v, v8, x[:, Hq + Hkv:].float(), 0.5)):
            want = want.clone()
            if q8:
                vals = round_e4m3((rows / sc).double())
                assert torch.equal(e4m3_values()[got[slots[live]].long()], vals[live])
                want[slots[live]] = got[slots[live]]
            else:
                want[slots[live]] = rows.to(got.dtype)[live]
            assert torch.equal(got, want)                           # and nothing else changed


def test_rope_in_place_and_bad_tokens():
    T, Hq, Hkv, D, bs, nb = 6, 4, 2, 128, 16, 4
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    cs = _table(32, 128)
    pos = torch.tensor([0, 31, 32, -1, 7, 9])
    slots = torch.tensor([0, 5, 6, 7, 64, 63])
    before = x.clone()
    kp = torch.zeros(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_rope_and_cache_kv(q, q, k, v, pos.cuda(), cs.cuda(), kp, vp, 1.0, 1.0, slots.cuda(), False, err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.PA_DEV_BAD_POS | ops.PA_DEV_BAD_SLOT
    ok = torch.tensor([0, 1, 5])
    ref = _turn(before[:, :Hq].cpu().float()[ok], cs[pos[ok]], False).bfloat16()
    assert torch.equal(x[:, :Hq].cpu()[ok], ref)
    bad = torch.tensor([2, 3, 4])
    assert torch.equal(x.cpu()[bad], before.cpu()[bad])
    assert torch.equal(x[:, Hq:], before[:, Hq:])
    written = set(torch.nonzero(vp.view(-1, Hkv * D).abs().sum(1).cpu()).flatten().tolist())
    assert written == {0, 5, 63}


# ------------------------------------------------------------------ the block-scaled cache

def _need(top):
    """Smallest power of two s >= 2^-100 with top <= 448 s (fp32 values, so exact in double)."""
    s = torch.full_like(top, 2.0 ** -100)
    for e in range(-100, 121):
        s = torch.where(top > 448.0 * 2.0 ** e, torch.full_like(top, 2.0 ** (e + 1)), s)
    return s.clamp(max=2.0 ** 120)


class Model:
    """Reference of a block-scaled pool: values of codes and scales, in double."""

    def __init__(self, codes, scales):
        self.val = e4m3_values()[codes.long()]
        self.sc = scales.double()
        self.bs = codes.shape[1]

    def append(self, rows32, slots):
        live = [(int(s) // self.bs, int(s) % self.bs, i) for i, s in enumerate(slots.tolist()) if s >= 0]
        for blk in sorted({b for b, _, _ in live}):
            offs = [o for b, o, _ in live if b == blk]
            r = rows32[[i for b, _, i in live if b == blk]].double()
            mag = r.abs()
            top = torch.where(torch.isfinite(mag), mag, torch.zeros_like(mag)).amax(dim=(0, 2))
            s = _need(top)
            if 0 not in offs:
                s = torch.maximum(s, self.sc[blk])
                grow = s > self.sc[blk]
                scaled = round_e4m3(self.val[blk] * (self.sc[blk] / s)[None, :, None])
                self.val[blk] = torch.where(grow[None, :, None], scaled, self.val[blk])
            self.sc[blk] = s
            for j, o in enumerate(offs):
                self.val[blk, o] = round_e4m3(r[j] / s[:, None])

    def same(self, codes, scales):
        assert torch.equal(self.sc, scales.cpu().double())
        got = e4m3_values()[codes.cpu().long()]
        same = (got == self.val) | (torch.isnan(got) & torch.isnan(self.val))
        assert bool(same.all()), (int((~same).sum()), torch.nonzero(~same)[:8].tolist())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,rot,il", [(8, 2, 128, 16, 128, False), (4, 1, 64, 32, 32, True),
                                                (3, 3, 128, 32, 64, True), (16, 8, 64, 16, 64, False)])
def test_blk8_append_steps(dt, Hq, Hkv, D, bs, rot, il):
    """Chunks and single tokens of several sequences, call after call: blocks start, fill, and grow
    their scale when a later token is larger."""
    g = torch.Generator().manual_seed(D + bs + rot)
    nb = 24
    codes = [torch.randint(0, 256, (nb, bs, Hkv, D), generator=g).to(torch.uint8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-8, 3, (nb, Hkv), generator=g).float()) for _ in range(2)]
    models = [Model(c, s) for c, s in zip(codes, scales)]
    dc, ds = [c.cuda() for c in codes], [s.cuda() for s in scales]
    cs = _table(400, rot)
    tables = torch.randperm(nb, generator=g).view(3, 8)
    lens = [0, 0, 0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step, new in enumerate([(5, bs, 2 * bs + 3), (1, 1, 1), (1, 0, 1), (1, 1, 1), (bs, 7, 1), (1, 1, 1)]):
        pos, slots = [], []
        for b, n in enumerate(new):
            for i in range(lens[b], lens[b] + n):
                pos.append(i)
                slots.append(int(tables[b, i // bs]) * bs + i % bs)
            lens[b] += n
            slots.append(-1)                                     # padding after every sequence
            pos.append(-5)
        T = len(pos)
        pos, slots = torch.tensor(pos), torch.tensor(slots)
        size = torch.exp2(torch.randint(-3, 4, (T, 1, 1), generator=g).float()) * 2.0 ** step
        x = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * size).to(DT[dt])
        xd = x.cuda()
        q, k, v = xd.split([Hq, Hkv, Hkv], dim=1)
        qo = torch.full((T, Hq, D), 5.0, dtype=DT[dt], device="cuda")
        ops.pa_rope_and_cache_blk8(qo, q, k, v, pos.cuda(), cs.cuda(), dc[0], dc[1], ds[0], ds[1],
                                   slots.cuda(), il, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        live = slots >= 0
        at = pos.clamp_min(0)
        q32 = _turn(x[:, :Hq].float(), cs[at], il).to(DT[dt])
        assert torch.equal(qo.cpu()[live], q32[live]) and bool((qo.cpu()[~live] == 5.0).all())
        models[0].append(_turn(x[:, Hq:Hq + Hkv].float(), cs[at], il), slots)
        models[1].append(x[:, Hq + Hkv:].float(), slots)
        models[0].same(dc[0], ds[0])
        models[1].same(dc[1], ds[1])


def test_blk8_append_without_rotation_special_values():
    """Zeros, infinities, NaN, the smallest and largest magnitudes, a bad position inside a run."""
    Hkv, D, bs, nb = 2, 128, 16, 6
    g = torch.Generator().manual_seed(5)
    codes = [torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.full((nb, Hkv), 2.0 ** -4) for _ in range(2)]
    models = [Model(c, s) for c, s in zip(codes, scales)]
    dc, ds = [c.cuda() for c in codes], [s.cuda() for s in scales]
    x = torch.randn(8, 2 * Hkv, D, generator=g)
    x[0] = 0.0                                   # a block of zeros: the smallest scale
    x[1, :, 0] = float("inf")
    x[1, :, 1] = -float("inf")
    x[1, :, 2] = float("nan")
    x[2] *= 1e-42                                # subnormal
    x[3, :, 7] = 3.4028234663852886e38
    x[4] *= 1e-33
    x[5, :, 3] = 448.0 * 2.0 ** 3                # exactly on the border of a scale
    x[6] *= 2.0 ** 30                            # grows a block that holds rows
    slots = torch.tensor([0, 16, 32, 48, 64, 80, 3, -1])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for part in (slice(0, 6), slice(6, 8), slice(0, 1)):
        xd = x[part].cuda()
        ops.pa_rope_and_cache_blk8(None, None, xd[:, :Hkv], xd[:, Hkv:], None, None, dc[0], dc[1], ds[0],
                                   ds[1], slots[part].cuda(), False, err)
        models[0].append(x[part][:, :Hkv], slots[part])
        models[1].append(x[part][:, Hkv:], slots[part])
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        models[0].same(dc[0], ds[0])
        models[1].same(dc[1], ds[1])


def test_blk8_append_bad_position_slot_and_scale():
    Hq, Hkv, D, bs, nb = 2, 1, 128, 16, 4
    g = torch.Generator().manual_seed(6)
    x = torch.randn(6, Hq + 2 * Hkv, D, generator=g)
    cs = _table(64, 128)
    dc = [torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ds = [torch.full((nb, Hkv), 2.0 ** -6, device="cuda") for _ in range(2)]
    ds[1][2] = 0.3                                # block 2 of V: no power of two
    pos = torch.tensor([3, 64, 5, 6, 7, 8])       # token 1's position is past the table
    slots = torch.tensor([16, 17, 18, 64, 35, 36])   # token 3's slot is past the pool
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd = x.cuda()
    qo = torch.zeros(6, Hq, D, device="cuda")
    ops.pa_rope_and_cache_blk8(qo, xd[:, :2], xd[:, 2:3], xd[:, 3:], pos.cuda(), cs.cuda(), dc[0], dc[1],
                               ds[0], ds[1], slots.cuda(), False, err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.PA_DEV_BAD_POS | ops.PA_DEV_BAD_SLOT | ops.PA_DEV_BAD_SCALE
    m = Model(torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8), torch.full((nb, Hkv), 2.0 ** -6))
    keep = torch.tensor([16, -1, 18, -1, 35, 36])
    m.append(_turn(x[:, 2:3], cs[pos.clamp(0, 63)], False), keep)
    m.same(dc[0], ds[0])
    assert float(ds[1][2]) == pytest.approx(0.3) and not bool(dc[1][2].any())
    assert bool(dc[1][1].any())
    live = torch.tensor([0, 2, 4, 5])
    assert torch.equal(qo.cpu()[live], _turn(x[:, :2], cs[pos.clamp(0, 63)], False)[live])
    assert not bool(qo.cpu()[torch.tensor([1, 3])].any())


def test_copy_scales():
    g = torch.Generator().manual_seed(8)
    src = [torch.rand(9, 5, generator=g).cuda() for _ in range(2)]
    dst = [torch.zeros(7, 5).cuda() for _ in range(2)]
    pairs = torch.tensor([[8, 0], [3, 6], [9, 1], [0, 7], [-1, 2]]).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_copy_scales(dst[0], dst[1], src[0], src[1], pairs, err)
    torch.cuda.synchronize()
    assert int(err.item()) == ops.PA_DEV_BAD_PAIR
    for d, s in zip(dst, src):
        want = torch.zeros(7, 5)
        want[0], want[6] = s[8].cpu(), s[3].cpu()
        assert torch.equal(d.cpu(), want)
