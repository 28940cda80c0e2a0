"""Attention whose weights or value scales span many powers of two: inputs, 64-bit references and
bounds that follow each weight.

With w_t the weight of key t over the largest one, the exact row is sum w_t v_t / sum w_t. A
kernel's row differs from it by
 * the scores: products of 16-bit operands are exact in fp32, their sum over D dims is taken in
   D / 16 accumulation steps, doubled for the roundings of the score itself: 2 (D / 16) 2^-23
   scale sum_d |q_d k_td|, and forming s - m rounds at the size of the scores, |s| 2^-22: e_t,
   relative to w_t, in the numerator and in the sum;
 * the weights as the output product takes them: off by rel w_t + floor (both as fractions of the
   largest weight; of the largest w_t * (V scale of t) where V carries block scales, whose weights are
   normalised to that);
 * the sums over N keys, taken 16 keys at a time: two accumulations of at most 2^-23 each per step
   (a weight has two parts), with 64 more for the steps that join the parts of a row: N' =
   (N / 8 + 64) 2^-23 of the sum of the terms' magnitudes (the exp-sum likewise);
so |row' - row| <= [sum (e_t + rel + N') w_t |v_t| + floor sum |v_t|] / W + |row| sum (e_t + N') w_t / W
with W = sum w_t, plus half a step of the output type."""

import numpy as np
import torch

from paged_kv_cache_418_b200 import ops

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


def attend(q, k, v, ok, scale, rel, floor, vs=None):
    """Row of one token's heads q [Hq, D] over k, v [n, Hkv, D] (doubles; ok [n]: visible keys) and its
    bound; vs [n, Hkv]: the V scale of each key (v holds the scaled values), None: 1."""
    Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, tol = torch.zeros(Hq, D, dtype=torch.float64), torch.zeros(Hq, D, dtype=torch.float64)
    idx = torch.nonzero(ok).flatten()
    n = idx.numel()
    steps = (n / 8 + 64) * 2.0 ** -23
    for h in range(Hkv):
        qq, kk, vv = q[h * G:(h + 1) * G], k[idx, h], v[idx, h]
        s = qq @ kk.T * scale
        w = torch.exp(s - s.amax(dim=-1, keepdim=True))
        W = w.sum(dim=-1, keepdim=True)
        e = 2 * (D / 16) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().T) + 2.0 ** -22 * s.abs().amax()
        x = torch.ones(n, dtype=torch.float64) if vs is None else vs[idx, h]
        if vs is not None:                       # s + log2 of the V scale, rounded at its size
            e = e + 2.0 ** -22 * (torch.log2(x).abs().amax() + 1)
        most = (w * x).amax(dim=-1, keepdim=True)
        o = (w @ vv) / W
        out[h * G:(h + 1) * G] = o
        near = ((w * (e + rel + steps)) @ vv.abs()) / W
        far = most * floor * (vv.abs() / x[:, None]).sum(dim=0)[None] / W
        total = (w * (e + steps)).sum(dim=-1, keepdim=True) / W
        tol[h * G:(h + 1) * G] = near + far + o.abs() * total
    return out, tol


def check(got, ref, tol, what=""):
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    half = torch.finfo(got.dtype).eps / 2
    bound = tol * (1 + half) + half * ref.abs() + torch.finfo(got.dtype).smallest_normal * half
    over = (g - ref).abs() / bound
    assert float(over.max()) <= 1, f"{what}: {int((over > 1).sum())} of {over.numel()} beyond the bound, worst {float(over.max()):.3g} times it"


class Cache:
    """A paged cache of one type per pool ("f16", "bf16", "fp8"; or blk8: codes with scales
    2^exps [blocks of the sequence, Hkv]) that holds each sequence's k, v [n, Hkv, D] (float32),
    and the doubles it holds."""

    def __init__(self, seqs, bs, kt, vt, exps=None, seed=0):
        Hkv, D = seqs[0][0].shape[1:]
        need = [-(-k.shape[0] // bs) for k, _ in seqs]
        nb = sum(need) + 2
        perm = torch.from_numpy(np.random.default_rng(seed).permutation(nb))
        self.tables = torch.full((len(seqs), max(need)), -7, dtype=torch.int32)
        self.ctx = [k.shape[0] for k, _ in seqs]
        self.blk8, self.bs = exps is not None, bs
        self.k64, self.v64, self.vs = [], [], []
        pools = [torch.full((nb, bs, Hkv, D), 0x7F, dtype=torch.uint8) if t == "fp8" else
                 torch.full((nb, bs, Hkv, D), float("nan"), dtype=DT[t]) for t in (kt, vt)]
        self.scales = [torch.full((nb, Hkv), float("nan")) for _ in range(2)]
        at = 0
        for b, (n, kv) in enumerate(zip(self.ctx, seqs)):
            ids = perm[at:at + need[b]]
            at += need[b]
            self.tables[b, :need[b]] = ids.int()
            t = torch.arange(n)
            for which, (x, kind) in enumerate(zip(kv, (kt, vt))):
                f = torch.ones(n, Hkv, dtype=torch.float64)
                if self.blk8:
                    ex = torch.zeros(need[b], Hkv) if which == 0 else exps[b].float()
                    self.scales[which][ids] = torch.exp2(ex)
                    f = torch.exp2(ex.double())[t // bs]
                if kind == "fp8":
                    code = (x.double() / f[..., None]).float().to(E4M3)
                    pools[which][ids[t // bs], t % bs] = code.view(torch.uint8)
                    held = code.double() * f[..., None]
                else:
                    pools[which][ids[t // bs], t % bs] = x.to(DT[kind])
                    held = x.to(DT[kind]).double()
                (self.k64 if which == 0 else self.v64).append(held)
                if which:
                    self.vs.append(f)
        self.k, self.v, self.ks, self.vsc = (x.cuda() for x in pools + self.scales)
        self.bt = self.tables.cuda()
        self.cl = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")


def decode(c, q, scale, window=0, sinks=0, out_dtype=torch.float32, kscale=1.0, vscale=1.0):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd, mc = q.cuda(), max(c.ctx)
    ws = ops.window_workspace_for(qd, c.k, mc, window, sinks)
    if c.blk8:
        ops.pa_decode_blk8(out, qd, c.k, c.v, c.ks, c.vsc, c.bt, c.cl, scale, mc, window, sinks, ws, err)
    else:
        ops.pa_decode_window_kv(out, qd, c.k, c.v, kscale, vscale, c.bt, c.cl, scale, window, sinks, mc, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def prefill(c, q, new, scale, window=0, sinks=0, out_dtype=torch.float32):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    qd, mc = q.cuda(), max(c.ctx)
    if c.blk8:
        ops.pa_prefill_blk8(out, qd, c.k, c.v, c.ks, c.vsc, c.bt, c.cl, qs, max(new), scale, mc, window, sinks, err)
    else:
        ops.pa_prefill_window_kv(out, qd, c.k, c.v, 1.0, 1.0, c.bt, c.cl, qs, max(new), scale, window, sinks, mc, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def sees(n, pos, window, sinks):
    t = torch.arange(n)
    ok = t <= pos
    return ok & ((t > pos - window) | (t < sinks)) if window else ok


def sink(seed, T, n, Hq, Hkv, D, share, qt):
    """q [T, Hq, D] and k, v [n, Hkv, D] whose key 0 takes about `share` of every row's weight and has
    the value 0; the other scores are about N(0, 1)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, Hq, D, generator=g)
    q[..., 0] = 8
    k, v = torch.randn(n, Hkv, D, generator=g), torch.randn(n, Hkv, D, generator=g)
    k[..., 0] = 0
    k[0] = 0
    k[0, :, 0] = float(np.log(share / (1 - share) * n * 1.65) * D ** 0.5 / 8)
    v[0] = 0
    return q.to(DT[qt]), k, v


def spread(seed, lens, Hkv, D, kind, qt, new=None, G=4):
    """Sequences over the block-scaled cache (blocks of 16): "zeros20" / "zeros100": every other block has
    no value at all (scale 2^-100, as the append leaves it) beside values near 2^20 / 2^100, its scores 4
    higher; "low": 1000 such tokens whose scores are 7 lower; "any": scales 2^-100 .. 2^120 at random."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(new) if new else len(lens), G * Hkv, D, generator=g).to(DT[qt])
    q[..., 0] = 4
    seqs, exps = [], []
    for n in lens:
        nb = -(-n // 16)
        k, v = torch.randn(n, Hkv, D, generator=g), torch.randn(n, Hkv, D, generator=g)
        block = torch.arange(n) // 16
        if kind == "any":
            e = torch.randint(-100, 121, (nb, Hkv), generator=g)
            k[..., 0] = 0
        else:
            none = torch.arange(nb) % 2 == 0 if kind != "low" else torch.arange(nb) >= 4
            e = torch.where(none, -100, int(kind[5:]) if kind != "low" else 20)[:, None].expand(nb, Hkv).contiguous()
            v[none[block]] = 0
            k[..., 0] = torch.where(none[block], -7.0 if kind == "low" else 4.0, 0.0)[:, None] * D ** 0.5 / 4
        seqs.append((k, v * torch.exp2(e.float())[block][..., None]))
        exps.append(e)
    return q, Cache(seqs, 16, "fp8", "fp8", exps)
