"""Inputs and 64-bit references of the windowed, block-scaled and rotary tests.

Attention tolerances. With fp32 output the kernels differ from the exact result by
 * the scores: products of 16-bit operands are exact in fp32 and their sum over D
   dims is taken in D / 16 accumulation steps (D fused multiply-adds on fp32 pools),
   so |s' - s| <= e_s = steps * 2^-23 * scale * sum_d |q_d k_d| (+ a few roundings of
   s itself, covered by doubling the steps), and a score error e moves a weighted
   average of values by at most 2 e max|v|;
 * the weights: two 16-bit parts hold at least 16 bits (2^-16 relative), ex2 2^-22
   (prefill over 8-bit V: one f16 part, half a step is 2^-11: w = 2^-11 + 2^-15);
 * the sums over N keys: at most N roundings of 2^-24 each;
so tol = max|v| (2 e_s + w + (N + 64) 2^-24), w = 2^-15 unless said, plus half a step of the output type.
"""

from __future__ import annotations

import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def e4m3_values() -> torch.Tensor:
    """The 256 E4M3 values in double, from the format's definition."""
    c = torch.arange(256)
    e, f = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(e > 0, torch.exp2(e - 7) * (1 + f / 8), torch.exp2(e - 6) * (f / 8))
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(c >= 128, -v, v)


def round_e4m3(x: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value of each double, ties to even, saturating at +-448; NaN stays."""
    y = x.clamp(-512.0, 512.0)                  # infinities too
    e = torch.floor(torch.log2(y.abs().clamp_min(1e-300))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    r = torch.round(y / step) * step
    return torch.where(torch.isnan(x), x, r.clamp(-448.0, 448.0))


def visible(ctx: int, pos: int, window: int, sinks: int) -> torch.Tensor:
    t = torch.arange(ctx)
    ok = t <= pos
    if window > 0:
        ok &= (t > pos - window) | (t < sinks)
    return ok


class Paged:
    """A paged cache whose slots that hold no visible token are NaN, whose table entries
    of blocks without a visible token are out of range, and its doubles."""

    def __init__(self, seed, ctx, Hkv, D, bs, k_kind, v_kind, keep, blk8=False, spread=0,
                 k_scale=1.0, v_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.bs, self.blk8 = list(ctx), bs, blk8
        B = len(ctx)
        need = [-(-c // bs) for c in ctx]
        nb = sum(need) + 3
        width = max(need + [1])
        perm = rng.permutation(nb)
        self.tables = np.full((B, width), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        vals = e4m3_values()
        self.k64 = [torch.zeros(c, Hkv, D, dtype=torch.float64) for c in ctx]
        self.v64 = [torch.zeros(c, Hkv, D, dtype=torch.float64) for c in ctx]
        self.pools, self.scales = [], []
        for which, (kind, scale, out) in enumerate(((k_kind, k_scale, self.k64),
                                                    (v_kind, v_scale, self.v64))):
            if kind == "fp8":
                pool = torch.full((nb, bs, Hkv, D), 0x7F, dtype=torch.uint8)
            else:
                pool = torch.full((nb, bs, Hkv, D), float("nan"), dtype=DT[kind])
            sc = torch.full((nb, Hkv), float("nan"))
            if blk8:        # scales 2^e, e spread over +-spread (V) or a few steps (K)
                s = spread if which else min(spread, 3)
                sc[:] = torch.exp2(torch.randint(-s - 6, s - 5, (nb, Hkv), generator=g).float())
            for b, c in enumerate(ctx):
                if kind == "fp8":
                    # signs, exponents 3..10 of the format's 16, any fraction
                    code = (torch.randint(0, 2, (c, Hkv, D), generator=g) * 128
                            + torch.randint(3, 11, (c, Hkv, D), generator=g) * 8
                            + torch.randint(0, 8, (c, Hkv, D), generator=g)).to(torch.uint8)
                    x, val = code, vals[code.long()]
                else:
                    x = torch.randn(c, Hkv, D, generator=g).to(DT[kind])
                    val = x.double()
                for t in torch.nonzero(keep[b]).flatten().tolist():
                    ph = int(self.tables[b, t // bs])
                    pool[ph, t % bs] = x[t]
                    f = sc[ph].double()[:, None] if blk8 else (scale if kind == "fp8" else 1.0)
                    out[b][t] = val[t] * f
            self.pools.append(pool)
            self.scales.append(sc)
        for b, c in enumerate(ctx):             # freed blocks
            for i in range(need[b]):
                if not bool(keep[b][i * bs:(i + 1) * bs].any()):
                    self.tables[b, i] = 1 << 29

    def dev(self):
        d = [p.cuda() for p in self.pools]
        s = [x.cuda() for x in self.scales]
        return d[0], d[1], s[0], s[1], torch.from_numpy(self.tables).cuda(), \
            torch.tensor(self.ctx, dtype=torch.int32, device="cuda")


def attend(q, k64, v64, ok, scale, w=2.0 ** -15):
    """Exact attention of one query token's heads q [Hq, D] (double) over keys [c, Hkv, D];
    also the tolerance of each head for fp32 output (w: relative rounding of a weight)."""
    Hq, D = q.shape
    Hkv = k64.shape[1]
    out = torch.zeros(Hq, D, dtype=torch.float64)
    tol = torch.zeros(Hq, 1, dtype=torch.float64)
    idx = torch.nonzero(ok).flatten()
    if idx.numel() == 0:
        return out, tol
    for h in range(Hkv):
        G = Hq // Hkv
        qq, kk, vv = q[h * G:(h + 1) * G], k64[idx, h], v64[idx, h]
        s = qq @ kk.T * scale
        p = torch.softmax(s, dim=-1)
        out[h * G:(h + 1) * G] = p @ vv
        e_s = 2 * max(D / 16, 1) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().T).amax(dim=-1)
        n = idx.numel()
        tol[h * G:(h + 1) * G, 0] = vv.abs().max() * (2 * e_s + w + (n + 64) * 2.0 ** -24)
    return out, tol


def check(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what=""):
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    half = torch.finfo(got.dtype).eps / 2
    # half a step of the output type (of the value before rounding), subnormals included
    bound = tol * (1 + half) + half * ref.abs() + torch.finfo(got.dtype).smallest_normal * half
    bad = (g - ref).abs() > bound
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {float((g - ref).abs().max()):.3e}"
