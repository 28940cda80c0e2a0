"""Cases of the rotary append, the windowed attention and the block-scaled 8-bit attention.

Three operators over the paged cache, each in its plain form and as the library's calls:

* the append of a step's keys and values with the position rotation applied on the way
  (``pa_rope_and_cache_kv``; ``pa_rope_and_cache_blk8`` into pools of E4M3 codes with one
  power-of-two scale per physical block and KV head);
* attention with a sliding window and a few first tokens that stay visible
  (``pa_decode_window_kv`` for single tokens, ``pa_prefill_window_kv`` for chunks);
* attention over the block-scaled 8-bit cache (``pa_decode_blk8``, ``pa_prefill_blk8``).

A case's sequence lengths follow from the case alone (a low-discrepancy spread over its
range), so its work is known; tables and values follow from the seed.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}
_MIN_EXP, _MAX_EXP = -100, 120          # a block scale is 2^e, e in this range


# ---------------------------------------------------------------------------- cases

def listed():
    append = dict(interleaved=False, kv="same")
    return [
        # a decode step of four short fp32 sequences (the repository's tiny workload): latency only
        dict(append, name="append step fp32", op="rope_kv", batch=4, lo=1, hi=33, new_lo=1, new_hi=1,
             hq=4, hkv=4, d=64, bs=16, rot=64, dtype="f32"),
        # eight sequences' 512-token chunks of a GQA model entering a bf16 cache
        dict(append, name="append chunks bf16", op="rope_kv", batch=8, lo=512, hi=2560, new_lo=512,
             new_hi=512, hq=64, hkv=8, d=128, bs=16, rot=128, dtype="bf16"),
        # a decode step of 128 sequences entering the block-scaled 8-bit cache
        dict(append, name="append step blk8", op="rope_blk8", batch=128, lo=16, hi=2048, new_lo=1,
             new_hi=1, hq=64, hkv=8, d=128, bs=16, rot=128, dtype="bf16"),
        # ragged chunks that begin and end inside blocks, half of each head rotated, MHA
        dict(append, name="append chunks blk8", op="rope_blk8", batch=7, lo=400, hi=1500, new_lo=37,
             new_hi=389, hq=32, hkv=32, d=128, bs=16, rot=64, dtype="f16", interleaved=True),
        # the tiny fp32 workload under a window shorter than its contexts
        dict(name="window decode fp32", op="dec_win", batch=4, lo=1, hi=33, hq=4, hkv=4, d=64, bs=16,
             dtype="f32", kv="same", window=16, sinks=4),
        # 64 MHA sequences, most of them longer than the window
        dict(name="window decode MHA fp16", op="dec_win", batch=64, lo=128, hi=2048, hq=32, hkv=32,
             d=128, bs=16, dtype="f16", kv="same", window=1000, sinks=4),
        # long contexts of a GQA model under a 4096-token window
        dict(name="window decode long bf16", op="dec_win", batch=8, lo=20000, hi=32768, hq=64, hkv=8,
             d=128, bs=32, dtype="bf16", kv="same", window=4096, sinks=64),
        # chunked prefill of a GQA model under a window
        dict(name="window prefill chunks", op="pre_win", batch=8, lo=512, hi=2560, new_lo=512,
             new_hi=512, hq=64, hkv=8, d=128, bs=16, dtype="bf16", kv="same", window=1024, sinks=4),
        # a GQA model's decode batch over the block-scaled cache
        dict(name="blk8 decode GQA", op="dec_blk8", batch=128, lo=16, hi=4096, hq=64, hkv=8, d=128,
             bs=16, dtype="bf16", window=0, sinks=0),
        # one sequence with a very long context: all the parallelism is along it
        dict(name="blk8 decode one long", op="dec_blk8", batch=1, lo=100001, hi=100001, hq=32, hkv=8,
             d=128, bs=16, dtype="bf16", window=0, sinks=0),
        # a whole long prompt over the block-scaled cache
        dict(name="blk8 prefill prompt", op="pre_blk8", batch=1, lo=8192, hi=8192, new_lo=8192,
             new_hi=8192, hq=32, hkv=8, d=128, bs=16, dtype="bf16", window=0, sinks=0),
        # small ragged chunks (some of one token), MHA, window over the block-scaled cache
        dict(name="blk8 prefill ragged", op="pre_blk8", batch=5, lo=90, hi=700, new_lo=1, new_hi=77,
             hq=16, hkv=16, d=128, bs=32, dtype="f16", window=333, sinks=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_kv", "rope_blk8", "dec_win", "dec_blk8", "pre_win", "pre_blk8"])
    pre = op in ("pre_win", "pre_blk8")
    d = 128 if pre else rng.choice([64, 128, 128])
    g = rng.choice([1, 2, 4, 8, 16])
    hkv = rng.choice([h for h in (1, 2, 4, 8, 16, 32) if h * g <= 64])
    dtype = rng.choice(["f16", "bf16"] if pre else ["f32", "f16", "bf16"])
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, bs=rng.choice([16, 32]), dtype=dtype)
    if op in ("rope_kv", "rope_blk8"):
        c["batch"] = _log_int(rng, 1, 200)
        c["new_lo"] = 1
        c["new_hi"] = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(2, min(2000, 4000 // c["batch"])))
        c["lo"] = c["new_hi"]
        c["hi"] = c["new_hi"] + _log_int(rng, 1, 3000)
        c["rot"] = rng.choice([16, 32, 48, d // 2, d, d])
        c["interleaved"] = rng.random() < 0.5
        c["kv"] = rng.choice(["same", "same", "fp8"]) if op == "rope_kv" else "same"
        return c
    c["sinks"] = rng.choice([0, 1, 4, 16, rng.randrange(2, 200)])
    if op in ("dec_win", "pre_win"):
        c["window"] = _log_int(rng, 1, 5000)
        c["kv"] = rng.choice(["same", "same", "fp8"])
    elif rng.random() < 0.5:
        c["window"] = c["sinks"] = 0
    else:
        c["window"] = _log_int(rng, 1, 5000)
    per_token = hkv * d * (2 if op in ("dec_blk8", "pre_blk8") else 2 * _ES[dtype])
    if pre:
        c["batch"] = _log_int(rng, 1, 12)
        c["new_lo"] = 1
        c["new_hi"] = _log_int(rng, 1, max(2, min(3000, 5000 // c["batch"])))
        c["lo"] = c["new_hi"]
        c["hi"] = c["new_hi"] + _log_int(rng, 1, 2500)
    else:
        c["batch"] = _log_int(rng, 1, 200)
        most = int(min(100000, 4.0e8 / per_token / c["batch"], 4.0e8 / (c["batch"] * c["hq"])))
        c["hi"] = _log_int(rng, 1, max(2, most))
        c["lo"] = max(1, int(c["hi"] * rng.random()))
    return c


def _spread(n, lo, hi, shift):
    """n whole numbers over [lo, hi]; the first is hi."""
    f = (np.arange(n) * 0.6180339887498949 + shift) % 1.0
    v = lo + np.floor(f * (hi - lo + 1)).astype(np.int64)
    v[0] = hi
    return v


def _lengths(case):
    """(context lengths after the step, new tokens) of each sequence."""
    ctx = _spread(case["batch"], case["lo"], case["hi"], 0.31)
    if "new_hi" not in case:
        return ctx, np.ones_like(ctx)
    return ctx, np.minimum(_spread(case["batch"], case["new_lo"], case["new_hi"], 0.77), ctx)


def _visible(pos, window, sinks):
    """How many keys a query at each position sees."""
    pos = np.asarray(pos, dtype=np.int64)
    if window <= 0:
        return pos + 1
    lo = np.maximum(0, pos + 1 - window)
    return pos + 1 - lo + np.minimum(sinks, lo)


def work(case):
    ctx, new = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    es = _ES[case["dtype"]]
    if case["op"] in ("rope_kv", "rope_blk8"):
        t = int(new.sum())
        code = 1 if case["op"] == "rope_blk8" or case["kv"] == "fp8" else es
        rows = t * d * (2 * hq * es + 2 * hkv * (es + code))
        table = t * case["rot"] * 4 + 16 * t
        return {"bytes": rows + table, "flops": 3.0 * t * (hq + hkv) * case["rot"]}
    window, sinks = case["window"], case["sinks"]
    code = 1 if case["op"].endswith("blk8") or case["kv"] == "fp8" else es
    read = pairs = 0
    for c, n in zip(ctx.tolist(), new.tolist()):
        seen = _visible(np.arange(c - n, c), window, sinks)
        pairs += int(seen.sum())
        # keys some query of the sequence sees: the window of its first query on, and the sinks
        lo = max(0, c - n + 1 - window) if window > 0 else 0
        read += c - lo + min(sinks, lo)
    t = int(new.sum())
    blocks = read / case["bs"] if case["op"].endswith("blk8") else 0
    return {"bytes": read * hkv * d * 2 * code + blocks * hkv * 8 + t * hq * d * 2 * es,
            "flops": 4.0 * pairs * hq * d}


# ---------------------------------------------------------------------------- inputs

def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pow2_scale(amax):
    """Smallest 2^e (e in the allowed range) with amax / 2^e <= 448, exactly."""
    m, e = torch.frexp(amax)                            # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)           # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, _MIN_EXP)).clamp(_MIN_EXP, _MAX_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    rs = np.random.RandomState((int(seed) * 31 + 7) % (1 << 31))
    ctx, new = _lengths(case)
    b, bs, hq, hkv, d = case["batch"], case["bs"], case["hq"], case["hkv"], case["d"]
    dt = _DT[case["dtype"]]
    used = -(-ctx // bs)
    total = int(used.sum())
    nb = total + max(4, total // 16)
    width = int(used.max())
    perm = rs.permutation(nb)
    tables = np.full((b, width), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(used.tolist()):
        tables[i, :n] = perm[at:at + n]
        at += n
    start = np.concatenate([[0], np.cumsum(new)])
    t = int(start[-1])
    seq = np.repeat(np.arange(b), new)
    pos = ctx[seq] - new[seq] + (np.arange(t) - start[:-1][seq])
    slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs

    def on(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(case=case, tables=on(tables), ctx=on(ctx.astype(np.int32)), max_ctx=int(ctx.max()),
             scale=d ** -0.5, positions=on(pos), slots=on(slots), qstart=on(start.astype(np.int32)),
             seq=on(seq), row=on(np.arange(t) - start[:-1][seq]), max_new=int(new.max()),
             k_scale=1.0, v_scale=1.0)
    append = case["op"] in ("rope_kv", "rope_blk8")
    blk8 = case["op"].endswith("blk8")
    shape = (nb, bs, hkv, d)
    # pools: a cache in use (stale blocks and tails hold other requests' old values)
    if blk8:
        for name in ("k", "v"):
            size = torch.exp(0.7 * normal(nb, 1, hkv, 1))           # blocks differ in magnitude
            x = normal(*shape) * size
            sc = _pow2_scale(x.abs().amax(dim=(1, 3)))
            s[name + "_scales"] = sc
            s[name + "_pool"] = _e4m3(x / sc[:, None, :, None]).view(torch.uint8)
            del x
    elif case["kv"] == "fp8":
        s["k_scale"], s["v_scale"] = 0.0625, 0.03125
        for name, sc in (("k", s["k_scale"]), ("v", s["v_scale"])):
            s[name + "_pool"] = _e4m3(normal(*shape) / sc).view(torch.uint8)
    else:
        for name in ("k", "v"):
            s[name + "_pool"] = normal(*shape, dtype=dt)
    if append:
        # one fused projection per token, as a model's QKV product leaves it
        qkv = normal(t, (hq + 2 * hkv), d)
        if blk8:
            qkv *= torch.exp(0.7 * normal(t, 1, 1))
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], dim=1)
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device=dev)
        half = case["rot"] // 2
        angle = (torch.arange(s["max_ctx"], device=dev, dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)[None])
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)
        return s
    s["q"] = normal(t, hq, d).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if case["op"].startswith("dec"):            # the scratch that a server sets aside once
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------- the library's calls

def _run_own(s):
    from paged_kv_cache_418_b200 import ops
    c = s["case"]
    op = c["op"]
    if op == "rope_kv":
        ops.pa_rope_and_cache_kv(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"],
                                 s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["slots"],
                                 interleaved=c["interleaved"])
    elif op == "rope_blk8":
        ops.pa_rope_and_cache_blk8(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"],
                                   s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], s["slots"],
                                   interleaved=c["interleaved"])
    elif op == "dec_win":
        ops.pa_decode_window_kv(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                s["tables"], s["ctx"], s["scale"], c["window"], c["sinks"],
                                s["max_ctx"], s["workspace"])
    elif op == "dec_blk8":
        ops.pa_decode_blk8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                           s["tables"], s["ctx"], s["scale"], s["max_ctx"], c["window"], c["sinks"],
                           s["workspace"])
    elif op == "pre_win":
        ops.pa_prefill_window_kv(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                 s["tables"], s["ctx"], s["qstart"], s["max_new"], s["scale"],
                                 c["window"], c["sinks"], s["max_ctx"])
    else:
        ops.pa_prefill_blk8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                            s["tables"], s["ctx"], s["qstart"], s["max_new"], s["scale"], s["max_ctx"],
                            c["window"], c["sinks"])


# ---------------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, interleaved):
    """Rotate the first 2 * half elements of each head; products and sums in fp32."""
    half = cos.shape[1]
    x = x.float()
    cos, sin = cos[:, None, :], sin[:, None, :]
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        out[..., 0:2 * half:2] = a * cos - b * sin
        out[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        out[..., :half] = a * cos - b * sin
        out[..., half:2 * half] = b * cos + a * sin
    return out


def _append_scaled(pool, scales, rows, slots):
    """Rows into a block-scaled pool: a block written at offset 0 starts anew, any other
    block's scale grows to hold the new rows and its other rows are rounded to it."""
    nb, bs, hkv, d = pool.shape
    block, off = slots // bs, slots % bs
    amax = torch.zeros(nb, hkv, device=pool.device)
    amax.index_reduce_(0, block, rows.abs().amax(dim=2), "amax")
    touched = torch.zeros(nb, dtype=torch.bool, device=pool.device).index_fill_(0, block, True)
    first = torch.zeros(nb, dtype=torch.int32, device=pool.device)
    first.index_add_(0, block, (off == 0).to(torch.int32))
    started = first > 0
    need = _pow2_scale(amax)
    grown = torch.where(started[:, None], need, torch.maximum(scales, need))
    scale = torch.where(touched[:, None], grown, scales)
    ratio = torch.where(touched[:, None] & ~started[:, None], scales / scale, torch.ones_like(scale))
    codes = pool.view(torch.float8_e4m3fn)
    kept = _e4m3(codes.float() * ratio[:, None, :, None])
    kept = kept.view(torch.uint8).view(nb * bs, hkv, d)
    kept[slots] = _e4m3(rows / scale[block][:, :, None]).view(torch.uint8)
    pool.copy_(kept.view(nb, bs, hkv, d))
    scales.copy_(scale)


def _run_append(s):
    c = s["case"]
    half = c["rot"] // 2
    table = s["cos_sin"][s["positions"]]
    cos, sin = table[:, :half], table[:, half:]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["interleaved"]))
    k, v = _rotate(s["k"], cos, sin, c["interleaved"]), s["v"].float()
    if c["op"] == "rope_blk8":
        _append_scaled(s["k_pool"], s["k_scales"], k, s["slots"])
        _append_scaled(s["v_pool"], s["v_scales"], v, s["slots"])
        return
    nb, bs, hkv, d = s["k_pool"].shape
    for_pool = ((s["k_pool"], k, s["k_scale"]), (s["v_pool"], v, s["v_scale"]))
    (kp, kr, ks), (vp, vr, vs) = for_pool
    if c["kv"] == "fp8":
        kr, vr = _e4m3(kr / ks).view(torch.uint8), _e4m3(vr / vs).view(torch.uint8)
    else:
        kr, vr = kr.to(kp.dtype), vr.to(vp.dtype)
    kp.view(nb * bs, hkv, d)[s["slots"]] = kr
    vp.view(nb * bs, hkv, d)[s["slots"]] = vr


def _gather(s, name, at):
    """fp32 rows of the tokens `at` [B, L] of each sequence: [B, L, Hkv, D]."""
    c, pool = s["case"], s[name + "_pool"]
    bs = c["bs"]
    block = torch.gather(s["tables"], 1, at // bs).long().clamp_min(0)
    off = at % bs
    rows = pool[block, off]
    if c["op"].endswith("blk8"):
        return rows.view(torch.float8_e4m3fn).float() * s[name + "_scales"][block][..., None]
    if c["kv"] == "fp8":
        return rows.view(torch.float8_e4m3fn).float() * s[name + "_scale"]
    return rows.float()


def _weights(scores, seen):
    scores = scores.masked_fill(~seen, float("-inf"))
    p = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    return p / p.sum(dim=-1, keepdim=True)


def _run_decode(s):
    c = s["case"]
    window, sinks, n = c["window"], c["sinks"], s["max_ctx"]
    ctx = s["ctx"].long()[:, None]
    if 0 < window and window + sinks < n:
        j = torch.arange(window + sinks, device=ctx.device)[None]
        lo = (ctx - window).clamp_min(0)
        at = torch.where(j < sinks, j, lo + j - sinks)
        seen = torch.where(j < sinks, j < torch.minimum(lo, ctx), at < ctx)
    else:
        at = torch.arange(n, device=ctx.device)[None].expand(c["batch"], n)
        seen = at < ctx
        if window > 0:
            seen = seen & ((at >= ctx - window) | (at < sinks))
    at = torch.minimum(at, (ctx - 1).clamp_min(0))
    b, hkv, d = c["batch"], c["hkv"], c["d"]
    q = s["q"].float().view(b, hkv, c["hq"] // hkv, d)
    k = _gather(s, "k", at).permute(0, 2, 3, 1)                     # [B, Hkv, D, L]
    p = _weights(torch.matmul(q, k) * s["scale"], seen[:, None, None, :])
    del k
    v = _gather(s, "v", at).permute(0, 2, 1, 3)
    s["out"].copy_(torch.matmul(p, v).view(b, c["hq"], d))


def _run_prefill(s):
    c = s["case"]
    window, sinks, n, m = c["window"], c["sinks"], s["max_ctx"], s["max_new"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    ctx = s["ctx"].long()
    new = (s["qstart"][1:] - s["qstart"][:-1]).long()
    at = torch.arange(n, device=ctx.device)[None].expand(b, n)
    pos = (ctx - new)[:, None] + torch.arange(m, device=ctx.device)[None]          # [B, M]
    seen = at[:, None, :] <= pos[:, :, None]
    if window > 0:
        seen = seen & ((at[:, None, :] > pos[:, :, None] - window) | (at[:, None, :] < sinks))
    seen = seen & (at[:, None, :] < ctx[:, None, None])
    at = torch.minimum(at, ctx[:, None] - 1)
    q = torch.zeros(b, m, hq, d, device=ctx.device)
    q[s["seq"], s["row"]] = s["q"].float()
    q = q.view(b, m, hkv, g, d).permute(0, 2, 3, 1, 4)                             # [B, Hkv, G, M, D]
    k = _gather(s, "k", at).permute(0, 2, 3, 1)[:, :, None]                        # [B, Hkv, 1, D, N]
    scores = torch.matmul(q, k) * s["scale"]
    p = _weights(scores, seen[:, None, None])
    v = _gather(s, "v", at).permute(0, 2, 1, 3)[:, :, None]
    out = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)
    s["out"].copy_(out[s["seq"], s["row"]])


def run(state):
    op = state["case"]["op"]
    if own:
        _run_own(state)
    elif op in ("rope_kv", "rope_blk8"):
        _run_append(state)
    elif op in ("dec_win", "dec_blk8"):
        _run_decode(state)
    else:
        _run_prefill(state)
    if op not in ("rope_kv", "rope_blk8"):
        return state["out"]
    k, v = state["k_pool"], state["v_pool"]
    if k.dtype == torch.uint8:                  # codes, as the E4M3 values that they are
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    if op == "rope_blk8":
        return [state["q_out"], k, v, state["k_scales"], state["v_scales"]]
    return [state["q_out"], k, v]


# ---------------------------------------------------------------------------- the definition in 64 bits

def _round_e4m3_64(x):
    """Nearest E4M3 value of each double, ties to even, saturating."""
    e = torch.floor(torch.log2(x.abs().clamp_min(1e-300))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _code_values_64(pool):
    c = torch.arange(256, device=pool.device)
    e, f = ((c >> 3) & 15).double(), (c & 7).double()
    val = torch.where(e > 0, torch.exp2(e - 7.0) * (1.0 + f / 8.0), torch.exp2(e - 6.0) * (f / 8.0))
    val = torch.where(c >= 128, -val, val)
    return val[pool.long()]


def _exact_append(s):
    c = s["case"]
    half = c["rot"] // 2
    cs = s["cos_sin"].double()[s["positions"]]
    unit = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]

    def turn(x):
        x = x.double().clone()
        first = slice(0, 2 * half, 2) if c["interleaved"] else slice(0, half)
        second = slice(1, 2 * half, 2) if c["interleaved"] else slice(half, 2 * half)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = turn(s["q"]), turn(s["k"]), s["v"].double()
    nb, bs, hkv, d = s["k_pool"].shape
    slots = s["slots"]
    out, scales = [q], []
    for name, rows in (("k", k), ("v", v)):
        pool = s[name + "_pool"]
        if c["op"] == "rope_kv":
            held = _code_values_64(pool) if c["kv"] == "fp8" else pool.double()
            if c["kv"] == "fp8":
                rows = _round_e4m3_64(rows / s[name + "_scale"])
            held = held.view(nb * bs, hkv, d).clone()
            held[slots] = rows
            out.append(held.view(nb, bs, hkv, d))
            continue
        held, sc = _code_values_64(pool), s[name + "_scales"].double().clone()
        block = slots // bs
        host = block.cpu().tolist()
        where = {}
        for i, x in enumerate(host):
            where.setdefault(x, []).append(i)
        for x, toks in where.items():
            idx = torch.tensor(toks, device=pool.device)
            rws = rows[idx]
            top = rws.abs().amax(dim=(0, 2)).clamp_min(1e-300)
            # (a quotient that is a power of two must not be lifted by the logarithm's last bit)
            e = torch.ceil(torch.log2(top / 448.0) - 1e-9).clamp(_MIN_EXP, _MAX_EXP)
            new = torch.exp2(e)
            o = slots[idx] % bs
            if not bool((o == 0).any()):
                new = torch.maximum(new, sc[x])
                held[x] = _round_e4m3_64(held[x] * (sc[x] / new)[None, :, None])
            held[x][o] = _round_e4m3_64(rws / new[None, :, None])
            sc[x] = new
        out.append(held)
        scales.append(sc)
    return out + scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope_kv", "rope_blk8"):
        return _exact_append(s)
    ctx, new = _lengths(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["batch"]):
        c, n = int(ctx[b]), int(new[b])
        blocks = s["tables"][b, : -(-c // bs)].long()
        lo = max(0, c - n + 1 - case["window"]) if case["window"] > 0 else 0
        keep = torch.arange(c, device="cuda")
        keep = keep[(keep >= lo) | (keep < case["sinks"])] if case["window"] > 0 else keep
        kv = []
        for name in ("k", "v"):
            pool = s[name + "_pool"][blocks[keep // bs], keep % bs]
            if case["op"].endswith("blk8"):
                x = _code_values_64(pool) * s[name + "_scales"].double()[blocks[keep // bs]][..., None]
            elif case["kv"] == "fp8":
                x = _code_values_64(pool) * s[name + "_scale"]
            else:
                x = pool.double()
            kv.append(x)
        pos = torch.arange(c - n, c, device="cuda")[:, None]
        ok = keep[None] <= pos
        if case["window"] > 0:
            ok &= (keep[None] > pos - case["window"]) | (keep[None] < case["sinks"])
        for h in range(hkv):
            q = s["q"][at:at + n, h * g:(h + 1) * g].double()
            z = torch.einsum("ngd,ld->gnl", q, kv[0][:, h]) * (d ** -0.5)
            z.masked_fill_(~ok[None], float("-inf"))
            p = torch.softmax(z, dim=-1)
            out[at:at + n, h * g:(h + 1) * g] = torch.einsum("gnl,ld->ngd", p, kv[1][:, h])
        at += n
    return out
