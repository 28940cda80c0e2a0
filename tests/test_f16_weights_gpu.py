"""The plain tensor-core kernels whose softmax weights are f16 (fp16 queries; FP8 pools in the decode):
scores that rise by far more than 2^16 along a sequence, and a first key that takes nearly all of the
weight and has no value of its own. 64-bit references, bounds that follow each weight (range_testlib)."""

import pytest
import torch

from paged_kv_cache_418_b200 import ops
from range_testlib import DT, Cache, attend, check, sees, sink

pytestmark = pytest.mark.gpu

D = 128


def _rising(seed, T, n, Hq, Hkv, qt, span):
    """Scores that rise by `span` (natural units) from the first key to the last."""
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(*s, D, generator=g) for s in ((T, Hq), (n, Hkv), (n, Hkv)))
    q[..., 0] = 8
    k[..., 0] = (torch.arange(n) * (span * D ** 0.5 / 8 / n))[:, None]
    return q.to(DT[qt]), k, v


def _inputs(kind, *args):
    return _rising(*args, 60.0) if kind == "rising" else sink(args[0], args[1], args[2], args[3], args[4], D, 0.99, args[5])


@pytest.mark.parametrize("kernel", ["", "mq"])
@pytest.mark.parametrize("kind", ["rising", "sink"])
@pytest.mark.parametrize("qt,kt,vt,Hq,Hkv,bs", [("f16", "f16", "f16", 8, 2, 16), ("f16", "f16", "f16", 16, 1, 32),
                                                ("f16", "fp8", "f16", 4, 2, 16), ("f16", "f16", "fp8", 2, 2, 32),
                                                ("bf16", "bf16", "bf16", 8, 2, 16)])
def test_prefill(monkeypatch, kernel, kind, qt, kt, vt, Hq, Hkv, bs):
    monkeypatch.setenv("PA_PREFILL_KERNEL", kernel) if kernel else monkeypatch.delenv("PA_PREFILL_KERNEL", raising=False)
    T, n = 70, 1500
    q, k, v = _inputs(kind, bs + Hq, T, n, Hq, Hkv, qt)
    c = Cache([(k, v)], bs, kt, vt)
    qs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if "fp8" in (kt, vt):
        ops.pa_prefill_kv(out, q.cuda(), c.k, c.v, 1.0, 1.0, c.bt, c.cl, qs, T, D ** -0.5, n, err)
    else:
        ops.pa_prefill(out, q.cuda(), c.k, c.v, c.bt, c.cl, qs, T, D ** -0.5, n, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # f16: half a step of the last ones, 2^-25 and twice for the two parts, over the largest weight, 2^10 or more
    rel, floor = (2.0 ** -20, 2.0 ** -34) if qt == "f16" else (2.0 ** -16, 0.0)
    for i in range(T):
        ref, tol = attend(q[i].double(), c.k64[0], c.v64[0], sees(n, n - T + i, 0, 0), D ** -0.5, rel, floor)
        check(out[i], ref, tol, f"token {i}")


@pytest.mark.parametrize("kind", ["rising", "sink"])
@pytest.mark.parametrize("qt,kvt,Hq,Hkv,bs", [("f16", "f16", 32, 4, 16), ("f16", "f16", 16, 4, 32), ("bf16", "fp8", 64, 8, 16),
                                              ("f16", "fp8", 32, 8, 32), ("bf16", "bf16", 32, 4, 16)])
def test_tensor_core_decode(monkeypatch, kind, qt, kvt, Hq, Hkv, bs):
    monkeypatch.setenv("PA_DECODE_KERNEL", "tc")
    # (rising: enough sequences that a CTA's share holds most of one)
    lens = [1500, 40, 4096] if kind == "sink" else [900 + i for i in range(200)]
    data = [_inputs(kind, b + Hq, 1, n, Hq, Hkv, qt) for b, n in enumerate(lens)]
    q = torch.cat([x[0] for x in data])
    c = Cache([(k, v) for _, k, v in data], bs, kvt, kvt)
    out = torch.full(q.shape, float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd, mc = q.cuda(), max(lens)
    ws = ops.workspace_for(qd, c.k, mc)
    if kvt == "fp8":
        ops.pa_decode_fp8(out, qd, c.k, c.v, 1.0, 1.0, c.bt, c.cl, D ** -0.5, mc, 0, ws, err)
    else:
        ops.pa_decode(out, qd, c.k, c.v, c.bt, c.cl, D ** -0.5, mc, 0, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # f16: lo parts 2^11 up, the largest weight 2^7 or more
    rel, floor = (2.0 ** -16, 0.0) if kvt == "bf16" else (2.0 ** -20, 2.0 ** -43)
    for b, n in list(enumerate(lens))[::23 if kind == "rising" else 1]:
        ref, tol = attend(q[b].double(), c.k64[b], c.v64[b], sees(n, n - 1, 0, 0), D ** -0.5, rel, floor)
        check(out[b], ref, tol, f"sequence {b}")


@pytest.mark.parametrize("kind", ["rising", "sink"])
@pytest.mark.parametrize("qt,kt,vt,Hq,Hkv", [("f16", "f16", "f16", 8, 2), ("f16", "fp8", "f16", 16, 2), ("f16", "fp8", "fp8", 32, 4),
                                             ("bf16", "bf16", "bf16", 8, 2)])
def test_shared_prefix_decode(kind, qt, kt, vt, Hq, Hkv):
    """40 groups of three over the same blocks: so many that one CTA walks the whole prefix."""
    bs, pre, tails, groups = 16, 1024, [3, 40, 700], 40
    n0 = pre + max(tails)
    _, k, v = _inputs(kind, Hq, 1, n0, Hq, Hkv, qt)
    q = torch.cat([_inputs(kind, Hq + b, 1, n0, Hq, Hkv, qt)[0] for b in range(3)])
    c = Cache([(k[:pre + t], v[:pre + t]) for t in tails], bs, kt, vt)
    c.bt[:, :pre // bs] = c.bt[:1, :pre // bs].clone()
    dev = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    B = 3 * groups
    bt, cl, qd = c.bt.repeat(groups, 1), c.cl.repeat(groups), q.cuda().repeat(groups, 1, 1)
    shared, offsets, members = dev([pre // bs] * B), dev(range(0, B + 1, 3)), dev(range(B))
    out = torch.full(qd.shape, float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mc = max(c.ctx)
    ws = ops.shared_prefix_workspace_for(qd, c.k, mc, pre // bs)
    if "fp8" in (kt, vt):
        ops.pa_decode_shared_prefix_kv(out, qd, c.k, c.v, 1.0, 1.0, bt, cl, shared, offsets, members, 3, pre // bs,
                                       D ** -0.5, mc, 0, ws, err)
    else:
        ops.pa_decode_shared_prefix(out, qd, c.k, c.v, bt, cl, shared, offsets, members, 3, pre // bs, D ** -0.5, mc,
                                    0, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    rel, floor = (2.0 ** -20, 2.0 ** -34) if qt == "f16" else (2.0 ** -16, 0.0)
    for b in range(3):
        n = c.ctx[b]
        ref, tol = attend(q[b].double(), c.k64[b], c.v64[b], sees(n, n - 1, 0, 0), D ** -0.5, rel, floor)
        for g in (0, groups // 2, groups - 1):
            check(out[3 * g + b], ref, tol, f"sequence {b} of group {g}")


@pytest.mark.parametrize("call", ["prefill", "prefill mq", "decode", "window decode", "window prefill"])
def test_scores_of_millions(monkeypatch, call):
    """Scores near 4e6, where fp32 steps are 1/4 and more, that rise by halves: the weights stay inside f16
    (what remains of the softmax is a matter of rounding; the rows are means of the values all the same)."""
    n, T, Hq, Hkv = 1500, 1 if "decode" in call else 40, 16, 4
    monkeypatch.setenv("PA_DECODE_KERNEL", "tc")
    monkeypatch.setenv("PA_PREFILL_KERNEL", "mq") if call.endswith("mq") else monkeypatch.delenv("PA_PREFILL_KERNEL", raising=False)
    g = torch.Generator().manual_seed(1)
    q, k = torch.zeros(T, Hq, D), torch.zeros(n, Hkv, D)
    q[..., 0], q[..., 1] = 1000, 1
    k[..., 0], k[..., 1] = 4000, (torch.arange(n) * 0.5)[:, None]
    v = torch.rand(n, Hkv, D, generator=g) + 1
    c = Cache([(k, v)], 16, "f16", "f16")
    qd, out = q.half().cuda(), torch.full(q.shape, float("nan"), device="cuda")
    qs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    if call == "window decode":
        ops.pa_decode_window_kv(out, qd, c.k, c.v, 1.0, 1.0, c.bt, c.cl, 1.0, n, 0, n, ops.window_workspace_for(qd, c.k, n, n, 0))
    elif call == "window prefill":
        ops.pa_prefill_window_kv(out, qd, c.k, c.v, 1.0, 1.0, c.bt, c.cl, qs, T, 1.0, n, 0, n)
    elif call == "decode":
        ops.pa_decode(out, qd, c.k, c.v, c.bt, c.cl, 1.0, n, 0, ops.workspace_for(qd, c.k, n))
    else:
        ops.pa_prefill(out, qd, c.k, c.v, c.bt, c.cl, qs, T, 1.0, n)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
    assert float(out.min()) >= 0.99 and float(out.max()) <= 2.01
