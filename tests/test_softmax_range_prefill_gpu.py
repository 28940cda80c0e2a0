"""Windowed and block-scaled prefill of rows whose first key takes nearly all of the weight and has
no value of its own, for every type of V pool (bounds: range_testlib)."""

import pytest
import torch

from range_testlib import DT, Cache, attend, check, prefill, sees, sink, spread

pytestmark = pytest.mark.gpu

# Errors of a prefill's weights (fractions of the largest). f16 and 8-bit V pools: f16 weights of which
# the largest is 2^10 or more, so that half a step of the last ones, 2^-25, is 2^-35 of it, and of each
# of two parts; of a weight, two parts are off by 2^-21 and one (8-bit V with bf16 outputs) by 2^-11. bf16 V: two bf16 parts, 2^-17 and no
# floor. ex2: 2^-22.
PREFILL = {"f16": (2.0 ** -20, 2.0 ** -34), "fp8": (2.0 ** -20, 2.0 ** -34), "bf16": (2.0 ** -16, 0.0)}
ONE = (2.0 ** -11 + 2.0 ** -20, 2.0 ** -34)


def _run(q, c, n, T, window, sinks, vt, odt="f32"):
    out = prefill(c, q, [T], 128 ** -0.5, window, sinks, DT[odt])
    for i in range(T):
        ref, tol = attend(q[i].double(), c.k64[0], c.v64[0], sees(n, n - T + i, window, sinks), 128 ** -0.5,
                          *(ONE if vt == "fp8" and odt == "bf16" else PREFILL[vt]))
        check(out[i], ref, tol, f"token {i}")


@pytest.mark.parametrize("n,share,T", [(1000, 0.99, 5), (4096, 0.999, 70)])
@pytest.mark.parametrize("qt,kt,vt,Hq,Hkv", [("f16", "f16", "f16", 8, 1), ("f16", "f16", "f16", 2, 2), ("f16", "fp8", "f16", 4, 1),
                                             ("bf16", "fp8", "fp8", 8, 1), ("f16", "fp8", "fp8", 2, 2),
                                             ("f16", "f16", "fp8", 4, 1), ("bf16", "bf16", "bf16", 8, 1)])
def test_sink_window_prefill(n, share, T, qt, kt, vt, Hq, Hkv):
    q, k, v = sink(n + Hq, T, n, Hq, Hkv, 128, share, qt)
    c = Cache([(k, v)], 16, kt, vt)
    for odt in ("f32", qt):
        _run(q, c, n, T, n // 2 + 3, 1, vt, odt)


@pytest.mark.parametrize("qt,Hq,Hkv,n,share,T", [("f16", 8, 1, 4096, 0.999, 70), ("bf16", 2, 2, 1000, 0.99, 200),
                                                 ("bf16", 8, 1, 131072, 0.99, 3)])
def test_sink_blk8_prefill(qt, Hq, Hkv, n, share, T):
    q, k, v = sink(n + Hq, T, n, Hq, Hkv, 128, share, qt)
    _run(q, Cache([(k, v)], 32, "fp8", "fp8", [torch.zeros(-(-n // 32), Hkv)]), n, T, 0, 0, "fp8", qt)


def test_sink_window_prefill_of_a_long_context():
    n, T = 131072, 3
    q, k, v = sink(3, T, n, 8, 1, 128, 0.999, "f16")
    _run(q, Cache([(k, v)], 32, "f16", "f16"), n, T, n, 0, "f16")


@pytest.mark.parametrize("odt,qt,kt,Hq,Hkv,n,share,T,blk8", [
    ("f32", "f16", "f16", 4, 1, 1000, 0.99, 5, False), ("f16", "f16", "fp8", 2, 2, 4096, 0.999, 70, False),
    ("f32", "f16", "fp8", 8, 1, 1000, 0.5, 300, True), ("f16", "f16", "fp8", 8, 1, 1000, 0.5, 300, True),
    ("f32", "bf16", "fp8", 8, 1, 1000, 0.5, 70, True), ("f32", "bf16", "bf16", 8, 1, 2000, 0.9, 40, False)])
def test_two_parts_over_8_bit_values(odt, qt, kt, Hq, Hkv, n, share, T, blk8):
    """fp32 and f16 outputs: over 8-bit V too the weights enter in two parts."""
    q, k, v = sink(n + T, T, n, Hq, Hkv, 128, share, qt)
    v[0] = torch.randn(Hkv, 128, generator=torch.Generator().manual_seed(1))
    c = Cache([(k, v)], 16, kt, "fp8", [torch.zeros(-(-n // 16), Hkv)] if blk8 else None)
    window, sinks = (0, 0) if blk8 else (n // 2 + 3, 1)
    _run(q, c, n, T, window, sinks, "fp8", odt)


@pytest.mark.parametrize("kind", ["zeros20", "zeros100", "low", "any"])
@pytest.mark.parametrize("lens,new,Hkv,G,qt", [([70], [5], 2, 4, "f16"), ([1070, 300, 1200, 33], [3, 200, 120, 33], 1, 8, "bf16"),
                                               ([1100] * 3, [150, 1, 64], 2, 2, "f16"), ([1100, 64], [300, 64], 3, 1, "bf16")])
def test_blk8_prefill_of_scales_far_apart(kind, lens, new, Hkv, G, qt):
    """Blocks whose contribution is nothing beside others' count in the row sum all the same."""
    q, c = spread(len(lens) + G, lens, Hkv, 128, kind, qt, new, G)
    out = prefill(c, q, new, 128 ** -0.5)
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in list(range(0, m, 7)) + [m - 1]:
            ref, tol = attend(q[at + i].double(), c.k64[b], c.v64[b], sees(n, n - m + i, 0, 0), 128 ** -0.5,
                              *PREFILL["fp8"], vs=c.vs[b])
            check(out[at + i], ref, tol, f"sequence {b}, token {i}")
        at += m
