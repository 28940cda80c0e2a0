"""Softmax weights and block scales over many powers of two, against 64-bit references with bounds
that follow each weight (range_testlib): a first key that takes nearly all of the weight and has
no value of its own, for every type of V pool."""

import pytest
import torch

from range_testlib import Cache, attend, check, decode, sees, sink, spread

pytestmark = pytest.mark.gpu

# Errors of a decode's weights (fractions of the largest): f16 and 8-bit V 2^-22 of a weight and
# 2^-43 of the largest, ex2 2^-22; bf16 V 2^-17 and no floor.
DECODE = {"f16": (2.0 ** -20, 2.0 ** -43), "fp8": (2.0 ** -20, 2.0 ** -43), "bf16": (2.0 ** -16, 0.0)}


@pytest.mark.parametrize("n,share", [(1000, 0.99), (4096, 0.999)])
@pytest.mark.parametrize("qt,kt,vt,D,Hq,Hkv", [("f16", "f16", "f16", 128, 8, 1), ("f16", "f16", "f16", 64, 3, 3),
                                               ("f32", "fp8", "fp8", 128, 16, 8), ("bf16", "bf16", "fp8", 128, 2, 2),
                                               ("f16", "fp8", "f16", 64, 16, 4), ("bf16", "bf16", "bf16", 128, 8, 1)])
def test_sink_window_decode(n, share, qt, kt, vt, D, Hq, Hkv):
    q, k, v = sink(n + D + Hq, 1, n, Hq, Hkv, D, share, qt)
    c = Cache([(k, v)], 16, kt, vt)
    window, sinks = n // 2 + 3, 1
    ref, tol = attend(q[0].double(), c.k64[0], c.v64[0], sees(n, n - 1, window, sinks), D ** -0.5, *DECODE[vt])
    check(decode(c, q, D ** -0.5, window, sinks)[0], ref, tol)


@pytest.mark.parametrize("qt,D,Hq,Hkv,n,share", [("f16", 128, 8, 1, 4096, 0.999), ("bf16", 64, 4, 4, 1000, 0.99),
                                                 ("f32", 128, 16, 8, 1000, 0.9), ("bf16", 128, 8, 1, 131072, 0.99)])
def test_sink_blk8_decode(qt, D, Hq, Hkv, n, share):
    q, k, v = sink(n + D + Hq, 1, n, Hq, Hkv, D, share, qt)
    c = Cache([(k, v)], 32, "fp8", "fp8", [torch.zeros(-(-n // 32), Hkv)])
    ref, tol = attend(q[0].double(), c.k64[0], c.v64[0], sees(n, n - 1, 0, 0), D ** -0.5, *DECODE["fp8"])
    check(decode(c, q, D ** -0.5)[0], ref, tol)


def test_sink_window_decode_of_a_long_context():
    n = 131072
    q, k, v = sink(3, 1, n, 8, 1, 128, 0.999, "f16")
    c = Cache([(k, v)], 32, "f16", "f16")
    ref, tol = attend(q[0].double(), c.k64[0], c.v64[0], sees(n, n - 1, n, 0), 128 ** -0.5, *DECODE["f16"])
    check(decode(c, q, 128 ** -0.5, n, 0)[0], ref, tol)


@pytest.mark.parametrize("kind", ["zeros20", "zeros100", "low", "any"])
@pytest.mark.parametrize("lens,Hkv,D,qt", [([64], 1, 128, "bf16"), ([1070], 8, 128, "f16"), ([3000], 2, 64, "f32"),
                                           ([17, 900, 33, 1] * 60, 3, 64, "bf16"), ([1100, 64] * 90, 8, 128, "bf16")])
def test_blk8_decode_of_scales_far_apart(kind, lens, Hkv, D, qt):
    """Blocks whose contribution is nothing beside others' count in the exp-sum all the same."""
    q, c = spread(len(lens) + D, lens, Hkv, D, kind, qt)
    out = decode(c, q, D ** -0.5)
    for b in sorted(set(range(min(len(lens), 4))) | {len(lens) - 1}):
        ref, tol = attend(q[b].double(), c.k64[b], c.v64[b], sees(lens[b], lens[b] - 1, 0, 0), D ** -0.5,
                          *DECODE["fp8"], vs=c.vs[b])
        check(out[b], ref, tol, f"sequence {b}")
