"""Host threads that call the windowed and block-scaled decode at the same time, with numbers of KV
heads that take one kernel with different amounts of shared memory."""

import threading

import pytest
import torch

from paged_kv_cache_418_b200 import ops
from range_testlib import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("blk8", [False, True])
def test_threads_with_different_numbers_of_kv_heads(blk8):
    g = torch.Generator().manual_seed(3)
    calls, failed, outs = [], [], []
    for Hkv in (8, 3, 8, 1):
        seqs = [(torch.randn(40, Hkv, 128, generator=g), torch.randn(40, Hkv, 128, generator=g))]
        t = "fp8" if blk8 else "bf16"
        c = Cache(seqs, 16, t, t, [torch.zeros(3, Hkv)] if blk8 else None)
        q = torch.randn(1, Hkv, 128, generator=g).bfloat16().cuda()
        out, ws, stream = torch.zeros_like(q), ops.window_workspace_for(q, c.k, 40, 30, 1), torch.cuda.Stream()
        outs.append(out)

        nb, B, mb = c.k.shape[0], 1, c.bt.shape[1]
        dt = ops.pa_dtype(q)
        # the C entry points with ready arguments: little but the call itself between two calls
        if blk8:
            fn, args = ops.LIB.pa_decode_blk8, (
                out.data_ptr(), dt, q.data_ptr(), dt, c.k.data_ptr(), c.v.data_ptr(), c.ks.data_ptr(), c.vsc.data_ptr(),
                c.bt.data_ptr(), mb, c.cl.data_ptr(), B, Hkv, Hkv, 128, 16, nb, 0.09, 30, 1, 40, ws.data_ptr(), ws.nbytes,
                None, stream.cuda_stream)
        else:
            fn, args = ops.LIB.pa_decode_window_kv, (
                out.data_ptr(), dt, q.data_ptr(), dt, c.k.data_ptr(), dt, 1.0, c.v.data_ptr(), dt, 1.0,
                c.bt.data_ptr(), mb, c.cl.data_ptr(), B, Hkv, Hkv, 128, 16, nb, 0.09, 30, 1, 40, ws.data_ptr(), ws.nbytes,
                None, stream.cuda_stream)

        def call(fn=fn, args=args, keep=(c, q, out, ws, stream)):
            rc = fn(*args)
            if rc:
                raise ops.PAError("decode", rc)
        calls.append(call)
    torch.cuda.synchronize()
    assert len(calls) == 4
    for f in calls:
        f()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    go = threading.Barrier(len(calls))

    def many(f):
        try:
            go.wait()
            for _ in range(10000):
                f()
        except ops.PAError as e:
            failed.append(e)

    threads = [threading.Thread(target=many, args=(f,)) for f in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    for o, x in zip(outs, first):
        assert torch.equal(o, x)
