"""What the binding of the rotary append, the windowed attention and the block-scaled cache refuses
before the library is called. CPU only."""

import pytest
import torch

from paged_kv_cache_418_b200 import ops

BF, I64, I32 = torch.bfloat16, torch.int64, torch.int32


class Recorder:
    """In place of the library: counts the calls that reach it and takes no pointer."""

    def __init__(self, real):
        self.calls = []
        self.pa_status_string = real.pa_status_string

    def __getattr__(self, name):
        def f(*args):
            self.calls.append((name, args))
            return 0
        return f


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on device 0 (nothing reads it: the library is a Recorder)."""

    def get_device(self):
        return 0


@pytest.fixture
def lib(monkeypatch):
    lib = Recorder(ops.LIB)
    monkeypatch.setattr(ops, "LIB", lib)
    monkeypatch.setattr(ops, "_stream", lambda stream: 0)
    return lib


def _calls():
    """Every entry point with arguments it takes."""
    kc = torch.zeros(4, 16, 2, 128, dtype=BF)
    c8, sc = torch.zeros(4, 16, 2, 128, dtype=torch.uint8), torch.ones(4, 2)
    q, k = torch.zeros(3, 8, 128, dtype=BF), torch.zeros(3, 2, 128, dtype=BF)
    p, cs = torch.zeros(3, dtype=I64), torch.zeros(8, 128)
    bt, cl, qs = torch.zeros(3, 4, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(4, dtype=I32)
    ws, err, pairs = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1, dtype=I32), torch.zeros(1, 2, dtype=I64)
    return {"pa_rope_and_cache_kv": [q, q, k, k, p, cs, kc, kc, 1.0, 1.0, p, False, err],
            "pa_rope_and_cache_blk8": [q, q, k, k, p, cs, c8, c8, sc, sc, p, False, err],
            "pa_copy_scales": [sc, sc, sc, sc, pairs, err],
            "pa_decode_window_kv": [q, q, kc, kc, 1.0, 1.0, bt, cl, 0.1, 5, 0, 64, ws, err],
            "pa_decode_blk8": [q, q, c8, c8, sc, sc, bt, cl, 0.1, 64, 0, 0, ws, err],
            "pa_prefill_window_kv": [q, q, kc, kc, 1.0, 1.0, bt, cl, qs, 1, 0.1, 5, 0, 64, err],
            "pa_prefill_blk8": [q, q, c8, c8, sc, sc, bt, cl, qs, 1, 0.1, 64, 0, 0, err]}


NAMES = sorted(_calls())


def _gpu(args):
    return [x.as_subclass(OnGpu) if isinstance(x, torch.Tensor) else x for x in args]


def _refused(lib, name, args, status=2):
    with pytest.raises(ops.PAError) as e:
        getattr(ops, name)(*args)
    assert e.value.status == status and not lib.calls


@pytest.mark.parametrize("name", NAMES)
def test_taken_on_a_device(lib, name):
    getattr(ops, name)(*_gpu(_calls()[name]))
    assert [c[0] for c in lib.calls] == [name]


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(lib, name):
    """All of them on the host, and each alone beside device tensors."""
    args = _calls()[name]
    _refused(lib, name, args)
    for i, x in enumerate(args):
        if isinstance(x, torch.Tensor):
            one = _gpu(args)
            one[i] = x
            _refused(lib, name, one)


def test_copy_scales_refuses_what_is_no_list_of_pairs(lib):
    args = _gpu(_calls()["pa_copy_scales"])
    for bad in (torch.zeros(3, dtype=I64), torch.zeros(3, 1, dtype=I64), torch.zeros(3, 3, dtype=I64),
                torch.zeros(1, 3, 2, dtype=I64)):
        _refused(lib, "pa_copy_scales", args[:4] + _gpu([bad]))
    for i in range(4):
        one = list(args)
        one[i] = torch.ones(4).as_subclass(OnGpu)
        _refused(lib, "pa_copy_scales", one)
    ops.pa_copy_scales(*args[:4], torch.zeros(0, 2, dtype=I64).as_subclass(OnGpu))
    assert lib.calls[0][1][5] == 0                 # no pairs


@pytest.mark.parametrize("name,places", [("pa_decode_window_kv", (9, 10, 11)), ("pa_decode_blk8", (9, 10, 11)),
                                         ("pa_prefill_window_kv", (9, 11, 12, 13)), ("pa_prefill_blk8", (9, 11, 12, 13))])
def test_lengths_past_32_bits_are_refused(lib, name, places):
    """(2^32 + 5 would be read as 5, 2^32 as 0: every token.)"""
    args = _gpu(_calls()[name])
    for i in places:
        for x in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1):
            one = list(args)
            one[i] = x
            _refused(lib, name, one)
        one = list(args)
        one[i] = 2 ** 31 - 1
        getattr(ops, name)(*one)
        assert 2 ** 31 - 1 in lib.calls.pop()[1]


def test_workspace_of_lengths_past_32_bits_is_refused():
    for args in ((2 ** 32 + 5, 0, 0), (64, 2 ** 32, 0), (64, 5, 2 ** 31)):
        with pytest.raises(ops.PAError):
            ops.pa_window_workspace_size(1, 8, 2, 128, *args)


@pytest.mark.parametrize("name", ["pa_rope_and_cache_kv", "pa_rope_and_cache_blk8"])
def test_one_token_of_an_odd_buffer(lib, name):
    """A single token has no next one: its stride does not count, whatever the buffer behind it is."""
    args = _gpu(_calls()[name])
    rows = torch.zeros(2, 12 * 128 + 3, dtype=BF)            # 1539 elements: no multiple of 16 bytes
    q, k = rows[:, :8 * 128].view(2, 8, 128)[:1], rows[:, 8 * 128:10 * 128].view(2, 2, 128)[:1]
    assert q.stride(0) == 1539
    args[:4] = _gpu([q, q, k, k])
    args[4], args[10] = args[4][:1], args[10][:1]
    getattr(ops, name)(*args)
    strides = lib.calls[0][1][1:8:2]
    assert all(s * 2 % 16 == 0 for s in strides), strides


@pytest.mark.parametrize("name", NAMES)
def test_an_error_flag_holds_32_bits(lib, name):
    args = _gpu(_calls()[name])
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.bool), torch.zeros(1, dtype=torch.int16),
                torch.zeros(0, dtype=I32)):
        _refused(lib, name, args[:-1] + _gpu([bad]))
    getattr(ops, name)(*args[:-1], None)


def test_in_place_rotation_takes_one_stride():
    """Rotated in place with another output stride, one token's result would land on another's input."""
    import test_window_abi as abi
    for fn, base in (("pa_rope_and_cache_kv", abi.ROPE), ("pa_rope_and_cache_blk8", abi.BLK)):
        kw = dict(T=2, q=32, qo=32, qs=1024, qos=2048, nb=0)
        assert abi.call(fn, base, **kw) == 2
        assert abi.call(fn, base, **dict(kw, pos=None)) == 2
        assert abi.call(fn, base, **dict(kw, pos=None, qo=64)) == 1          # (what is refused next)
        assert abi.call(fn, base, **dict(kw, pos=None, qos=1024)) == 1
        assert abi.call(fn, base, **dict(kw, pos=None, T=1)) == 1


def test_workspace_of_a_batch_of_empty_sequences():
    """A bound of 0 tokens is a batch whose rows are all zeros; the decode wants its scratch all the same."""
    n = ops.pa_window_workspace_size
    assert n(3, 8, 2, 128, 0) == n(3, 8, 2, 128, 1) > 0 and n(3, 8, 2, 128, 0, 5, 1) > 0
    assert n(3, 8, 2, 128, -1) == 0 and n(0, 8, 2, 128, 0) == 0
