"""The binding's own work on the host, without a GPU: tensors that report a CUDA device over
host memory, and a library that notes the calls it gets."""
from __future__ import annotations


import pytest
import torch

from paged_kv_sliding_gb300 import pkv


class OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def _dev(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


class Library:
    """Stands in for libpkv: every call succeeds and is noted in `calls`."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return pkv.PKV_OK
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(pkv, "_lib", lib)
    monkeypatch.setattr(pkv, "_append_descs", {})
    monkeypatch.setattr(pkv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


def _append(**over):
    k = _dev(4, 2, 64)
    pkv.norm_rope_append(None, k, k, slots=_dev(4, dtype=torch.int64), k_cache=_dev(3, 4, 2, 64), v_cache=_dev(3, 4, 2, 64),
                         **over)


@pytest.mark.parametrize("name", ["k_scale", "v_scale", "eps", "weight_offset"])
def test_an_append_takes_the_value_that_a_scalar_has_now(lib, name):
    """A scale kept in a tensor of one number and changed in place."""
    x = torch.tensor(0.5)
    for value in (0.5, 2.0, 0.25):
        x.fill_(value)
        _append(**{name: x})
        desc = lib.calls[-1][1][0]
        assert isinstance(desc, pkv.AppendDesc) and getattr(desc, name) == value


def test_an_append_takes_the_truth_that_a_flag_has_now(lib):
    x = torch.tensor(False)
    for value in (False, True, False):
        x.fill_(value)
        _append(interleaved=x)
        assert lib.calls[-1][1][0].interleaved == int(value)


def test_an_append_refuses_what_is_no_number(lib):
    for bad in ("half", None, torch.zeros(2)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            _append(k_scale=bad)
    assert not lib.calls


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(monkeypatch, lib):
    """A main stream (0), the current one, and a side stream (7). Tensors made while the fixture
    stands know the stream whose memory they are (`home`) and the ones they are said to be
    used on (`used`)."""
    main, side = Stream(0), Stream(7)
    now = [main]

    class current:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            now.append(self.stream)

        def __exit__(self, *exc):
            now.pop()

    def made(make):
        def on_device(*args, device=None, **kw):
            t = make(*args, **kw)
            t = t if isinstance(t, OnDevice) else t.as_subclass(OnDevice)
            t.home, t.used = now[-1], {now[-1]}
            return t
        return on_device

    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, made(getattr(torch, name)))
    monkeypatch.setattr(OnDevice, "record_stream", lambda self, s: self.used.add(s), raising=False)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(pkv, "_raw_stream", lambda device: now[-1].cuda_stream)
    return main, side


def _pool():
    return pkv.PagePool.empty(num_rows=4, max_pages=3, num_pages=8, page_size=4)


def _ints(n):
    return torch.zeros(n, dtype=torch.int32)


POOL_CALLS = {"extend": lambda p, s: p.extend(_ints(2), _ints(2), total=0, stream=s),
              "fork": lambda p, s: p.fork(_ints(2), _ints(2), stream=s),
              "free": lambda p, s: p.free(_ints(2), stream=s),
              "compact": lambda p, s: p.compact(stream=s)}


@pytest.mark.parametrize("name", POOL_CALLS)
def test_a_pool_is_recorded_on_the_streams_that_use_it(streams, lib, name):
    """The workspace and status word too, which a caller cannot reach."""
    main, side = streams
    call = POOL_CALLS[name]
    for how in ("explicit", "current"):
        pool = _pool()
        mine = (pool.table, pool.lens, pool.refs, pool._workspace, pool._status)
        assert all(t.home is main for t in mine)
        call(pool, None)
        assert all(t.used == {main} for t in mine)
        if how == "explicit":
            call(pool, side)
        else:
            with torch.cuda.stream(side):
                call(pool, None)
        assert lib.calls[-1][1][-1] == side.cuda_stream
        assert all(t.used == {main, side} for t in mine), how


def test_the_pool_that_a_compaction_writes_is_recorded_too(streams):
    main, side = streams
    pool, out = _pool(), _pool()
    pool.compact(out=out, stream=side)
    for p in (pool, out):
        assert all(side in t.used for t in (p.table, p.lens, p.refs, p._workspace, p._status))


def _plan():
    plan = object.__new__(pkv.Plan)
    plan._lib, plan._handle, plan._kv_torch = pkv._lib, None, torch.bfloat16
    return plan


RESULTS = {
    **POOL_CALLS,
    "append": lambda p, s: pkv.norm_rope_append(_dev(4, 2, 64), None, stream=s),
    "run": lambda p, s: _plan().run(_dev(4, 2, 64), _dev(3, 4, 2, 64), _dev(3, 4, 2, 64), return_lse=True, stream=s),
    "indices": lambda p, s: pkv.build_kv_indices(_ints(8).view(2, 4), _ints(2), _ints(2), _ints(2), capacity=5, stream=s),
    "merge": lambda p, s: pkv.merge_state(_dev(4, 2, 64), _dev(4, 2, dtype=torch.float32), _dev(4, 2, 64),
                                          _dev(4, 2, dtype=torch.float32), stream=s),
}


@pytest.mark.parametrize("name", [n for n in RESULTS if n != "free"])
def test_results_of_a_call_on_a_stream_are_its_own_memory(streams, name):
    """Not memory that the current stream may still be using, and kept for the current stream
    once the caller has dropped it."""
    main, side = streams
    pool = _pool()
    got = RESULTS[name](pool, side)
    for t in got if isinstance(got, tuple) else (got,):
        assert t.home is side and t.used == {main, side}
    got = RESULTS[name](pool, None)
    for t in got if isinstance(got, tuple) else (got,):
        assert t.home is main and t.used == {main}


def test_a_pools_status_is_clear_when_it_has_been_read(streams, monkeypatch):
    """The clearing write is waited for: on its own stream it could erase what a call queued
    next on another stream records."""
    pool = _pool()
    order = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: order.append("wait"))
    monkeypatch.setattr(OnDevice, "item", lambda self: order.append("read") or 5, raising=False)
    monkeypatch.setattr(OnDevice, "zero_", lambda self: order.append("clear") or self, raising=False)
    assert pool.device_status() == 5
    assert order == ["wait", "read", "clear", "wait"]


class OnAnother(OnDevice):
    """A host tensor that says it is on cuda:1, which is not the current device."""

    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def test_a_pools_calls_refuse_memory_of_another_device(streams, lib, monkeypatch):
    pool = _pool()
    with monkeypatch.context() as there:
        there.setattr(torch.cuda, "current_device", lambda: 1)
        zeros = [torch.zeros(*n, dtype=torch.int32).as_subclass(OnAnother) for n in ((4, 3), (4,), (8,))]
        other = pkv.PagePool(*zeros, page_size=4)
    lib.calls.clear()
    slots = torch.zeros(2, dtype=torch.int64).as_subclass(OnAnother)
    for bad in (lambda: pool.extend(_ints(2), _ints(2), slots=slots), lambda: pool.compact(out=other),
                lambda: pool.free(_ints(2).as_subclass(OnAnother)), lambda: other.free(_ints(2))):
        with pytest.raises(ValueError, match="cuda:1|device"):
            bad()
    assert not lib.calls
