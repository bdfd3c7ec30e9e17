"""Calls on a stream other than the current one, while that stream or the current one is busy:
what the binding makes for a call is not memory that is still in use, and is not handed
out again before the call is done with it."""
from __future__ import annotations

import pytest
import torch

from paged_kv_sliding_gb300 import inputs

pytestmark = pytest.mark.gpu

BUSY = 60_000_000  # clock ticks: about 30 ms


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_sliding_gb300 import build, pkv as binding
    build.build()
    binding.load_library()
    return binding


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _fill_all(size, n=64):
    """Tensors of `size` bytes from the current stream's memory, what was just dropped first."""
    return [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(n)]


@pytest.mark.parametrize("how", ["explicit", "current"])
def test_a_pool_dropped_behind_its_call(pkv, how):
    side = torch.cuda.Stream()
    rows, add = _i32(0, 1, 2), _i32(40, 9, 100)
    for call in (lambda p, s: p.extend(rows, add, total=149, stream=s), lambda p, s: p.free(rows, stream=s),
                 lambda p, s: p.compact(stream=s), lambda p, s: p.fork(rows[:1], rows[2:], stream=s)):
        pool = pkv.PagePool.empty(num_rows=4, max_pages=400, num_pages=900, page_size=4)
        sizes = {t.numel() * t.element_size() for t in (pool.table, pool.lens, pool.refs, pool._workspace, pool._status)}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
            got = call(pool, None) if how == "current" else None
        if how == "explicit":
            got = call(pool, side)
        del pool, got
        marks = [m for size in sizes for m in _fill_all(size)]
        side.synchronize()
        assert all((m == 77).all() for m in marks)


def _calls(pkv):
    """Calls that make their results, over inputs that lie ready."""
    w = inputs.tiny_extend().to("cuda")
    plan = pkv.plan_for(w)
    k = torch.randn(64, 4, 64, device="cuda").to(torch.bfloat16)
    s = torch.randn(64, 4, device="cuda")
    pool = pkv.PagePool.empty(num_rows=4, max_pages=40, num_pages=90, page_size=4)
    table = torch.arange(400, dtype=torch.int32, device="cuda").view(4, 100)
    calls = {"run": lambda st: plan.run(w.q, w.k_cache, w.v_cache, return_lse=True, stream=st),
             "append": lambda st: (pkv.norm_rope_append(k, None, q_weight=k[0, 0].contiguous(), stream=st),),
             "merge": lambda st: pkv.merge_state(k, s, k, s, stream=st),
             "indices": lambda st: pkv.build_kv_indices(table, _0123, _0123, _60s, capacity=240, stream=st),
             "extend": lambda st: (pool.extend(_0123[:2], _60s[:2], total=120, stream=st),)}
    _0123, _60s = _i32(0, 1, 2, 3), _i32(60, 60, 60, 60)
    return calls, pool


@pytest.mark.parametrize("name", ["run", "append", "merge", "indices", "extend"])
def test_results_are_not_memory_that_the_current_stream_still_reads(pkv, name):
    calls, _ = _calls(pkv)
    side = torch.cuda.Stream()
    for t in calls[name](None):  # a tensor of each result's size
        size = t.numel() * t.element_size()
        marks = _fill_all(size)
        copies = [torch.empty_like(m) for m in marks]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        for m, c in zip(marks, copies):
            c.copy_(m)
        del marks, m
        got = calls[name](side)  # its inputs lie ready: nothing to wait for
        side.synchronize()
        torch.cuda.synchronize()
        assert all((c == 77).all() for c in copies)
        del got


@pytest.mark.parametrize("name", ["run", "append", "merge", "indices", "extend"])
def test_results_dropped_behind_their_call(pkv, name):
    calls, _ = _calls(pkv)
    side = torch.cuda.Stream()
    sizes = {t.numel() * t.element_size() for t in calls[name](None)}
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    calls[name](side)
    with torch.cuda.stream(side):  # the next tensors of that stream follow the call
        later = [m for size in sizes for m in _fill_all(size)]
    marks = [m for size in sizes for m in _fill_all(size)]
    torch.cuda.synchronize()
    assert all((m == 77).all() for m in marks + later)


def test_results_dropped_while_the_current_stream_reads_them(pkv):
    """Made on the side stream, read on the current one, dropped: not written again by the
    side stream's next call until they are read."""
    calls, _ = _calls(pkv)
    side = torch.cuda.Stream()
    want = [t.clone() for t in calls["run"](None)]
    torch.cuda.synchronize()
    got = calls["run"](side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in got]
    sizes = [t.numel() * t.element_size() for t in got]
    del got
    with torch.cuda.stream(side):
        later = [m for size in sizes for m in _fill_all(size)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, copies)) and all((m == 77).all() for m in later)


def test_a_status_that_was_read_does_not_erase_the_next(pkv):
    """Read and clear, then at once a call on another stream that has something to record."""
    w = inputs.batch_decode(127, batch=8).to("cuda")
    plan = pkv.plan_for(w)
    good, side = plan._kv_indices.clone(), torch.cuda.Stream()
    plan._kv_indices.fill_(10 ** 6)  # no page: recorded, not read
    pool = pkv.PagePool.empty(num_rows=2, max_pages=2, num_pages=2, page_size=4)
    out, lse = torch.empty_like(w.q), torch.empty(w.q.shape[:2], device="cuda")
    nobody = _i32(7)
    torch.cuda.synchronize()
    for _ in range(200):
        assert plan.device_status() in (pkv.PKV_OK, pkv.PKV_ERR_DEVICE_BOUNDS)
        plan.run(w.q, w.k_cache, w.v_cache, out, lse, stream=side)
        assert plan.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
        assert pool.device_status() == pkv.PKV_OK
        pool.free(nobody, stream=side)
        assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
    plan._kv_indices.copy_(good)
    torch.cuda.synchronize()
    assert plan.device_status() == pkv.PKV_OK
    plan.run(w.q, w.k_cache, w.v_cache, out, lse)
    assert plan.device_status() == pkv.PKV_OK


def test_lengths_of_the_page_list_are_read_behind_what_writes_them(pkv):
    """No capacity given: it is read from kv_lens, which the call's stream is about to write."""
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10)
    rows, start, lens, more = _i32(3, 0), _i32(0, 2), _i32(0, 0), _i32(4, 5)
    side = torch.cuda.Stream()
    pkv.build_kv_indices(table, rows, start, lens)  # (kernels loaded on their first use wait for the device)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        lens.copy_(more)
    indptr, indices = pkv.build_kv_indices(table, rows, start, lens, stream=side)
    side.synchronize()
    assert indptr.tolist() == [0, 4, 9] and indices.tolist() == [30, 31, 32, 33, 2, 3, 4, 5, 6]


def test_captured_calls_behind_other_nodes_and_other_streams(pkv):
    """In a graph, each call right behind a memset, a copy and the join of two streams (the
    kernels' early start is meant for a kernel ahead of them alone); replayed over changing
    contents, against the same calls one by one."""
    hkv, d, P, pages = 2, 64, 4, 60
    w = inputs.batch_decode(127, batch=8).to("cuda")
    plan = pkv.plan_for(w, num_sinks=4)
    pool = pkv.PagePool.empty(num_rows=6, max_pages=20, num_pages=pages, page_size=P)
    rows, add, child = _i32(0, 1, 2), _i32(9, 3, 14), _i32(4)
    k = torch.randn(26, hkv, d, device="cuda").to(torch.bfloat16)
    q, fresh = w.q.clone(), w.q.clone()
    caches = [torch.zeros(pages, P, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.zeros(26, dtype=torch.int64, device="cuda")
    src, dst = torch.zeros_like(child), torch.zeros_like(child)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()

    def step():
        now = torch.cuda.current_stream()
        for x in (pool.table, pool.lens, pool.refs):
            x.zero_()
        slots.zero_()  # a memset ahead of the ranking
        pool.extend(rows, add, slots=slots)
        side.wait_stream(now)
        with torch.cuda.stream(side):  # beside the append
            q.copy_(fresh)  # a copy ahead of the attention
            plan.run(q, w.k_cache, w.v_cache, out, lse)
            src.fill_(5)
        pkv.norm_rope_append(None, k, k, slots=slots, k_cache=caches[0], v_cache=caches[1])
        now.wait_stream(side)
        pool.fork(rows[2:], child, src=src, dst=dst)  # behind both streams
        side.wait_stream(now)
        with torch.cuda.stream(side):
            pkv.copy_pages(*caches, src, dst)
        pkv.norm_rope_append(q, None, q_out=q)
        now.wait_stream(side)
        pool.free(rows[:1])

    state = (pool.table, pool.lens, pool.refs, *caches, slots, src, dst, out, lse, q)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(20):
        k.copy_(torch.randn(k.shape, device="cuda"))
        fresh.copy_(torch.randn(q.shape, device="cuda"))
        add.copy_(_i32(*((9, 3, 14), (1, 20, 5), (4, 4, 18))[i % 3]))
        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in state]
        for x in state[3:]:
            x.zero_()
        for c, old in zip(caches, want[3:5]):
            c.copy_(old)
        g.replay()
        torch.cuda.synchronize()
        assert pool.device_status() == plan.device_status() == pkv.PKV_OK
        assert all(torch.equal(x, y) for x, y in zip(state, want)), i
    assert pool.lens.tolist() == [0, 20, 5, 0, 5, 0]
