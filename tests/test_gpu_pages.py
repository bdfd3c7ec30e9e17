"""The page pool's calls against the plain model (oracle/pages.py): whole numbers, so every
array has to be equal, the entries out of use included; page copies bit for bit; and a
serving step in which extend, append, fork, copy, compact and attention with sinks follow
one another."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle.pages import Pool, Refused
from paged_kv_sliding_gb300.inputs import Workload
from tests.test_gpu_sinks import _check as check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_sliding_gb300 import build, pkv as binding
    build.build()
    binding.load_library()
    return binding


def _dev(a, dtype=np.int32):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(a, dtype=dtype)), device="cuda")


def _pair(pkv, rows, cols, pages, P, seed=0):
    """An empty pool on the device, its table full of marks, and its model."""
    table = np.random.default_rng(seed).integers(-9, 10 ** 6, size=(rows, cols))
    return (pkv.PagePool(_dev(table), _dev(np.zeros(rows)), _dev(np.zeros(pages)), page_size=P),
            Pool(table, np.zeros(rows), np.zeros(pages), P))


def _same(pool, model, what=""):
    for name in ("table", "lens", "refs"):
        assert np.array_equal(getattr(pool, name).cpu().numpy(), getattr(model, name)), f"{what}: {name}"


def _both(call, model_call, pool, model, what):
    """Run a call on the device and in the model; the model's next state and outputs."""
    got = call()
    try:
        new, *out = model_call() if isinstance(r := model_call(), tuple) else (r,)
    except Refused as e:
        assert pool.device_status() == e.code, what
        _same(pool, model, what + " (refused)")
        for x in got if isinstance(got, tuple) else (got,):
            assert x is None or (x == -1).all(), what
        return model, None
    assert pool.device_status() == 0, what
    _same(pool, new, what)
    return new, out


@pytest.mark.parametrize("rows,cols,pages,P", [(5, 3, 7, 4), (12, 9, 40, 4), (40, 30, 700, 16), (64, 200, 5000, 1),
                                               (300, 5, 1030, 3)])
def test_random_sequences_match_the_model(pkv, rows, cols, pages, P):
    rng = np.random.default_rng(pages)
    pool, model = _pair(pkv, rows, cols, pages, P)
    refused = 0
    for step in range(60):
        k = rng.integers(8)
        some = rng.permutation(rows)[: rng.integers(1, max(2, rows // 2))]
        what = f"step {step} op {k}"
        if k <= 2:
            add = rng.integers(0, 2 * P + 2, size=len(some))
            slots = torch.empty(int(add.sum()), dtype=torch.int64, device="cuda")
            model, out = _both(lambda: pool.extend(_dev(some), _dev(add), slots=slots),
                               lambda: model.extend(some, add), pool, model, what)
            if out:
                assert slots.cpu().tolist() == out[0], what
        elif k <= 4:
            empty = [r for r in some if model.lens[r] == 0]
            if not empty:
                continue
            parents = rng.integers(0, rows, size=len(empty))
            got = []
            model, out = _both(lambda: got.append(pool.fork(_dev(parents), _dev(empty))) or got[0],
                               lambda: model.fork(parents, empty), pool, model, what)
            if out:
                assert [x.cpu().tolist() for x in got[0]] == out, what
        elif k <= 6:
            model, out = _both(lambda: pool.free(_dev(some)), lambda: model.free(some), pool, model, what)
        else:
            src, dst, count = pool.compact()
            assert pool.device_status() == 0
            model, a, z = model.compact()
            _same(pool, model, what)
            assert count.item() == len(a) and src[: len(a)].cpu().tolist() == a and dst[: len(a)].cpu().tolist() == z
        refused += out is None if k <= 6 else 0
    assert refused < 50


def test_a_large_pool(pkv):
    """300000 pages: every segment of the scan, ids of each in the row."""
    rng = np.random.default_rng(1)
    rows, cols, pages, P = 400, 900, 300000, 16
    pool, model = _pair(pkv, rows, cols, pages, P)
    who, add = rng.permutation(rows), rng.integers(1, cols * P, size=rows)
    model, out = _both(lambda: pool.extend(_dev(who), _dev(add)), lambda: model.extend(who, add), pool, model, "fill")
    drop = who[::3]
    model, _ = _both(lambda: pool.free(_dev(drop)), lambda: model.free(drop), pool, model, "free")
    model, out = _both(lambda: pool.extend(_dev(drop), _dev(add[1::3][: len(drop)].repeat(2)[: len(drop)])),
                       lambda: model.extend(drop, add[1::3][: len(drop)].repeat(2)[: len(drop)]), pool, model, "again")
    model = model.free(who[1::3])
    pool.free(_dev(who[1::3]))
    src, dst, count = pool.compact()
    model, a, z = model.compact()
    assert pool.device_status() == 0 and count.item() == len(a) > 1000
    assert src[: len(a)].cpu().tolist() == a and dst[: len(a)].cpu().tolist() == z
    _same(pool, model, "compact")


@pytest.mark.parametrize("n", [8192, 8193, 10001, 20000])
def test_calls_of_many_entries(pkv, n):
    """More than 32 entries to a warp of the ranking (8192 in all), repeated and refused ones in
    either of a warp's groups and across warps."""
    rng = np.random.default_rng(n)
    rows, cols, P = n + 50, 4, 3
    pool, model = _pair(pkv, rows, cols, 3 * n, P)
    who, add = rng.permutation(rows)[:n], rng.integers(0, 2 * P + 1, size=n)
    per = -(-n // 256)  # entries of a warp

    def extend(who, add, what):
        nonlocal model
        slots = torch.empty(int(np.sum(add)) + 3, dtype=torch.int64, device="cuda")
        model, out = _both(lambda: pool.extend(_dev(who), _dev(add), slots=slots), lambda: model.extend(who, add), pool,
                           model, what)
        assert slots.cpu().tolist() == (out[0] if out else [-1] * int(np.sum(add))) + [-1] * 3, what
        return out

    assert extend(who, add, "extend")
    for i, j in ((per, 2 * per - 1), (per + 1, n - 1), (2 * per - 1, n - 2), (0, 31 % per)):
        twice = who.copy()
        twice[j] = twice[i]
        assert not extend(twice, add, f"entries {i} and {j}")
    for i in (n - 1, 2 * per - 1):
        far = add.copy()
        far[i] = cols * P + 1
        assert not extend(who, far, f"entry {i} beyond its row")
    assert extend(who, np.minimum(add, 1), "again")
    empty, full = np.flatnonzero(model.lens == 0), np.flatnonzero(model.lens)
    model = model.free(full[:: 2])
    pool.free(_dev(full[:: 2]))
    children = np.concatenate([empty, full[:: 2]])
    children = rng.permutation(np.concatenate([children, np.flatnonzero(model.lens)[: max(0, n - len(children))]]))
    extra = [int(r) for r in children if model.lens[r]]
    model = model.free(extra)
    pool.free(_dev(extra))
    parents = rng.integers(0, rows, size=len(children))
    got = []
    for i, j in ((0, len(children) - 1), (33, 40)):
        twice = children.copy()
        twice[j] = twice[i]
        _both(lambda: pool.fork(_dev(parents), _dev(twice)), lambda: model.fork(parents, twice), pool, model, "fork twice")
    model, out = _both(lambda: got.append(pool.fork(_dev(parents), _dev(children))) or got[0],
                       lambda: model.fork(parents, children), pool, model, "fork")
    assert out and [x.cpu().tolist() for x in got[0]] == out


@pytest.mark.parametrize("P", [1, 16, 7, 1000])
def test_slots_of_rows_that_grow_by_many_tokens(pkv, P):
    """Around the tokens that a CTA writes in one pass, from lengths inside a page and at its
    end, and growth within one page."""
    first = np.array([1, P, P + 1, 3 * P - 1, 5, 999, 0, 2 * P, 11], dtype=np.int64)
    add = np.array([1023, 1024, 1025, 5000, 4096, 1, 2049, 3073, 0], dtype=np.int64)
    pool, model = _pair(pkv, len(first), 15000 // P + 4, 40000 // P + 60, P)
    who = np.random.default_rng(P).permutation(len(first))
    for some in (first, add, add[::-1].copy()):
        slots = torch.full((int(some.sum()) + 5,), 77, dtype=torch.int64, device="cuda")
        model, out = _both(lambda: pool.extend(_dev(who), _dev(some), slots=slots), lambda: model.extend(who, some), pool,
                           model, "extend")
        assert out and slots.cpu().tolist() == out[0] + [-1] * 5


def _filled(pkv, P=4):
    pool, model = _pair(pkv, 8, 6, 30, P)
    rows, add = [0, 3, 5, 6], [9, 8, 1, 17]
    pool.extend(_dev(rows), _dev(add))
    return pool, model.extend(rows, add)[0]


@pytest.mark.parametrize("rows,add", [([0, 0], [1, 1]), ([8], [1]), ([-1], [1]), ([0], [-1]), ([0, 3], [1, 17]),
                                      ([1], [25]), ([1, 2, 4, 7], [24, 24, 24, 24]), ([1, 3, 1], [2, 2, 2]),
                                      ([0], [2 ** 31 - 1])])
def test_extend_refuses_and_leaves_the_pool(pkv, rows, add):
    pool, model = _filled(pkv)
    slots = torch.zeros(200, dtype=torch.int64, device="cuda")
    with pytest.raises(Refused):
        model.extend(rows, add)
    _both(lambda: pool.extend(_dev(rows), _dev(add), slots=slots), lambda: model.extend(rows, add), pool, model, "extend")


def test_slots_beyond_their_capacity_are_refused(pkv):
    pool, model = _filled(pkv)
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    _both(lambda: pool.extend(_dev([0, 1]), _dev([2, 3]), slots=slots), lambda: model.extend([0, 1], [2, 3], capacity=4),
          pool, model, "slots")
    slots = torch.full((7,), 77, dtype=torch.int64, device="cuda")
    model, out = _both(lambda: pool.extend(_dev([0, 1]), _dev([2, 3]), slots=slots), lambda: model.extend([0, 1], [2, 3]),
                       pool, model, "room")
    assert slots.cpu().tolist() == out[0] + [-1, -1]  # behind the last one: no slot
    nobody = _dev([])
    pool.extend(nobody, nobody, slots=slots)
    assert (slots == -1).all() and pool.device_status() == 0
    _same(pool, model)


@pytest.mark.parametrize("parents,children", [([0], [3]), ([0, 0], [1, 1]), ([9], [1]), ([0], [-3]), ([0], [0])])
def test_fork_refuses_and_leaves_the_pool(pkv, parents, children):
    pool, model = _filled(pkv)
    _both(lambda: pool.fork(_dev(parents), _dev(children)), lambda: model.fork(parents, children), pool, model, "fork")


def test_fork_without_enough_pages(pkv):
    pool, model = _pair(pkv, 6, 6, 4, 4)
    pool.extend(_dev([0]), _dev([13]))
    model, _ = model.extend([0], [13])
    _both(lambda: pool.fork(_dev([0]), _dev([1])), lambda: model.fork([0], [1]), pool, model, "no page")


def test_a_row_that_is_parent_and_child(pkv):
    """Row 1 is empty: as a parent it gives nothing, though the same call fills it."""
    for parents, children in (([1, 0], [2, 1]), ([0, 1], [1, 2]), ([1], [1])):
        pool, model = _filled(pkv)
        model, out = _both(lambda: pool.fork(_dev(parents), _dev(children)), lambda: model.fork(parents, children), pool,
                           model, "chain")
        assert out and model.lens[2] == 0


@pytest.mark.parametrize("rows", [[0, 0], [3, 8], [-1], [0, 3, 5, 6, 0], [2 ** 31 - 1, 6]])
def test_free_takes_each_row_by_itself(pkv, rows):
    """A row named twice is freed once, one that is none is recorded."""
    pool, model = _filled(pkv)
    pool.free(_dev(rows))
    model = model.free(rows)
    assert pool.device_status() == (pkv.PKV_ERR_DEVICE_BOUNDS if model.bad else 0)
    _same(pool, model, "free")


def test_broken_tables_are_recorded(pkv):
    """Ids out of range, pages nobody counted and lengths that are none: recorded where they
    are met, never followed."""
    for value in (-1, 30, 2 ** 31 - 1, 29):  # 29 is in range but free
        pool, model = _filled(pkv)
        pool.table[0, 1] = value
        model.table[0, 1] = value
        pool.compact()  # packs the rest; the entry stays what it is
        assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
        assert pool.table[0, 1] == value and torch.equal(pool.lens, _dev(model.lens))
        pool, model = _filled(pkv)
        pool.table[0, 1] = value
        model.table[0, 1] = value
        src, dst = pool.fork(_dev([0]), _dev([1]))
        assert pool.device_status() == (0 if value == 29 else pkv.PKV_ERR_DEVICE_BOUNDS)
        assert pool.table[1, 1] == value and src[0] == pool.table[0, 2] and pool.refs[dst[0]] == 1
        pool.free(_dev([1, 3]))
        assert pool.device_status() == (0 if value == 29 else pkv.PKV_ERR_DEVICE_BOUNDS)
        pool.free(_dev([0]))  # here 29 has no count left to give
        assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
        _same(pool, Pool(pool.table.cpu().numpy(), *[getattr(model.free([3, 0]), x) for x in ("lens", "refs")], 4), "rest")
    pool, model = _filled(pkv)
    pool.table[0, 2] = 99  # the page to copy
    src, dst = pool.fork(_dev([0]), _dev([1]))
    assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS and src[0] == dst[0] == -1
    for length in (25, -3):  # more than a row's six pages, and none
        pool, model = _filled(pkv)
        pool.lens[3] = length
        model.lens[3] = length
        pool.free(_dev([3, 6]))
        model = model.free([3, 6])
        assert model.bad == 1 and pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
        _same(pool, model, "length")
        _both(lambda: pool.fork(_dev([3]), _dev([1])), lambda: model.fork([3], [1]), pool, model, "fork")
        _both(lambda: pool.extend(_dev([3]), _dev([0])), lambda: model.extend([3], [0]), pool, model, "extend")


@pytest.mark.parametrize("value", [-1, -2 ** 31, 30, 2 ** 31 - 1])
def test_extend_records_a_last_page_that_is_none(pkv, value):
    """Its tokens have no slot (a negative entry would pass for padding, a large one for a
    slot beyond the caches); those of the row's new pages and of other rows have theirs."""
    pool, model = _filled(pkv)
    pool.table[0, 2] = value  # row 0: 9 tokens, one of them in this page of four
    model, want = model.extend([5, 0, 3], [2, 8, 1])
    slots = torch.full((13,), 77, dtype=torch.int64, device="cuda")
    pool.extend(_dev([5, 0, 3]), _dev([2, 8, 1]), slots=slots)
    assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
    assert slots.cpu().tolist() == want[:2] + [-1] * 3 + want[5:] + [-1] * 2
    model.table[0, 2] = value  # left as it is
    _same(pool, model, "extend")
    pool, _ = _filled(pkv)
    pool.table[3, 1] = value  # a full page: not met
    pool.extend(_dev([0, 3]), _dev([0, 5]), slots=slots)
    assert pool.device_status() == 0 and (slots[:5] >= 0).all()
    pool.table[0, 2] = value
    pool.extend(_dev([0]), _dev([0]), slots=slots)  # no token, nothing met
    assert pool.device_status() == 0 and (slots == -1).all()


def test_compact_out_of_place_and_without_room(pkv):
    pool, model = _filled(pkv)
    pool.free(_dev([0, 5]))
    model = model.free([0, 5])
    before = [x.clone() for x in (pool.table, pool.lens, pool.refs)]
    out = pkv.PagePool(torch.full((8, 7), 55, dtype=torch.int32, device="cuda"), _dev(np.full(8, 9)), _dev(np.full(30, 9)),
                       page_size=4)
    new, a, z = model.compact()
    assert len(a) >= 2
    small = torch.full((len(a) - 1,), -5, dtype=torch.int32, device="cuda")
    src, dst, count = pool.compact(src=small, dst=small.clone())
    assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS and count.item() == 0
    _same(pool, model, "no room")
    src, dst, count = pool.compact(out=out)
    assert pool.device_status() == out.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(before, (pool.table, pool.lens, pool.refs)))
    assert count.item() == len(a) and src[: len(a)].cpu().tolist() == a and dst[: len(a)].cpu().tolist() == z
    assert np.array_equal(out.refs.cpu().numpy(), new.refs) and np.array_equal(out.lens.cpu().numpy(), new.lens)
    for r in range(8):
        k = new.pages(r)
        assert out.table[r, :k].cpu().tolist() == new.table[r, :k].tolist() and (out.table[r, k:] == 55).all()
    out2 = pool.compact(src=small[:0], dst=small[:0].clone())  # in place, no room at all
    assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS and out2[2].item() == 0


@pytest.mark.parametrize("length", [25, -3])
def test_compact_out_of_place_hands_on_a_length_that_is_none(pkv, length):
    """More than a row's six pages, and a negative one: recorded, and in the new pool what it
    was in the old, not what that memory held."""
    pool, model = _filled(pkv)
    pool.lens[3] = length
    out = pkv.PagePool(torch.full((8, 7), 55, dtype=torch.int32, device="cuda"), _dev(np.full(8, 1)), _dev(np.full(30, 9)),
                       page_size=4)
    pool.compact(out=out)
    assert pool.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS
    assert torch.equal(out.lens, pool.lens) and (out.table[3] == 55).all() and torch.equal(out.refs, pool.refs)
    out.free(_dev([3]))
    assert out.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS


def test_compact_of_full_and_empty_pools(pkv):
    for rows, add in (([], []), ([0, 1, 2, 3, 4], [24, 24, 24, 24, 24])):
        pool, model = _pair(pkv, 8, 6, 30, 4)
        pool.extend(_dev(rows), _dev(add))
        model = model.extend(rows, add)[0]
        _, _, count = pool.compact()
        assert pool.device_status() == 0 and count.item() == 0
        _same(pool, model)
    pool, _ = _pair(pkv, 4, 2, 0, 4)  # no pages at all
    assert pool.compact()[2].item() == 0 and pool.device_status() == 0
    pool.extend(_dev([0]), _dev([1]))
    assert pool.device_status() == pkv.PKV_ERR_OOM
    pool.extend(_dev([0]), _dev([0]))
    assert pool.device_status() == 0


@pytest.mark.parametrize("shape,dtype", [((50, 16, 8, 128), torch.bfloat16), ((50, 1, 1, 16), torch.uint8),
                                         ((50, 5, 3, 64), torch.float8_e4m3fn), ((3, 40, 7, 2, 64), torch.bfloat16),
                                         ((2, 33, 1, 1, 8), torch.bfloat16), ((1, 9, 512, 8, 128), torch.float32)])
def test_copies(pkv, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(0)
    raw = [torch.randint(0, 256, shape[:-1] + (shape[-1] * dtype.itemsize,), generator=g, device="cuda", dtype=torch.uint8)
           for _ in range(2)]
    k, v = (x.view(dtype) for x in raw)
    pages = shape[-4]
    ids = np.random.default_rng(3).permutation(pages)
    n = pages // 2
    for count in (None, 0, 1, n - 2, n + 9, -4):
        src, dst = ids[:n].copy(), ids[n: 2 * n].copy()
        src[1], dst[2] = -1, -7  # skipped
        want = [x.clone() for x in raw]
        for x in want:
            for a, z in list(zip(src, dst))[: n if count is None else max(0, count)]:
                if a >= 0 and z >= 0:
                    x.view((-1,) + shape[-4:-1] + (x.shape[-1],))[:, z] = x.view((-1,) + shape[-4:-1] + (x.shape[-1],))[:, a]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.copy_pages(k, v, _dev(src), _dev(dst), count=None if count is None else _dev([count]), status=status)
        torch.cuda.synchronize()
        assert status.item() == 0 and all(torch.equal(x, y) for x, y in zip(raw, want)), count


def test_copies_record_ids_beyond_the_caches(pkv):
    k = torch.arange(8, device="cuda", dtype=torch.float32).view(8, 1, 1, 1).expand(8, 4, 1, 64).contiguous()
    v = k.clone() + 100
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for st in (status, None):
        pkv.copy_pages(k, v, _dev([0, 8, 1]), _dev([5, 6, 2 ** 31 - 1]), status=st)
    torch.cuda.synchronize()
    assert status.item() == pkv.PKV_ERR_DEVICE_BOUNDS
    assert k[:, 0, 0, 0].tolist() == [0, 1, 2, 3, 4, 0, 6, 7] and v[:, 0, 0, 0].tolist() == [100, 101, 102, 103, 104, 100, 106, 107]


def test_copies_beyond_32_bit_offsets(pkv):
    pages = 5000  # of 1 MiB: 4.9 GiB a cache
    k = torch.zeros(pages, 512, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[4321], v[4321] = 3.0, 4.0
    pkv.copy_pages(k, v, _dev([4321, 0]), _dev([4999, 4998]))
    assert (k[4999] == 3).all() and (v[4999] == 4).all() and not k[4997].any() and not k[4998].any()


def test_captured_and_replayed(pkv):
    """free, extend, fork and copy in one graph, replayed over changing contents."""
    pool, model = _pair(pkv, 16, 12, 120, 8)
    k = torch.randn(120, 8, 1, 64, device="cuda").to(torch.bfloat16)
    v = k.clone()
    rows, add, parents, children = (_dev(x) for x in ([0, 1, 2, 3], [20, 7, 0, 33], [0, 3, 3], [8, 9, 10]))
    slots = torch.zeros(120, dtype=torch.int64, device="cuda")  # 114 tokens at most
    src, dst = torch.zeros_like(parents), torch.zeros_like(parents)

    def step():
        pool.free(children)
        pool.free(rows)
        pool.extend(rows, add, slots=slots)
        pool.fork(parents, children, src=src, dst=dst)
        pkv.copy_pages(k, v, src, dst)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for x in (pool.table, pool.lens, pool.refs):
        x.zero_()
    model = Pool(np.zeros((16, 12)), np.zeros(16), np.zeros(120), 8)
    other, _ = model.extend([11, 12], [50, 9])
    pool.extend(_dev([11, 12]), _dev([50, 9]))
    model = other
    for more in ([20, 7, 0, 33], [1, 2, 3, 4], [90, 8, 16, 0]):
        add.copy_(_dev(more))
        g.replay()
        model = model.free(children.tolist()).free(rows.tolist())
        model, want = model.extend(rows.tolist(), more)
        model, a, z = model.fork(parents.tolist(), children.tolist())
        assert pool.device_status() == 0
        _same(pool, model, str(more))
        assert slots.cpu().tolist() == want + [-1] * (120 - len(want)) and src.cpu().tolist() == a and dst.cpu().tolist() == z
        for x, y in zip(a, z):
            assert x < 0 or (torch.equal(k[x], k[y]) and torch.equal(v[x], v[y]))


def test_another_stream(pkv):
    """The calls of a step on a side stream, their outputs allocated by the binding."""
    pool, model = _pair(pkv, 16, 12, 120, 8)
    k = torch.randn(120, 8, 1, 64, device="cuda").to(torch.bfloat16)
    v = k.clone()
    rows, add, parents, children = (_dev(x) for x in ([0, 1, 2], [20, 7, 33], [0, 2], [8, 9]))
    q = torch.randn(60, 2, 64, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots = pool.extend(rows, add, total=60, stream=side)
    pkv.norm_rope_append(q, q[:, :1], q[:, 1:], slots=slots, k_cache=k, v_cache=v, stream=side)
    src, dst = pool.fork(parents, children, stream=side)
    pkv.copy_pages(k, v, src, dst, stream=side)
    pool.free(rows, stream=side)
    moves = pool.compact(stream=side)
    pkv.copy_pages(k, v, *moves[:2], count=moves[2], stream=side)
    side.synchronize()
    model, want = model.extend([0, 1, 2], [20, 7, 33])
    model, a, z = model.fork([0, 2], [8, 9])
    assert slots.cpu().tolist() == want and src.cpu().tolist() == a and dst.cpu().tolist() == z
    model, a, z = model.free([0, 1, 2]).compact()
    assert pool.device_status() == 0 and moves[2].item() == len(a)
    _same(pool, model)
    for row, first in ((8, 0), (9, 27)):  # the forks hold their parents' tokens
        n = int(model.lens[row])
        at = [int(model.table[row, t // 8]) * 8 + t % 8 for t in range(n)]
        assert torch.equal(k.view(-1, 1, 64)[at], q[first: first + n, :1])
        assert torch.equal(v.view(-1, 1, 64)[at], q[first: first + n, 1:])


def test_refusals_of_the_binding(pkv):
    pool, _ = _pair(pkv, 4, 3, 10, 4)
    i = _dev([0, 1])
    for bad in (lambda: pool.extend(i, i.long()), lambda: pool.extend(i, i[:1]), lambda: pool.fork(i.cpu(), i),
                lambda: pool.free(_dev([0, 1, 2, 3])[::2]), lambda: pool.extend(i, i, slots=i),
                lambda: pool.fork(i, i, src=i[:1]), lambda: pkv.PagePool(pool.table, pool.lens[:3], pool.refs, page_size=4),
                lambda: pkv.PagePool(pool.table.long(), pool.lens, pool.refs, page_size=4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkv.PkvError):
        pkv.PagePool(pool.table, pool.lens, pool.refs, page_size=0).free(i)
    with pytest.raises(pkv.PkvError):
        pool.free(_dev([0, 1, 2, 3, 0]))  # more entries than rows
    k = torch.zeros(10, 4, 1, 64, device="cuda")
    for bad in (lambda: pkv.copy_pages(k, k[:9], i, i), lambda: pkv.copy_pages(k, k.half(), i, i),
                lambda: pkv.copy_pages(k, k, i, i[:1]), lambda: pkv.copy_pages(k[:, ::2], k[:, ::2], i, i),
                lambda: pkv.copy_pages(k.cpu(), k.cpu(), i, i), lambda: pkv.copy_pages(k, k, i.long(), i.long())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkv.PkvError):  # pages of 4 bytes
        pkv.copy_pages(k[:, :1, :, :1].contiguous(), k[:, :1, :, :1].contiguous(), i, i)


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [16, 5])
def test_a_serving_step_end_to_end(pkv, oracle_lib, P, kv_type):
    """Prompts go into fresh pages, rows fork and diverge by a token each, one request ends,
    the pool is compacted; after every stage a windowed decode with sinks over the pool's
    own table is the oracle's, and compaction changes no bit of it."""
    hq, hkv, d, W, sinks, rows, cols, pages = 8, 2, 64, 40, 6, 8, 40, 200
    dtype = torch.bfloat16 if kv_type == "bf16" else torch.float8_e4m3fn
    scale = 1.0 if kv_type == "bf16" else 0.125
    k_cache, v_cache = (torch.zeros(pages, P, hkv, d, device="cuda").to(dtype) for _ in range(2))
    pool = pkv.PagePool.empty(num_rows=rows, max_pages=cols, num_pages=pages, page_size=P)
    a = torch.arange(400, dtype=torch.float64, device="cuda")[:, None] * 100.0 ** (-torch.arange(0, d, 2, device="cuda") / d)[None]
    table = torch.cat([a.cos(), a.sin()], 1).float()
    wq, wk = (torch.rand(d, device="cuda").to(torch.bfloat16) + 0.5 for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(P)

    def append(which, counts):
        start = pool.lens[_dev(which).long()].cpu().numpy()
        slots = pool.extend(_dev(which), _dev(counts), total=int(np.sum(counts)))
        pos = np.concatenate([s + np.arange(c) for s, c in zip(start, counts)])
        n = len(pos)
        qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.view(n, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
        return pkv.norm_rope_append(q, k, v, positions=_dev(pos), cos_sin=table, slots=slots, k_cache=k_cache,
                                    v_cache=v_cache, q_weight=wq, k_weight=wk, k_scale=scale, v_scale=scale)

    def decode(which, q):
        lens = pool.lens[_dev(which).long()]
        n_pages = (lens + P - 1) // P
        indptr, indices = pkv.build_kv_indices(pool.table, _dev(which), _dev(np.zeros(len(which))), n_pages.int())
        host, last = indptr.cpu().numpy(), (lens - (n_pages - 1) * P).cpu().numpy()
        plan = pkv.Plan(kind="decode", kv_indptr=host, kv_indices=indices, kv_last_page_len=last, num_qo_heads=hq,
                        num_kv_heads=hkv, head_dim=d, page_size=P, num_pages=pages, window_left=W, num_sinks=sinks,
                        k_scale=scale, v_scale=scale, kv_dtype=kv_type)
        out, lse = plan.run(q, k_cache, v_cache, return_lse=True)
        assert plan.device_status() == pool.device_status() == 0
        w = Workload(name="step", kind="decode", qo_indptr=np.arange(len(which) + 1, dtype=np.int32), kv_indptr=host,
                     kv_indices=indices.cpu().numpy()[: host[-1]], kv_last_page_len=last.astype(np.int32),
                     num_qo_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, num_pages=pages, window_left=W,
                     causal=True, sm_scale=d ** -0.5, q=q.cpu(), k_cache=k_cache.cpu(), v_cache=v_cache.cpu())
        check_attention(oracle_lib, w, out, lse, sinks, f"rows {which}", k_scale=scale, v_scale=scale)
        return out, lse

    prompts = [0, 1, 2]
    append(prompts, [100, 33, 3])
    q = append(prompts, [1, 1, 1])
    decode(prompts, q)
    src, dst = pool.fork(_dev([0, 0, 1]), _dev([4, 5, 6]))
    pkv.copy_pages(k_cache, v_cache, src, dst)
    everyone = [0, 1, 2, 4, 5, 6]
    q = append(everyone, [1] * 6)  # the forks diverge here
    out, _ = decode(everyone, q)
    assert not torch.equal(out[0], out[3])
    q = append([0, 4, 5], [30, 17, 1])[-1:]
    pool.free(_dev([1, 0]))
    rest = [2, 4, 5, 6]
    q = append(rest, [1] * 4)
    before = decode(rest, q)
    src, dst, count = pool.compact()
    pkv.copy_pages(k_cache, v_cache, src, dst, count=count)
    live = int((pool.refs > 0).sum())
    assert count.item() > 0 and (pool.refs[:live] > 0).all()
    k_cache[live:], v_cache[live:] = torch.zeros((), device="cuda").to(dtype), torch.zeros((), device="cuda").to(dtype)
    after = decode(rest, q)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    decode(rest, append(rest, [1] * 4))


def test_a_captured_step_replayed(pkv, oracle_lib):
    """One decode step in one graph: a token for every row, its key and value appended, the
    page table rebuilt, and attention under a window with sinks; replayed step after step
    with only the inputs, the positions and the plan's lengths renewed."""
    hq, hkv, d, P, W, sinks, B, pages = 8, 2, 128, 16, 30, 5, 12, 400
    rng = np.random.default_rng(6)
    k_cache, v_cache = (torch.randn(pages, P, hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    pool = pkv.PagePool.empty(num_rows=20, max_pages=30, num_pages=pages, page_size=P)
    rows = _dev(rng.permutation(20)[:B])
    start = rng.integers(1, 120, size=B)
    pool.extend(rows, _dev(start))
    a = torch.arange(400, dtype=torch.float64, device="cuda")[:, None] * 50.0 ** (-torch.arange(0, d, 2, device="cuda") / d)[None]
    table = torch.cat([a.cos(), a.sin()], 1).float()
    weight = (torch.rand(d, device="cuda") + 0.5).to(torch.bfloat16)
    qkv = torch.zeros(B + 3, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device="cuda")  # three padding rows
    q, k, v = (x.view(B + 3, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    positions, slots = torch.zeros(B + 3, dtype=torch.int32, device="cuda"), torch.zeros(B + 3, dtype=torch.int64, device="cuda")
    ones, zeros = torch.ones_like(rows), torch.zeros_like(rows)
    q_out = torch.full((B + 3, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, hq, device="cuda")
    kv_indptr, kv_indices = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(360, dtype=torch.int32, device="cuda")
    long_rows = rows.long()

    def host_lens(lens):
        n = -(-lens // P)
        return dict(kv_indptr=np.concatenate([[0], np.cumsum(n)]), kv_last_page_len=lens - (n - 1) * P)

    plan = pkv.Plan(kind="decode", **host_lens(start + 1), kv_indices=kv_indices, num_qo_heads=hq, num_kv_heads=hkv,
                    head_dim=d, page_size=P, num_pages=pages, window_left=W, num_sinks=sinks, capacity={"max_batch": B})

    def step():
        pool.extend(rows, ones, slots=slots)
        pkv.norm_rope_append(q, k, v, positions=positions, cos_sin=table, slots=slots, k_cache=k_cache, v_cache=v_cache,
                             q_weight=weight, k_weight=weight, q_out=q_out)
        pkv.build_kv_indices(pool.table, rows, zeros, (pool.lens[long_rows] + P - 1) // P, kv_indptr=kv_indptr,
                             kv_indices=kv_indices)
        plan.run(q_out[:B], k_cache, v_cache, out, lse)

    def renew(lens):
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        positions[:B] = _dev(lens)
        plan.update(**host_lens(lens + 1))

    def check(lens, what):
        torch.cuda.synchronize()
        assert plan.device_status() == pool.device_status() == 0
        assert (q_out[B:] == 7.0).all() and slots[B:].tolist() == [-1] * 3 and pool.lens[long_rows].tolist() == (lens + 1).tolist()
        at = host_lens(lens + 1)
        n = int(at["kv_indptr"][-1])
        assert torch.equal(k_cache.view(-1, hkv, d)[slots[:B]], pkv.norm_rope_append(
            k[:B].contiguous(), None, positions=positions[:B], cos_sin=table, q_weight=weight))
        w = Workload(name=what, kind="decode", qo_indptr=np.arange(B + 1, dtype=np.int32),
                     kv_indptr=at["kv_indptr"].astype(np.int32), kv_indices=kv_indices.cpu().numpy()[:n],
                     kv_last_page_len=at["kv_last_page_len"].astype(np.int32), num_qo_heads=hq, num_kv_heads=hkv, head_dim=d,
                     page_size=P, num_pages=pages, window_left=W, causal=True, sm_scale=d ** -0.5, q=q_out[:B].cpu(),
                     k_cache=k_cache.cpu(), v_cache=v_cache.cpu())
        check_attention(oracle_lib, w, out, lse, sinks, what)

    lens = start.copy()
    renew(lens)
    step()
    check(lens, "first")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(20):
        lens = lens + 1
        renew(lens)
        g.replay()
        if i % 5 == 4:
            check(lens, f"replay {i}")
