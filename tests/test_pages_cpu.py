"""The page pool without a GPU: the plain model's invariants, and the calls' refusals on the
host."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from oracle.pages import BOUNDS, OOM, Pool, Refused
from paged_kv_sliding_gb300 import build as pkv_build
from paged_kv_sliding_gb300 import pkv


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def _consistent(pool):
    """refs are what the table says, and a partly filled page belongs to one row."""
    refs = np.zeros_like(pool.refs)
    for r in range(len(pool.lens)):
        used = pool.table[r, : pool.pages(r)]
        assert len(set(used.tolist())) == len(used)
        np.add.at(refs, used, 1)
        if pool.lens[r] % pool.P:
            assert pool.refs[used[-1]] == 1
    assert np.array_equal(refs, pool.refs)


def test_model_keeps_its_invariants():
    rng = np.random.default_rng(0)
    pool = Pool(np.zeros((12, 9)), np.zeros(12), np.zeros(40), 4)
    refused = 0
    for step in range(400):
        try:
            k = rng.integers(4)
            some = rng.permutation(12)[: rng.integers(1, 6)]
            if k == 0:
                pool, slots = pool.extend(some, rng.integers(0, 12, size=len(some)))
                assert len(set(slots)) == len(slots)
            elif k == 1:
                empty = [r for r in some if pool.lens[r] == 0]
                pool, _, _ = pool.fork(rng.integers(0, 12, size=len(empty)), empty)
            elif k == 2:
                pool = pool.free(some.tolist() + some.tolist())  # freed once
                assert pool.bad == 0
            else:
                pool, src, dst = pool.compact()
                assert (pool.refs[: (pool.refs > 0).sum()] > 0).all()
        except Refused as e:
            assert e.code in (OOM, BOUNDS)
            refused += 1
        _consistent(pool)
    assert 0 < refused < 300


def _pool(**over):
    d = pkv.PoolDesc()
    d.table = d.lens = d.refs = d.workspace = d.status = 0x1000
    d.row_stride, d.num_rows, d.num_pages, d.page_size, d.workspace_bytes = 8, 4, 32, 16, 1 << 20
    for k, v in over.items():
        setattr(d, k, v)
    return d


BAD_POOLS = [(dict(num_rows=-1), 1), (dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(row_stride=-1), 1),
             (dict(row_stride=1 << 31), 2), (dict(table=None), 1), (dict(lens=None), 1), (dict(refs=None), 1),
             (dict(status=None), 1), (dict(refs=0x1004), 1), (dict(workspace=None), 1), (dict(workspace_bytes=100), 1),
             (dict(workspace=0x1008), 1), (dict(lens=0x1002), 1)]


@pytest.mark.parametrize("over,status", BAD_POOLS)
def test_bad_pools(lib, over, status):
    d, ok, p = _pool(**over), _pool(), ctypes.c_void_p(0x1000)
    assert lib.pkv_pages_extend(d, p, p, 1, None, 0, None) == status and lib.pkv_last_error()
    assert lib.pkv_pages_fork(d, p, p, 1, p, p, None) == status
    assert lib.pkv_pages_free(d, p, 1, None) == status
    assert lib.pkv_pages_compact(d, ok, p, p, 1, p, None) == status
    assert lib.pkv_pages_compact(ok, d, p, p, 1, p, None) == status


def test_pools_of_about_2_31_rows_or_pages_are_refused(lib):
    """Where a scan's rounded-up segments would pass 32 bits."""
    p = ctypes.c_void_p(0x1000)
    for over in (dict(num_rows=2 ** 31 - 1), dict(num_rows=2 ** 31 - 4096), dict(num_pages=2 ** 31 - 4095)):
        d = _pool(workspace_bytes=1 << 40, **over)
        for n in (1, 4):
            assert lib.pkv_pages_extend(d, p, p, n, None, 0, None) == pkv.PKV_ERR_UNSUPPORTED, over
            assert lib.pkv_pages_fork(d, p, p, n, p, p, None) == pkv.PKV_ERR_UNSUPPORTED
            assert lib.pkv_pages_free(d, p, n, None) == pkv.PKV_ERR_UNSUPPORTED
        assert lib.pkv_pages_compact(d, d, p, p, 1, p, None) == pkv.PKV_ERR_UNSUPPORTED


def test_bad_calls(lib):
    d, p, odd = _pool(), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)
    bad = pkv.PKV_ERR_INVALID_ARG
    for n in (-1, 5):  # more entries than rows
        assert lib.pkv_pages_extend(d, p, p, n, None, 0, None) == bad
        assert lib.pkv_pages_fork(d, p, p, n, p, p, None) == bad
        assert lib.pkv_pages_free(d, p, n, None) == bad
    for a in (None, odd):
        assert lib.pkv_pages_extend(d, a, p, 1, None, 0, None) == bad
        assert lib.pkv_pages_extend(d, p, a, 1, None, 0, None) == bad
        assert lib.pkv_pages_fork(d, a, p, 1, p, p, None) == bad
        assert lib.pkv_pages_fork(d, p, p, 1, a, p, None) == bad
        assert lib.pkv_pages_free(d, a, 1, None) == bad
        assert lib.pkv_pages_compact(d, d, a, p, 1, p, None) == bad
        assert lib.pkv_pages_compact(d, d, p, p, 1, a, None) == bad
    assert lib.pkv_pages_extend(d, p, p, 1, odd, 4, None) == bad
    assert lib.pkv_pages_extend(d, p, p, 1, p, -1, None) == bad
    assert lib.pkv_pages_extend(None, p, p, 1, None, 0, None) == bad
    assert lib.pkv_pages_compact(d, None, p, p, 1, p, None) == bad
    assert lib.pkv_pages_compact(d, d, p, p, -1, p, None) == bad
    for over in (dict(num_rows=5), dict(num_pages=33), dict(page_size=8), dict(row_stride=7), dict(row_stride=9)):
        assert lib.pkv_pages_compact(d, _pool(**over), p, p, 1, p, None) == bad  # (9: one table, two strides)
    assert lib.pkv_pages_extend(d, None, None, 0, None, 0, None) == pkv.PKV_OK  # nothing to do: no launch
    assert lib.pkv_pages_fork(d, None, None, 0, None, None, None) == pkv.PKV_OK
    assert lib.pkv_pages_free(d, None, 0, None) == pkv.PKV_OK


def test_workspace(lib):
    size = ctypes.c_int64()
    assert lib.pkv_pages_workspace(100, 1000, ctypes.byref(size)) == pkv.PKV_OK and size.value >= 4 * 1000 + 16 * 100
    assert lib.pkv_pages_workspace(-1, 1000, ctypes.byref(size)) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_pages_workspace(1, -1, ctypes.byref(size)) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_pages_workspace(1, 1, None) == pkv.PKV_ERR_INVALID_ARG


def test_bad_copies(lib):
    p, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)

    def call(k=p, v=p, layers=1, layer_bytes=1 << 20, pages=8, page_bytes=4096, src=p, dst=p, n=2, count=None, status=None):
        return lib.pkv_copy_pages(k, v, layers, layer_bytes, pages, page_bytes, src, dst, n, count, status, None)

    for over in (dict(n=-1), dict(layers=-1), dict(pages=-1), dict(page_bytes=-16), dict(layer_bytes=-16), dict(k=None),
                 dict(v=None), dict(src=None), dict(dst=None), dict(k=odd), dict(v=odd), dict(src=ctypes.c_void_p(0x1001)),
                 dict(count=ctypes.c_void_p(0x1002)), dict(status=ctypes.c_void_p(0x1002))):
        assert call(**over) == pkv.PKV_ERR_INVALID_ARG, over
    for over in (dict(page_bytes=40), dict(layer_bytes=1000), dict(page_bytes=1 << 31)):
        assert call(**over) == pkv.PKV_ERR_UNSUPPORTED, over
    for over in (dict(n=0), dict(layers=0), dict(page_bytes=0)):
        assert call(**over, k=None) == pkv.PKV_OK, over


def test_pool_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    from tests.test_abi_cpu import HEADER
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    body = "".join(f'printf("%zu ", offsetof(pkv_page_pool, {f}));' for f, _ in pkv.PoolDesc._fields_)
    src = tmp_path / "a.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {' + body +
                   'printf("%zu", sizeof(pkv_page_pool)); return 0;}')
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "a")], check=True)
    got = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()
    want = [getattr(pkv.PoolDesc, f).offset for f, _ in pkv.PoolDesc._fields_] + [ctypes.sizeof(pkv.PoolDesc)]
    assert [int(x) for x in got] == want
