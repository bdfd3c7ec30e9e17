"""The binding's calls of gather_kv and of plans over 4-bit caches on streams, without a GPU."""
from __future__ import annotations

import pytest
import torch

from paged_kv_sliding_gb300 import pkv
from tests.test_binding_cpu import _dev, lib, streams  # noqa: F401


def test_results_of_a_gather_on_a_stream_are_its_own_memory(streams):  # noqa: F811
    main, side = streams
    i32 = lambda n: _dev(n, dtype=torch.int32)  # noqa: E731
    for stream, homes in ((side, (side, {main, side})), (None, (main, {main}))):
        for t in pkv.gather_kv(_dev(6, 4, 2, 64), _dev(6, 4, 2, 64), kv_indptr=i32(3), kv_indices=i32(5), out_indptr=i32(3),
                               total=7, stream=stream):
            assert (t.home, t.used) == homes


def test_a_run_over_4_bit_caches_on_a_stream(streams, lib):  # noqa: F811
    main, side = streams
    plan = object.__new__(pkv.Plan)
    plan._lib, plan._handle, plan._kv_torch = pkv._lib, None, torch.uint8
    caches = [_dev(3, 4, 2, 32, dtype=torch.uint8) for _ in range(2)]
    scales = {x: _dev(3, 4, 2, 4, dtype=torch.float8_e4m3fn) for x in ("k_block_scales", "v_block_scales")}
    for t in plan.run(_dev(4, 2, 64), *caches, return_lse=True, stream=side, **scales):
        assert t.home is side and t.used == {main, side}
    name, args = lib.calls[-1]
    assert name == "pkv_run_blocks" and args[-1] == side.cuda_stream


def _plan_of(monkeypatch, **over):
    """A decode plan over 3 pages of 4 tokens, 2 heads of 64, made without a library."""
    monkeypatch.setattr(pkv, "load_library", lambda *a: pkv._lib)
    args = dict(kind="decode", kv_indptr=[0, 1], kv_indices=_dev(1, dtype=torch.int32), kv_last_page_len=[1], num_qo_heads=4,
                num_kv_heads=2, head_dim=64, page_size=4, num_pages=3, kv_dtype="e2m1") | over
    return pkv.Plan(**args)


def _run(plan, shape=(3, 4, 2, 32), v_shape=None):
    caches = [_dev(*s, dtype=torch.uint8) for s in (shape, v_shape or shape)]
    scales = [_dev(*c.shape[:-1], c.shape[-1] // 8, dtype=torch.float8_e4m3fn) for c in caches]
    return plan.run(_dev(1, 4, 64), *caches, k_block_scales=scales[0], v_block_scales=scales[1])


@pytest.mark.parametrize("shape", [(3, 4, 2, 64), (3, 4, 2, 16), (3, 4, 1, 32), (3, 8, 2, 32), (3, 2, 2, 32), (2, 4, 2, 32),
                                   (12, 2, 32), (1, 3, 4, 2, 32)])
def test_a_run_refuses_4_bit_caches_of_another_shape_than_planned(streams, lib, monkeypatch, shape):  # noqa: F811
    """Bytes of an 8-bit cache, other heads, pages or head_dim, too few pages, of K or of V, whose block
    scales fit them."""
    plan = _plan_of(monkeypatch)
    before = len(lib.calls)
    for bad in (dict(shape=shape), dict(v_shape=shape)):
        with pytest.raises(ValueError):
            _run(plan, **bad)
    assert len(lib.calls) == before
    _run(plan)
    _run(plan, (5, 4, 2, 32))  # more pages than the plan names
    assert [name for name, _ in lib.calls[before:]] == ["pkv_run_blocks"] * 2
