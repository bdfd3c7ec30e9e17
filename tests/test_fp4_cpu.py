"""The float64 reference of 4-bit caches pinned by closed forms and torch's E4M3, and the host
checks of the calls that take them."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import fp4
from paged_kv_sliding_gb300 import build as pkv_build
from paged_kv_sliding_gb300 import pkv
from tests.test_abi_cpu import HEADER
from tests.test_binding_cpu import _dev
from tests.test_binding_cpu import lib as fake_lib  # noqa: F401


def test_e4m3_table_is_torchs():
    want = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp4.E4M3, want, equal_nan=True)
    x = np.concatenate([np.linspace(0, 449, 20001), fp4.E4M3[:127], (fp4.E4M3[1:127] + fp4.E4M3[:126]) / 2])
    got = fp4.scale_codes(x)
    assert np.array_equal(got, torch.tensor(x).clamp(max=448).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_halfway_values_go_to_even_codes():
    assert fp4.value_codes([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0]).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    assert fp4.value_codes([-0.25, -0.75, -5.0, -9.0]).tolist() == [8, 10, 14, 15]


def test_pack_and_unpack():
    c = np.random.default_rng(0).integers(0, 16, size=(3, 64)).astype(np.uint8)
    assert np.array_equal(fp4.unpack(fp4.pack(c)), c)
    assert fp4.pack(np.array([1, 2], dtype=np.uint8)).tolist() == [0x21]


def test_quantised_rows_are_near_and_exact_rows_stay():
    y = np.random.default_rng(1).standard_normal((5, 128))
    data, s = fp4.quantise(y, t=0.5)
    back = 0.5 * fp4.values(data, s)
    top = np.repeat(np.abs(y.reshape(5, 8, 16)).max(-1), 16, -1)
    assert (np.abs(back - y) <= top * (1 / 6 + 1 / 16)).all()  # half the widest step, and the scale's rounding
    again, s2 = fp4.quantise(back, t=0.5)
    keep = np.repeat(np.abs(fp4.values(data, np.full_like(s, 0x38))).reshape(5, 8, 16).max(-1) == 6, 16, -1)
    assert np.array_equal(fp4.values(again, s2)[keep], fp4.values(data, s)[keep])


def test_zero_rows():
    data, s = fp4.quantise(np.zeros((2, 64)))
    assert not data.any() and not s.any()


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def _append(lib, null=(), blocks=True, pointers=None, **over):
    d = pkv.AppendDesc()
    d.num_tokens, d.q_stride, d.k_stride, d.v_stride = 4, 512, 256, 256
    d.num_qo_heads, d.num_kv_heads, d.head_dim, d.page_size, d.num_pages = 4, 2, 128, 16, 8
    d.kv_dtype, d.rotary_dim, d.max_position = pkv.PKV_FP4_E2M1, 128, 100
    d.eps, d.k_scale, d.v_scale = 1e-6, 1.0, 1.0
    for k, v in over.items():
        setattr(d, k, v)
    names = ("q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions", "slots", "q_out", "k_out", "k_cache",
             "v_cache") + (("k_block_scales", "v_block_scales") if blocks else ()) + ("status",)
    args = [None if n in null else ctypes.c_void_p((pointers or {}).get(n, 0x1000)) for n in names]
    return (lib.pkv_norm_rope_append_blocks if blocks else lib.pkv_norm_rope_append)(ctypes.byref(d), *args, None)


def test_append_refusals(lib):
    bad = pkv.PKV_ERR_INVALID_ARG
    assert _append(lib, blocks=False) == bad  # a 4-bit cache without its scales
    assert _append(lib, null=("k_block_scales",)) == bad
    assert _append(lib, null=("v_block_scales",)) == bad
    assert _append(lib, kv_dtype=pkv.PKV_FP8_E4M3) == bad  # scales without a 4-bit cache
    assert _append(lib, pointers={"k_block_scales": 0x1004}) == bad
    assert _append(lib, kv_dtype=6) == bad and _append(lib, rotary_dim=136) == bad
    assert _append(lib, num_tokens=0) == pkv.PKV_OK


def _gather(lib, null=(), pointers=None, desc=True, **over):
    d = pkv.GatherDesc()
    d.total, d.num_indices, d.batch_size, d.num_kv_heads, d.head_dim, d.page_size, d.num_pages = 10, 4, 2, 2, 128, 16, 8
    d.kv_dtype, d.k_scale, d.v_scale = pkv.PKV_FP4_E2M1, 1.0, 1.0
    for k, v in over.items():
        setattr(d, k, v)
    names = ("k_cache", "v_cache", "k_block_scales", "v_block_scales", "kv_indptr", "kv_indices", "kv_start", "out_indptr",
             "k_out", "v_out", "status")
    args = [None if n in null else ctypes.c_void_p((pointers or {}).get(n, 0x1000)) for n in names]
    return lib.pkv_gather_kv(ctypes.byref(d) if desc else None, *args, None)


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), pkv.PKV_ERR_INVALID_ARG), (dict(total=1 << 31), pkv.PKV_ERR_UNSUPPORTED),
    (dict(num_indices=-1), pkv.PKV_ERR_INVALID_ARG), (dict(batch_size=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), pkv.PKV_ERR_INVALID_ARG), (dict(num_kv_heads=1 << 17), pkv.PKV_ERR_UNSUPPORTED),
    (dict(head_dim=96), pkv.PKV_ERR_UNSUPPORTED), (dict(page_size=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(num_pages=-1), pkv.PKV_ERR_INVALID_ARG), (dict(kv_dtype=1), pkv.PKV_ERR_INVALID_ARG),
    (dict(kv_dtype=pkv.PKV_BF16), pkv.PKV_ERR_INVALID_ARG),  # scales without a 4-bit cache
    (dict(k_scale=float("nan")), pkv.PKV_ERR_INVALID_ARG), (dict(v_scale=float("inf")), pkv.PKV_ERR_INVALID_ARG),
])
def test_gather_bad_descriptors(lib, over, status):
    assert _gather(lib, **over) == status
    assert lib.pkv_last_error()


@pytest.mark.parametrize("name", ["k_cache", "v_cache", "k_block_scales", "v_block_scales", "kv_indptr", "kv_indices",
                                  "out_indptr", "k_out", "v_out"])
def test_gather_missing_or_misaligned_tensors(lib, name):
    assert _gather(lib, null=(name,)) == pkv.PKV_ERR_INVALID_ARG
    assert _gather(lib, pointers={name: 0x1002}) == pkv.PKV_ERR_INVALID_ARG


def test_gather_from_no_pages_is_not_refused(lib):
    """(Without a GPU what passes the checks fails at the launch.)"""
    empty = ("k_cache", "v_cache", "k_block_scales", "v_block_scales", "kv_indices")
    if not torch.cuda.is_available():
        assert _gather(lib, null=empty, num_pages=0, num_indices=0) == pkv.PKV_ERR_CUDA
        assert _gather(lib, null=("kv_indices",), num_indices=0) == pkv.PKV_ERR_CUDA
    for name in empty:
        assert _gather(lib, null=(name,)) == pkv.PKV_ERR_INVALID_ARG


def test_gather_of_nothing(lib):
    assert _gather(lib, desc=False) == pkv.PKV_ERR_INVALID_ARG
    assert _gather(lib, total=0) == pkv.PKV_OK and _gather(lib, batch_size=0) == pkv.PKV_OK


def _desc(**over):
    d = pkv.PlanDesc()
    d.batch_size, d.num_qo_heads, d.num_kv_heads, d.head_dim, d.page_size, d.num_pages = 0, 8, 2, 128, 16, 4
    d.window_left, d.causal, d.sm_scale, d.kv_dtype = -1, 1, 0.1, pkv.PKV_FP4_E2M1
    zero = np.zeros(1, dtype=np.int32)
    d.qo_indptr = d.kv_indptr = d.kv_last_page_len = zero.ctypes.data
    d._keep = zero
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kind", [pkv.PKV_PREFILL, pkv.PKV_PREFILL_RAGGED])
def test_plans_over_4_bit_caches_are_decode_plans(lib, kind):
    out = ctypes.c_void_p()
    d = _desc(kind=kind)
    assert lib.pkv_plan_create(ctypes.byref(out), ctypes.byref(d), None) == pkv.PKV_ERR_UNSUPPORTED
    assert b"pkv_gather_kv" in lib.pkv_last_error()
    d = _desc(kind=pkv.PKV_DECODE, kv_dtype=6)
    assert lib.pkv_plan_create(ctypes.byref(out), ctypes.byref(d), None) == pkv.PKV_ERR_INVALID_ARG


@pytest.mark.parametrize("pages,page,refused", [(1 << 28, 16, True), ((1 << 28) - 1, 16, False), ((1 << 31) - 1, 3, True),
                                                ((1 << 31) - 1, 1, False)])
def test_pools_of_2_32_rows_are_refused(lib, pages, page, refused):
    """The decode counts rows in 32 bits; 2^32 - 1 is no row. (A batch of none: without a GPU what
    passes the checks fails later.)"""
    out = ctypes.c_void_p()
    d = _desc(kind=pkv.PKV_DECODE, num_pages=pages, page_size=page)
    assert (lib.pkv_plan_create(ctypes.byref(out), ctypes.byref(d), None) == pkv.PKV_ERR_UNSUPPORTED) == refused
    assert (b"2^32 rows" in lib.pkv_last_error()) == refused
    lib.pkv_plan_destroy(out)


def test_noalloc_decode_refuses_4_bit_caches(lib):
    d = _desc(kind=pkv.PKV_DECODE)
    assert lib.pkv_decode_noalloc(ctypes.byref(d), None, None, None, None, None, None) == pkv.PKV_ERR_UNSUPPORTED


def test_bad_copies_with_block_scales(lib):
    p, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)

    def call(k=p, v=p, ks=p, vs=p, layers=2, layer_bytes=1 << 20, scale_layer=4000, pages=8, page_bytes=320, scale_page=40,
             src=p, dst=p, n=2, count=None, status=None):
        return lib.pkv_copy_pages_blocks(k, v, ks, vs, layers, layer_bytes, scale_layer, pages, page_bytes, scale_page, src, dst,
                                         n, count, status, None)

    for over in (dict(n=-1), dict(layers=-1), dict(pages=-1), dict(page_bytes=-16), dict(layer_bytes=-16), dict(scale_page=-4),
                 dict(scale_layer=-4), dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(src=None), dict(dst=None),
                 dict(k=odd), dict(v=odd), dict(ks=odd), dict(vs=odd), dict(src=ctypes.c_void_p(0x1001)),
                 dict(count=ctypes.c_void_p(0x1002)), dict(status=ctypes.c_void_p(0x1002))):
        assert call(**over) == pkv.PKV_ERR_INVALID_ARG, over
    for over in (dict(page_bytes=40), dict(layer_bytes=1000), dict(page_bytes=1 << 31), dict(scale_page=42),
                 dict(scale_layer=4002), dict(scale_page=1 << 31)):
        assert call(**over) == pkv.PKV_ERR_UNSUPPORTED, over
    for over in (dict(n=0), dict(layers=0)):
        assert call(**over, k=None, ks=None) == pkv.PKV_OK, over


def test_run_without_a_plan(lib):
    assert lib.pkv_run_blocks(*[None] * 9) == pkv.PKV_ERR_INVALID_ARG


def test_gather_descriptor_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    body = "".join(f'printf("%zu ", offsetof(pkv_gather_desc, {f}));' for f, _ in pkv.GatherDesc._fields_)
    src = tmp_path / "a.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {' + body +
                   'printf("%zu", sizeof(pkv_gather_desc)); return 0;}')
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "a")], check=True)
    got = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()
    want = [getattr(pkv.GatherDesc, f).offset for f, _ in pkv.GatherDesc._fields_] + [ctypes.sizeof(pkv.GatherDesc)]
    assert [int(x) for x in got] == want


# ---------------------------------------------------------------- the binding's checks
def _bind_append(**over):
    k = _dev(4, 2, 64)
    args = dict(slots=_dev(4, dtype=torch.int64), k_cache=_dev(3, 4, 2, 32, dtype=torch.uint8),
                v_cache=_dev(3, 4, 2, 32, dtype=torch.uint8), k_block_scales=_dev(3, 4, 2, 4, dtype=torch.float8_e4m3fn),
                v_block_scales=_dev(3, 4, 2, 4, dtype=torch.float8_e4m3fn)) | over
    pkv.norm_rope_append(None, k, k, **args)


def test_an_append_passes_block_scales_on(fake_lib):  # noqa: F811
    _bind_append()
    name, args = fake_lib.calls[-1]
    assert name == "pkv_norm_rope_append_blocks" and args[0].kv_dtype == pkv.PKV_FP4_E2M1 and len(args) == 17
    assert args[0].head_dim == 64 and args[13] and args[14] and args[15] is None


@pytest.mark.parametrize("over", [
    dict(k_block_scales=None), dict(v_block_scales=None),
    dict(k_block_scales=torch.zeros(3, 4, 2, 4, dtype=torch.float8_e4m3fn)),  # host memory
    dict(k_block_scales="wrong shape"), dict(v_block_scales="wrong type"),
    dict(k_cache="whole columns"), dict(k_cache="bf16", v_cache="bf16")])
def test_an_append_refuses_wrong_block_scales(fake_lib, over):  # noqa: F811
    made = {"wrong shape": lambda: _dev(3, 4, 2, 8, dtype=torch.float8_e4m3fn),
            "wrong type": lambda: _dev(3, 4, 2, 4, dtype=torch.float32),
            "whole columns": lambda: _dev(3, 4, 2, 64, dtype=torch.uint8), "bf16": lambda: _dev(3, 4, 2, 64)}
    over = {k: made[v]() if isinstance(v, str) else v for k, v in over.items()}
    with pytest.raises(ValueError):
        _bind_append(**over)
    assert not fake_lib.calls


def _bind_gather(**over):
    i32 = lambda n: _dev(n, dtype=torch.int32)  # noqa: E731
    args = dict(kv_indptr=i32(3), kv_indices=i32(5), out_indptr=i32(3), total=7,
                k_out=_dev(7, 2, 64), v_out=_dev(7, 2, 64)) | over
    return pkv.gather_kv(_dev(6, 4, 2, 64), _dev(6, 4, 2, 64), **args)


def test_a_gather_describes_its_tensors(fake_lib):  # noqa: F811
    _bind_gather(k_scale=torch.tensor(0.5))
    d = fake_lib.calls[-1][1][0]
    assert (d.total, d.num_indices, d.batch_size, d.num_kv_heads, d.head_dim, d.page_size, d.num_pages) == (7, 5, 2, 2, 64, 4, 6)
    assert d.kv_dtype == pkv.PKV_BF16 and d.k_scale == 0.5 and d.v_scale == 1.0


@pytest.mark.parametrize("over", [
    dict(out_indptr="i32 2"), dict(kv_start="i32 3"), dict(kv_indices="i64"), dict(k_out="heads"), dict(v_out="rows"),
    dict(k_block_scales="scales"), dict(k_out=None, total=None), dict(k_out="f32")])
def test_a_gather_refuses_what_does_not_fit(fake_lib, over):  # noqa: F811
    made = {"i32 2": lambda: _dev(2, dtype=torch.int32), "i32 3": lambda: _dev(3, dtype=torch.int32),
            "i64": lambda: _dev(5, dtype=torch.int64), "heads": lambda: _dev(7, 3, 64), "rows": lambda: _dev(8, 2, 64),
            "scales": lambda: _dev(6, 4, 2, 4, dtype=torch.float8_e4m3fn), "f32": lambda: _dev(7, 2, 64, dtype=torch.float32)}
    over = {k: made[v]() if isinstance(v, str) else v for k, v in over.items()}
    with pytest.raises(ValueError):
        _bind_gather(**over)
    assert not fake_lib.calls


# ---------------------------------------------------------------- copies of pages
def _bind_copy(dtype=torch.uint8, shape=(3, 6, 5, 2, 32), **over):
    i = _dev(2, dtype=torch.int32)
    scales = {x + "_block_scales": _dev(*shape[:-1], shape[-1] // 8, dtype=torch.float8_e4m3fn) for x in "kv"}
    pkv.copy_pages(_dev(*shape, dtype=dtype), _dev(*shape, dtype=dtype), i, i, **(scales | over))


def test_a_copy_takes_block_scales_along(fake_lib):  # noqa: F811
    _bind_copy()
    name, args = fake_lib.calls[-1]
    assert name == "pkv_copy_pages_blocks" and len(args) == 16
    assert args[4:10] == (3, 6 * 5 * 2 * 32, 6 * 5 * 2 * 4, 6, 5 * 2 * 32, 5 * 2 * 4)
    _bind_copy(shape=(6, 5, 2, 32))
    assert fake_lib.calls[-1][1][4:10] == (1, 6 * 5 * 2 * 32, 6 * 5 * 2 * 4, 6, 5 * 2 * 32, 5 * 2 * 4)
    _bind_copy(k_block_scales=None, v_block_scales=None)
    assert fake_lib.calls[-1][0] == "pkv_copy_pages"


@pytest.mark.parametrize("over", [
    dict(k_block_scales=None), dict(v_block_scales=None), dict(dtype=torch.float8_e4m3fn),
    dict(k_block_scales=torch.zeros(3, 6, 5, 2, 4, dtype=torch.float8_e4m3fn)),  # host memory
    dict(v_block_scales=_dev(3, 6, 5, 2, 2, dtype=torch.float8_e4m3fn)),
    dict(k_block_scales=_dev(2, 6, 5, 2, 4, dtype=torch.float8_e4m3fn)),
    dict(k_block_scales=_dev(3, 6, 5, 2, 4, dtype=torch.float32))])
def test_copies_refuse_wrong_block_scales(fake_lib, over):  # noqa: F811
    with pytest.raises(ValueError):
        _bind_copy(**over)
    assert not fake_lib.calls
