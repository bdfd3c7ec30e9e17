"""pkv_norm_rope_append's refusals, on the host before any CUDA call, and its structure's
layout against the header."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_sliding_gb300 import build as pkv_build
from paged_kv_sliding_gb300 import pkv
from tests.test_abi_cpu import HEADER


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def _call(lib, null=(), pointers=None, **over):
    d = pkv.AppendDesc()
    d.num_tokens, d.q_stride, d.k_stride, d.v_stride = 4, 512, 256, 256
    d.num_qo_heads, d.num_kv_heads, d.head_dim, d.page_size, d.num_pages = 4, 2, 128, 16, 8
    d.kv_dtype, d.rotary_dim, d.max_position = pkv.PKV_BF16, 128, 100
    d.eps, d.k_scale, d.v_scale = 1e-6, 1.0, 1.0
    for k, v in over.items():
        setattr(d, k, v)
    names = ("q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions", "slots", "q_out", "k_out", "k_cache",
             "v_cache", "status")
    args = [None if n in null else ctypes.c_void_p((pointers or {}).get(n, 0x1000)) for n in names]
    return lib.pkv_norm_rope_append(ctypes.byref(d), *args, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_tokens=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(num_tokens=1 << 31), pkv.PKV_ERR_UNSUPPORTED),
    (dict(num_qo_heads=-4), pkv.PKV_ERR_INVALID_ARG),
    (dict(num_qo_heads=0, num_kv_heads=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(num_kv_heads=1 << 20), pkv.PKV_ERR_UNSUPPORTED),
    (dict(head_dim=96), pkv.PKV_ERR_UNSUPPORTED),
    (dict(kv_dtype=1), pkv.PKV_ERR_INVALID_ARG),
    (dict(rotary_dim=144), pkv.PKV_ERR_INVALID_ARG),
    (dict(rotary_dim=24), pkv.PKV_ERR_UNSUPPORTED),
    (dict(eps=-1.0), pkv.PKV_ERR_INVALID_ARG),
    (dict(eps=float("nan")), pkv.PKV_ERR_INVALID_ARG),
    (dict(k_scale=float("inf")), pkv.PKV_ERR_INVALID_ARG),
    (dict(weight_offset=float("nan")), pkv.PKV_ERR_INVALID_ARG),
    (dict(page_size=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(num_pages=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(max_position=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(q_stride=516), pkv.PKV_ERR_UNSUPPORTED),
    (dict(v_stride=-8), pkv.PKV_ERR_UNSUPPORTED),
])
def test_bad_descriptors(lib, over, status):
    assert _call(lib, **over) == status, lib.pkv_last_error()
    assert lib.pkv_last_error()


@pytest.mark.parametrize("null", [("q",), ("q_out",), ("k",), ("v",), ("slots",), ("k_cache",), ("v_cache",),
                                  ("cos_sin",), ("positions",), ("k_out", "k_cache", "v_cache")])
def test_missing_tensors(lib, null):
    assert _call(lib, null=null) == pkv.PKV_ERR_INVALID_ARG, null


@pytest.mark.parametrize("name", ["q", "k", "v", "q_weight", "cos_sin", "q_out", "k_cache", "slots", "positions"])
def test_misaligned_tensors(lib, name):
    assert _call(lib, pointers={name: 0x1002}) == pkv.PKV_ERR_INVALID_ARG


def test_null_descriptor_and_no_tokens(lib):
    assert lib.pkv_norm_rope_append(None, *[None] * 14) == pkv.PKV_ERR_INVALID_ARG
    assert _call(lib, num_tokens=0, null=("q", "k", "v")) == pkv.PKV_OK  # no launch


def test_descriptor_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    body = "".join(f'printf("%zu ", offsetof(pkv_append_desc, {f}));' for f, _ in pkv.AppendDesc._fields_)
    src = tmp_path / "a.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {' + body +
                   'printf("%zu", sizeof(pkv_append_desc)); return 0;}')
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "a")], check=True)
    got = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()
    want = [getattr(pkv.AppendDesc, f).offset for f, _ in pkv.AppendDesc._fields_] + [ctypes.sizeof(pkv.AppendDesc)]
    assert [int(x) for x in got] == want
