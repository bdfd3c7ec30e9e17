"""Windows with sinks, without a GPU: the oracle's visible set against brute force in
float64 and against its limits, and what the plan refuses on the host."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from paged_kv_sliding_gb300 import build as pkv_build
from paged_kv_sliding_gb300 import inputs as wl
from paged_kv_sliding_gb300 import pkv
from tests.helpers import dense_kv, run_oracle
from tests.test_abi_cpu import _desc


def _work(W, causal=True, q_start=None, qo=(6, 1, 9), kv=(30, 1, 21)):
    return wl.make_workload(name="sinks", qo_lens=list(qo), kv_lens=list(kv), num_qo_heads=4, num_kv_heads=2,
                            head_dim=64, page_size=4, window_left=W, causal=causal, seed=5, q_start=q_start)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("W,sinks", [(0, 1), (3, 4), (5, 2), (3, 100), (50, 3), (2, 0)])
def test_oracle_equals_brute_force(oracle_lib, W, sinks, causal):
    """Softmax over an explicit boolean mask, one row at a time, in float64."""
    w = _work(W, causal, q_start=[24, 0, 40])  # the last request's queries see sinks alone
    out, lse = run_oracle(oracle_lib, w, num_sinks=sinks)
    for b in range(w.batch):
        k, v = (x.double() for x in dense_kv(w, b))
        for i in range(int(w.qo_lens[b])):
            p = int(w.q_start[b]) + i
            seen = [j for j in range(k.shape[0]) if (not causal or j <= p) and (j >= p - W or j < sinks)]
            row = int(w.qo_indptr[b]) + i
            for h in range(4):
                if not seen:
                    assert np.isneginf(lse[row, h]) and not out[row, h].any()
                    continue
                x = (k[seen, h // 2] @ w.q[row, h].double()) * w.sm_scale
                assert abs(float(torch.logsumexp(x, 0)) - lse[row, h]) < 1e-12
                o = torch.softmax(x, 0) @ v[seen, h // 2]
                assert np.abs(o.numpy() - out[row, h]).max() < 1e-12


def test_oracle_limits(oracle_lib):
    """No sinks: the plain window. Sinks that cover the cache: no window."""
    w = _work(3)
    for a, b in ((run_oracle(oracle_lib, w, num_sinks=0), run_oracle(oracle_lib, w)),
                 (run_oracle(oracle_lib, w, num_sinks=30), run_oracle(oracle_lib, w.with_window(-1))),
                 (run_oracle(oracle_lib, w.with_window(-1), num_sinks=2), run_oracle(oracle_lib, w.with_window(-1)))):
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_plan_refuses_bad_sinks_on_the_host():
    pkv_build.build()
    lib = pkv.load_library()
    d, keep = _desc()
    h = ctypes.c_void_p(0x1234)
    assert lib.pkv_plan_create_sinks(ctypes.byref(h), ctypes.byref(d), -1, None, None) == pkv.PKV_ERR_INVALID_ARG
    assert h.value is None and b"num_sinks" in lib.pkv_last_error()
    assert lib.pkv_plan_create_sinks(ctypes.byref(h), ctypes.byref(d), (1 << 24) + 1, None,
                                     None) == pkv.PKV_ERR_UNSUPPORTED
    assert lib.pkv_plan_create_sinks(None, ctypes.byref(d), 4, None, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_plan_create_sinks(ctypes.byref(h), None, 4, None, None) == pkv.PKV_ERR_INVALID_ARG
    d, keep = _desc(head_dim=96)  # everything a plain plan refuses
    assert lib.pkv_plan_create_sinks(ctypes.byref(h), ctypes.byref(d), 4, None, None) == pkv.PKV_ERR_UNSUPPORTED
    d, keep = _desc()
    caps = pkv.PlanCaps()
    caps.max_batch, caps.max_total_q = 1, 100  # below the batch of 2
    assert lib.pkv_plan_create_sinks(ctypes.byref(h), ctypes.byref(d), 4, ctypes.byref(caps),
                                     None) == pkv.PKV_ERR_INVALID_ARG
