"""Attention under a window with sinks (the first keys stay visible), against the
float64 oracle: decode, prefill and ragged prefill, bf16 and 8-bit caches, TMA and
gather page sizes, both decode tiles, splits across the gap, positions whose window is
empty, gap pages that no longer exist, captured plans.

Tolerances come from the arithmetic. P is rounded once (bf16 2^-8, f16 2^-11 over 8-bit
caches) before the P V product and out once to bf16 (2^-8), so with A = sum p |v| (the
oracle over |V|) out is off by at most 2^-8 (A + |out|) plus the effect of the logit
error e, 2 e A. A logit is a d-term fp32 dot product of values whose products are of
order 1: e <= scale d 2^-23 sum|q k| with sum|q k| <= d, plus 2^-18 for ex2 and log2; lse
carries e. The soft cap adds its tanh error, 1e-6 of the cap.
"""
from __future__ import annotations

from dataclasses import replace

import numpy as np
import pytest
import torch

from paged_kv_sliding_gb300 import inputs as wl
from tests.helpers import dense_kv, run_oracle
from tests.test_gpu_capturable import _rebatch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_sliding_gb300 import build, pkv as binding
    build.build()
    binding.load_library()
    return binding


def _abs_v(w):
    v = w.v_cache.float().abs().to(w.v_cache.dtype)
    return replace(w, v_cache=v)


def _check(oracle_lib, w, out, lse, num_sinks, what, cap=0.0, **over):
    args = dict(num_sinks=num_sinks, **over)
    if cap:
        args["logits_soft_cap"] = cap
    ref, ref_lse = run_oracle(oracle_lib, w, **args)
    ref_abs, _ = run_oracle(oracle_lib, _abs_v(w), **args)
    d = w.head_dim
    e = w.sm_scale * over.get("k_scale", 1.0) * d * d * 2.0 ** -23 + 2.0 ** -18 + 1e-6 * cap
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    tol = (2.0 ** -8 + 2 * e) * ref_abs + 2.0 ** -8 * np.abs(ref) + 1e-7
    bad = np.abs(out - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of out, worst {(np.abs(out - ref) / tol).max():.2f} of the tolerance"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(empty, np.isneginf(lse)), what
    assert not out[empty].any(), what
    d_lse = np.abs(lse[~empty] - ref_lse[~empty])
    assert not d_lse.size or d_lse.max() <= e, f"{what}: lse off by {d_lse.max():.2e}, {e:.2e} allowed"


def _run(pkv, w, num_sinks, **over):
    wd = w.to("cuda")
    plan = pkv.plan_for(wd, num_sinks=num_sinks, **over)
    out, lse = plan.run(wd.q, wd.k_cache, wd.v_cache, return_lse=True)
    torch.cuda.synchronize()
    assert plan.device_status() == pkv.PKV_OK
    return out, lse, plan


def _workload(kind, seed, qo, kv, W, d=128, P=16, heads=(8, 2), causal=True, q_start=None):
    return wl.make_workload(name=f"sinks_{kind}_{seed}", kind=kind, qo_lens=qo, kv_lens=kv, num_qo_heads=heads[0],
                            num_kv_heads=heads[1], head_dim=d, page_size=P, window_left=W, causal=causal, seed=seed,
                            q_start=q_start)


DECODE_KV = [1, 3, 17, 40, 64, 129, 200, 700, 1500]


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("P", [1, 5, 8, 16, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode(pkv, oracle_lib, d, P, kv_type):
    for W, sinks in ((0, 1), (31, 4), (100, 70)):
        w = _workload("decode", d + P, [1] * len(DECODE_KV), DECODE_KV, W, d=d, P=P)
        w = w if kv_type == "bf16" else wl.to_kv8(w, kv_type)
        out, lse, plan = _run(pkv, w, sinks)
        assert plan.info["mask_mode"] == 4
        _check(oracle_lib, w, out, lse, sinks, f"d {d} P {P} {kv_type} W {W} sinks {sinks}")


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("P", [1, 5, 16, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_more_than_one_wave(pkv, oracle_lib, d, P, kv_type):
    """More items than SMs hold of the CTAs with long stages: those with short ones."""
    B = 3 * torch.cuda.get_device_properties(0).multi_processor_count // 8 + 1
    kv = np.random.default_rng(d + P).integers(1, 400, size=B)
    for W, sinks in ((0, 1), (31, 4), (100, 70)):
        w = _workload("decode", d + P, [1] * B, kv, W, d=d, P=P, heads=(16, 8))
        w = w if kv_type == "bf16" else wl.to_kv8(w, kv_type)
        out, lse, plan = _run(pkv, w, sinks)
        assert plan.info["kv_tile"] == (32 if kv_type == "bf16" else 64)
        _check(oracle_lib, w, out, lse, sinks, f"d {d} P {P} {kv_type} W {W} sinks {sinks}")


@pytest.mark.parametrize("d", [64, 128])
def test_decode_stages_of_one_wave_and_beyond(pkv, d):
    """Long stages as long as their CTAs fit in one wave (2 items to an SM, 3 at d 64)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    one = (3 if d == 64 else 2) * sms
    for items, keys, tile in ((1, 100, 64), (one, 100, 64), (one, 700, 64), (one + 1, 100, 32), (one + 1, 640, 32),
                              (one + 1, 641, 64), (one + sms // 4 + 1, 1536, 32), (one + sms // 4 + 1, 1537, 64)):
        w = _workload("decode", 1, [1] * items, [2000] * items, keys - 5, d=d, P=16, heads=(1, 1))
        plan = pkv.plan_for(w.to("cuda"), num_sinks=4, disable_split_kv=True)
        assert plan.info["num_work_items"] == items and plan.info["kv_tile"] == tile, (items, keys)


@pytest.mark.parametrize("split", [1, 16, 50, 64, 300])
@pytest.mark.parametrize("P", [1, 16])
def test_decode_splits_across_the_gap(pkv, oracle_lib, P, split):
    """Splits that end inside the sinks, at their end and beyond it."""
    for sinks in (1, 16, 50, 130):
        w = _workload("decode", 3, [1] * 4, [20, 400, 777, 1000], 140, P=P)
        out, lse, plan = _run(pkv, w, sinks, fixed_split_size=split)
        assert (plan.info["num_partials"] > 0) == (split < 141 + sinks)  # keys a row sees
        _check(oracle_lib, w, out, lse, sinks, f"P {P} split {split} sinks {sinks}")


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("P", [1, 3, 16, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill(pkv, oracle_lib, d, P, kv_type):
    qo, kv = [1, 33, 0, 300, 70], [1, 500, 9, 300, 900]
    for W, sinks, causal in ((0, 1, True), (40, 4, True), (150, 140, True), (200, 3, False)):
        w = _workload("prefill", d * P, qo, kv, W, d=d, P=P, heads=(4, 1), causal=causal)
        w = w if kv_type == "bf16" else wl.to_kv8(w, kv_type)
        out, lse, plan = _run(pkv, w, sinks)
        assert plan.info["mask_mode"] == (4 if causal else 5)
        _check(oracle_lib, w, out, lse, sinks, f"d {d} P {P} {kv_type} W {W} sinks {sinks} causal {causal}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("W,sinks", [(0, 1), (31, 5), (300, 129)])
def test_ragged_prefill(pkv, oracle_lib, d, W, sinks):
    w = _workload("prefill", d + W, [70, 1, 300, 0, 257], [103, 900, 700, 5, 257], W, d=d)
    ks, vs = zip(*(dense_kv(w, b) for b in range(w.batch)))
    kv_indptr = np.concatenate([[0], np.cumsum([x.shape[0] for x in ks])]).astype(np.int32)
    plan = pkv.Plan(kind="prefill_ragged", qo_indptr=w.qo_indptr, kv_indptr=kv_indptr, num_qo_heads=8, num_kv_heads=2,
                    head_dim=d, window_left=W, causal=True, sm_scale=w.sm_scale, num_sinks=sinks)
    out, lse = plan.run(w.q.cuda(), torch.cat(ks).cuda(), torch.cat(vs).cuda(), return_lse=True)
    torch.cuda.synchronize()
    assert plan.device_status() == pkv.PKV_OK
    _check(oracle_lib, w, out, lse, sinks, f"ragged d {d} W {W} sinks {sinks}")


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("P", [1, 16, 64])
def test_positions_whose_window_is_empty(pkv, oracle_lib, kind, P):
    """Queries far past the cache see the sinks alone, queries before it nothing, and
    requests without keys nothing."""
    qo = [1] * 5 if kind == "decode" else [3, 140, 5, 1, 4]
    kv = [100, 60, 30, 0, 2]
    w = _workload(kind, 17, qo, kv, 9, P=P, q_start=[400, 55, -200, 3, 50])
    out, lse, _ = _run(pkv, w, 4)
    assert torch.isneginf(lse).any()
    _check(oracle_lib, w, out, lse, 4, f"{kind} P {P}")


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("P", [1, 16, 64])
def test_gap_pages_are_not_read(pkv, oracle_lib, kind, P):
    """Entries of pages between the sinks and the window may name no page at all: same
    bits as with the whole table, and no bounds error."""
    n = 1 if kind == "decode" else 90
    kv, W, sinks = [900, 640, 2000], 63, 5
    w = _workload(kind, 29, [n] * 3, kv, W, P=P)
    whole, lse_whole, _ = _run(pkv, w, sinks)
    idx = w.kv_indices.copy()
    for b in range(3):
        first = int(w.kv_indptr[b])
        idx[first + -(-sinks // P): first + (kv[b] - n - W) // P] = -7
    assert (idx < 0).any()
    out, lse, _ = _run(pkv, replace(w, kv_indices=idx), sinks)
    assert torch.equal(out, whole) and torch.equal(lse, lse_whole)
    _check(oracle_lib, w, out, lse, sinks, f"gap {kind} P {P}")


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_no_sinks_and_no_window_are_the_plain_plan(pkv, kind):
    qo = [1, 1] if kind == "decode" else [50, 200]
    w = _workload(kind, 31, qo, [600, 300], 100)
    plain = _run(pkv, w, 0)
    assert plain[2].info["mask_mode"] == 2
    full = _run(pkv, w.with_window(-1), 0)
    for a, b in ((full, _run(pkv, w.with_window(-1), 7)), (plain, _run(pkv, w, 0))):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    covered = _run(pkv, w, 600)  # sinks over the whole cache: every causal key
    assert (covered[0].float() - full[0].float()).abs().max() < 2e-2


def test_scales_and_soft_cap(pkv, oracle_lib):
    for kind, qo in (("decode", [1, 1, 1]), ("prefill", [40, 130, 1])):
        w = wl.to_kv8(_workload(kind, 37, qo, [500, 131, 77], 60), "e4m3")
        out, lse, _ = _run(pkv, w, 6, k_scale=0.5, v_scale=2.0, logits_soft_cap=20.0)
        _check(oracle_lib, w, out, lse, 6, kind, cap=20.0, k_scale=0.5, v_scale=2.0)


def test_nothing_of_an_invisible_key_reaches_a_decode_row(pkv, oracle_lib):
    """Infinities and NaN in every slot that the row cannot see (the gap, other requests'
    and unused pages, behind the last token): the row is that of a clean cache."""
    for P in (1, 16):
        w = _workload("decode", 41, [1] * 3, [33, 300, 900], 47, P=P)
        clean = _run(pkv, w, 5)
        seen = torch.zeros(w.num_pages, P, dtype=torch.bool)
        for b, n in enumerate(w.kv_lens.tolist()):
            for j in range(n):
                if j < 5 or j >= n - 1 - 47:
                    seen[int(w.kv_indices[int(w.kv_indptr[b]) + j // P]), j % P] = True
        k, v = w.k_cache.clone(), w.v_cache.clone()
        k[~seen] = float("nan")
        v[~seen] = float("inf")
        dirty = _run(pkv, replace(w, k_cache=k, v_cache=v), 5)
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
        _check(oracle_lib, w, clean[0], clean[1], 5, f"P {P}")


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(pkv, oracle_lib, seed):
    rng = np.random.default_rng(500 + seed)
    kind = ["decode", "prefill"][seed % 2]
    B = int(rng.integers(1, 6))
    d, P = int(rng.choice([64, 128, 256])), int(rng.choice([1, 3, 8, 16, 32, 64, 128]))
    W, sinks = int(rng.integers(0, 300)), int(rng.integers(1, 200))
    qo = np.ones(B, dtype=np.int64) if kind == "decode" else rng.integers(0, 200, size=B)
    kv = qo - 1 + rng.integers(0, 1200, size=B) if kind == "decode" else qo + rng.integers(0, 700, size=B)
    q_start = (kv - qo + rng.integers(-20, 200, size=B)).astype(np.int32) if rng.random() < 0.3 else None
    hkv, group = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 3, 8, 20]))
    w = _workload(kind, seed, qo, kv, W, d=d, P=P, heads=(hkv * group, hkv), causal=bool(rng.random() < 0.8),
                  q_start=q_start)
    fmt = rng.choice(["bf16", "e4m3", "e5m2"])
    w = w if fmt == "bf16" else wl.to_kv8(w, str(fmt))
    over = {"fixed_split_size": int(rng.choice([16, 64, 100]))} if kind == "decode" and rng.random() < 0.5 else {}
    out, lse, _ = _run(pkv, w, sinks, **over)
    _check(oracle_lib, w, out, lse, sinks, f"{w.name} {fmt} d {d} P {P} W {W} sinks {sinks} {over}")


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_captured_plan_replays_after_updates(pkv, oracle_lib, kind):
    rng = np.random.default_rng(2)
    n = 20
    qo = np.ones(n, dtype=np.int64) if kind == "decode" else rng.integers(1, 120, size=n)
    w = _workload(kind, 43, qo, qo + rng.integers(100, 900, size=n), 200, heads=(8, 2))
    wd = w.to("cuda")
    rows = 24 if kind == "decode" else 2500
    idx = torch.zeros(w.num_pages, dtype=torch.int32, device="cuda")
    idx[: len(w.kv_indices)] = torch.as_tensor(w.kv_indices, device="cuda")
    q = torch.zeros(rows, 8, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(rows, 8, dtype=torch.float32, device="cuda")
    plan = pkv.plan_for(wd, num_sinks=19, kv_indices=idx, capacity={"max_batch": 24, "max_total_q": rows})
    plan.run(q, wd.k_cache, wd.v_cache, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(q, wd.k_cache, wd.v_cache, out, lse)
    batches = [w, _rebatch(w, qo[:9], qo[:9] + rng.integers(0, 700, size=9), seed=4),
               _rebatch(w, qo[:4], qo[:4] + np.array([0, 3, 2500, 18]), seed=5)]
    for i, x in enumerate(batches):
        m = x.q.shape[0]
        idx[: len(x.kv_indices)] = torch.as_tensor(x.kv_indices, device="cuda")
        q[:m] = x.q.cuda()
        plan.update(kv_indptr=x.kv_indptr, kv_last_page_len=x.kv_last_page_len,
                    qo_indptr=None if kind == "decode" else x.qo_indptr,
                    fixed_split_size=64 if kind == "decode" and i else -1)
        out.fill_(7.0)
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert plan.device_status() == pkv.PKV_OK
        assert (out[m:] == 7.0).all()
        _check(oracle_lib, x, out[:m], lse[:m], 19, f"{kind} batch {i}")


def test_a_wait_that_runs_out_is_reported(pkv):
    for kind, qo in (("decode", [1, 1]), ("prefill", [30, 200])):
        w = _workload(kind, 47, qo, [500, 400], 60)
        wd = w.to("cuda")
        plan = pkv.plan_for(wd, num_sinks=4, wait_limit_us=2000, wait_probe=True)
        plan.run(wd.q, wd.k_cache, wd.v_cache)
        assert plan.device_status() == pkv.PKV_ERR_TIMEOUT
        assert plan.device_status() == pkv.PKV_OK


def test_bad_page_ids_are_recorded(pkv):
    for kind, qo in (("decode", [1]), ("prefill", [30])):
        for P in (1, 16):
            w = _workload(kind, 53, qo, [300], 60, P=P)
            idx = w.kv_indices.copy()
            idx[0] = w.num_pages  # the sinks' page
            wd = replace(w, kv_indices=idx).to("cuda")
            plan = pkv.plan_for(wd, num_sinks=4)
            plan.run(wd.q, wd.k_cache, wd.v_cache)
            assert plan.device_status() == pkv.PKV_ERR_DEVICE_BOUNDS


def test_invisible_keys_of_a_prefill_may_hold_anything_in_k(pkv, oracle_lib):
    """NaN in K wherever no query looks (V finite in the request's own keys), and NaN in both
    in pages of nobody: the same bits as with a clean cache."""
    for P in (1, 16, 64):
        W, sinks, qo, kv = 30, 5, [40, 130, 1], [300, 700, 90]
        w = _workload("prefill", 59, qo, kv, W, P=P)
        clean = _run(pkv, w, sinks)
        seen, own = (torch.zeros(w.num_pages, P, dtype=torch.bool) for _ in range(2))
        for b in range(3):
            for j in range(kv[b]):
                at = int(w.kv_indices[int(w.kv_indptr[b]) + j // P]), j % P
                own[at] = True
                seen[at] = j < sinks or j >= kv[b] - qo[b] - W
        k, v = w.k_cache.clone(), w.v_cache.clone()
        k[~seen] = float("nan")
        v[~own] = float("nan")
        dirty = _run(pkv, replace(w, k_cache=k, v_cache=v), sinks)
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1]), P
        _check(oracle_lib, w, clean[0], clean[1], sinks, f"P {P}")
