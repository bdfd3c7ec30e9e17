"""Norm, rotation and cache append in one pass, against the same formulas in float64.

Tolerances: the fp32 arithmetic before the one rounding is a sum of d squares in a tree
(d / 8 + 5 adds), a reciprocal root (2 ulp), and five products and a sum, so a rotated
value is off by at most 2^-18 (|a| + |b|) of its pair; then half a step of the stored type
(bf16 2^-8, E4M3 2^-4 or 2^-10 below its normals, E5M2 2^-3 or 2^-17). V is not computed
with: it has to be the exact conversion.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_sliding_gb300.inputs import KV8_DTYPES

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": (2.0 ** -8, 0.0), "e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}
LARGEST = {"bf16": 3.0e38, "e4m3": 448.0, "e5m2": 57344.0}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_sliding_gb300 import build, pkv as binding
    build.build()
    binding.load_library()
    return binding


def _dtype(kv_type):
    return torch.bfloat16 if kv_type == "bf16" else KV8_DTYPES[kv_type]


def _inputs(n, hq, hkv, d, P, rotary, kv_type, seed=0, pad=()):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    qkv = (torch.randn(n, (hq + 2 * hkv) * d, generator=g, device="cuda") * 2).to(torch.bfloat16)
    q, k, v = (x.view(n, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    pages = -(-n // P) + 3
    slots = torch.as_tensor(rng.permutation(pages * P)[:n].astype(np.int64), device="cuda")
    for i in pad:
        slots[i] = -1 - i
    pos = torch.as_tensor(rng.integers(0, 500, size=n).astype(np.int32), device="cuda")
    table = None
    if rotary:
        a = torch.arange(500, dtype=torch.float64, device="cuda")[:, None] * \
            1000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)[None]
        table = torch.cat([a.cos(), a.sin()], 1).float()
    wq, wk = ((torch.randn(d, generator=g, device="cuda") * 0.3).to(torch.bfloat16) for _ in range(2))
    cache = [(torch.randn(pages, P, hkv, d, generator=g, device="cuda")).to(_dtype(kv_type)) for _ in range(2)]
    return dict(q=q, k=k, v=v, slots=slots, positions=pos, cos_sin=table, wq=wq, wk=wk, k_cache=cache[0], v_cache=cache[1])


def _reference(x, w, offset, eps, table, pos, interleaved):
    """y in float64, and |a| + |b| of each column's pair."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * (w.double() + offset)
    size = y.abs()
    if table is not None:
        r = table.shape[1]
        c, s = (t[:, None] for t in table.double()[pos.long().clamp(0, table.shape[0] - 1)].chunk(2, 1))
        first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        a, b = y[..., first].clone(), y[..., second].clone()
        y, size = y.clone(), size.clone()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


def _near(got, ref, size, kv_type, what):
    rel, low = HALF_STEP[kv_type]
    ref = ref.clamp(-LARGEST[kv_type], LARGEST[kv_type])
    tol = rel * ref.abs() + low + 2.0 ** -18 * size
    off = (got.double() - ref).abs()
    assert not (off > tol).any(), f"{what}: {float((off / tol.clamp(min=1e-30)).max()):.2f} of the tolerance"


def _check(pkv, s, kv_type="bf16", offset=0.0, eps=1e-6, interleaved=False, norm=True, k_scale=1.0, v_scale=1.0, what=""):
    n = s["q"].shape[0]
    before = [x.clone() for x in (s["k_cache"], s["v_cache"])]
    q_out = torch.full_like(s["q"], 9.0, memory_format=torch.contiguous_format)
    k_out = torch.full_like(s["k"], 9.0, memory_format=torch.contiguous_format)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wq, wk = (s["wq"], s["wk"]) if norm else (None, None)
    got = pkv.norm_rope_append(s["q"], s["k"], s["v"], positions=s["positions"], cos_sin=s["cos_sin"], slots=s["slots"],
                               k_cache=s["k_cache"], v_cache=s["v_cache"], q_weight=wq, k_weight=wk, eps=eps,
                               weight_offset=offset, interleaved=interleaved, k_scale=k_scale, v_scale=v_scale,
                               q_out=q_out, k_out=k_out, status=status)
    torch.cuda.synchronize()
    assert got is q_out and status.item() == 0
    keep = s["slots"] >= 0
    rows = s["slots"][keep]
    q_ref, q_size = _reference(s["q"], wq, offset, eps, s["cos_sin"], s["positions"], interleaved)
    k_ref, k_size = _reference(s["k"], wk, offset, eps, s["cos_sin"], s["positions"], interleaved)
    _near(q_out[keep], q_ref[keep], q_size[keep], "bf16", what + " q")
    _near(k_out[keep], k_ref[keep], k_size[keep], "bf16", what + " k_out")
    assert (q_out[~keep] == 9.0).all() and (k_out[~keep] == 9.0).all()
    hkv, d = s["k"].shape[1:]
    untouched = torch.ones(s["k_cache"].shape[0] * s["k_cache"].shape[1], dtype=torch.bool, device="cuda")
    untouched[rows] = False
    raw = torch.int16 if kv_type == "bf16" else torch.uint8
    for cache, old in zip((s["k_cache"], s["v_cache"]), before):
        assert torch.equal(cache.view(raw).view(-1, hkv, d)[untouched], old.view(raw).view(-1, hkv, d)[untouched]), what
    stored = s["k_cache"].view(raw).view(-1, hkv, d)[rows].view(_dtype(kv_type))
    _near(stored.float(), k_ref[keep] / k_scale, k_size[keep] / k_scale, kv_type, what + " k_cache")
    v = (s["v"][keep].float() / v_scale)
    v = v.to(torch.bfloat16) if kv_type == "bf16" else v.clamp(-LARGEST[kv_type], LARGEST[kv_type]).to(_dtype(kv_type))
    assert torch.equal(s["v_cache"].view(raw).view(-1, hkv, d)[rows], v.view(raw)), what
    assert n == 0 or keep.any()


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_types_and_rotations(pkv, d, interleaved, kv_type):
    for rotary in (0, 16, d // 2, d - 16, d):
        for n in (1, 2, 67):
            s = _inputs(n, 8, 2, d, 16, rotary, kv_type, seed=d + n)
            _check(pkv, s, kv_type, offset=1.0, interleaved=interleaved, k_scale=0.25, v_scale=0.5,
                   what=f"d {d} rotary {rotary} n {n}")


@pytest.mark.parametrize("heads", [(1, 1), (5, 1), (7, 7), (32, 8), (3, 2)])
@pytest.mark.parametrize("n", [1, 16, 341, 5000])
def test_heads_and_lengths(pkv, heads, n):
    """Both launch shapes (few rows and many), head counts that end inside a group of four."""
    s = _inputs(n, *heads, 128, 5, 128, "bf16", seed=n)
    _check(pkv, s, what=f"heads {heads} n {n}")


@pytest.mark.parametrize("n", [9, 4000])
def test_padding_rows_are_left_alone(pkv, n):
    s = _inputs(n, 8, 2, 128, 16, 128, "bf16", seed=1, pad=(0, 3, n - 2, n - 1))
    s["positions"][n - 1] = 10 ** 6  # a padding row's position is not looked at
    _check(pkv, s, what="padding")


def test_without_norm_and_with_odd_eps(pkv):
    for norm, eps in ((False, 1e-6), (True, 0.0), (True, 3.0)):
        _check(pkv, _inputs(50, 4, 4, 64, 16, 64, "bf16", seed=2), norm=norm, eps=eps, what=f"norm {norm} eps {eps}")


@pytest.mark.parametrize("kv_type", ["e4m3", "e5m2"])
def test_values_beyond_the_format_are_its_largest(pkv, kv_type):
    s = _inputs(40, 4, 2, 128, 16, 0, kv_type, seed=3)
    s["v"].mul_(1e6)
    s["k"].mul_(1e6)
    _check(pkv, s, kv_type, norm=False, what=kv_type)
    s["v"][0, 0, 0], s["v"][0, 0, 1], s["v"][0, 0, 2] = float("inf"), float("-inf"), float("nan")
    pkv.norm_rope_append(None, s["k"], s["v"], slots=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    row = s["v_cache"].view(torch.uint8).view(-1, 2, 128)[s["slots"][0]].view(_dtype(kv_type)).float()
    assert row[0, 0] == LARGEST[kv_type] and row[0, 1] == -LARGEST[kv_type] and torch.isnan(row[0, 2])


def test_a_row_with_nan_or_infinity_keeps_it_to_itself(pkv):
    s = _inputs(33, 4, 2, 128, 16, 128, "bf16", seed=4)
    clean = pkv.norm_rope_append(s["q"], None, positions=s["positions"], cos_sin=s["cos_sin"], q_weight=s["wq"]).clone()
    s["q"][7, 1, 5] = float("nan")
    s["q"][8, 2, 6] = float("inf")
    dirty = pkv.norm_rope_append(s["q"], None, positions=s["positions"], cos_sin=s["cos_sin"], q_weight=s["wq"])
    same = (clean == dirty).all(-1)
    assert (~same).nonzero().tolist() == [[7, 1], [8, 2]] and torch.isnan(dirty[7, 1]).all()


def test_parts_alone_and_in_place(pkv):
    """q alone, k without a cache, and q and k rotated where they are."""
    s = _inputs(70, 8, 2, 128, 16, 128, "bf16", seed=5)
    q, k = s["q"].contiguous(), s["k"].contiguous()
    args = dict(positions=s["positions"], cos_sin=s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"])
    k_out = torch.empty_like(k)
    q_out = pkv.norm_rope_append(q, k, k_out=k_out, **args)
    assert torch.equal(pkv.norm_rope_append(q, None, **args), q_out)
    assert pkv.norm_rope_append(None, k, k_out=(k2 := torch.empty_like(k)), **args) is None and torch.equal(k2, k_out)
    pkv.norm_rope_append(q, k, q_out=q, k_out=k, **args)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)


def test_no_tokens_and_padding_without_a_cache(pkv):
    s = _inputs(20, 4, 2, 128, 16, 128, "bf16", seed=10, pad=(2, 19))
    args = dict(cos_sin=s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"])
    got = pkv.norm_rope_append(s["q"][:0], s["k"][:0], s["v"][:0], positions=s["positions"][:0], slots=s["slots"][:0],
                               k_cache=s["k_cache"], v_cache=s["v_cache"], **args)
    assert got.shape == (0, 4, 128)
    k_out = torch.full((20, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((20, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    pkv.norm_rope_append(s["q"], s["k"], positions=s["positions"], slots=s["slots"], k_out=k_out, q_out=q_out, **args)
    skipped = (k_out == 9.0).all(-1).all(-1).nonzero().flatten().tolist()
    assert skipped == [2, 19] == (q_out == 9.0).all(-1).all(-1).nonzero().flatten().tolist()


def test_one_row_for_every_token(pkv):
    """A token stride of zero: the same row at every position."""
    s = _inputs(30, 4, 2, 128, 16, 128, "bf16", seed=11)
    q = s["q"][:1].contiguous()
    args = dict(positions=s["positions"], cos_sin=s["cos_sin"], q_weight=s["wq"])
    assert torch.equal(pkv.norm_rope_append(q.expand(30, -1, -1), None, **args),
                       pkv.norm_rope_append(q.expand(30, -1, -1).contiguous(), None, **args))


def test_v_of_a_bf16_cache_is_v_bit_for_bit(pkv):
    """Every bf16 there is, zeros of both signs, subnormals and infinities among them."""
    bits = torch.arange(1 << 16, device="cuda").to(torch.int16)
    v = bits.view(torch.bfloat16).view(-1, 2, 64)
    n = v.shape[0]
    k_cache = torch.zeros(n // 8, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    slots = torch.randperm(n, device="cuda")
    pkv.norm_rope_append(None, v, v, slots=slots, k_cache=k_cache, v_cache=v_cache)
    for cache in (k_cache, v_cache):  # k too: neither normalised nor rotated
        got = cache.view(-1, 2, 64)[slots]
        assert torch.equal(torch.isnan(got), torch.isnan(v))
        same = got.view(torch.int16) == v.view(torch.int16)
        assert (same | torch.isnan(v)).all()


SCALES = [0.75, 0.013, 0.021, 0.3, 7 / 1024, 45 / 1024, 3.0, 7.0, 9.37e-5, 1 - 2.0 ** -24, 1 + 2.0 ** -23, 1.1 * 2.0 ** -64,
          1.5 * 2.0 ** 63, 1.5 * 2.0 ** 64, 1.5 * 2.0 ** -65, 1.5 * 2.0 ** 126, 2.0 ** 127, 2.0 ** -126, 2.0 ** -127,
          2.0 ** -128, 2.0 ** -149, 3 * 2.0 ** -149]


@pytest.mark.parametrize("kv_type", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("scale", SCALES)
def test_values_over_a_scale_are_the_quotients_bit_for_bit(pkv, scale, kv_type):
    """Every bf16 there is over scales whose reciprocals are rounded (some of the quotients lie
    halfway between two stored values), at the ends of fp32 and below its normals: the fp32
    quotient, which numpy gives, rounded once more. k too: neither normalised nor rotated."""
    v = torch.arange(1 << 16).to(torch.int16).view(torch.bfloat16).view(-1, 2, 64)
    n = v.shape[0]
    with np.errstate(all="ignore"):
        want = torch.from_numpy(v.float().numpy() / np.float32(scale))
    if kv_type != "bf16":
        want = want.clamp(-LARGEST[kv_type], LARGEST[kv_type])
    want = want.to(_dtype(kv_type))
    raw = torch.int16 if kv_type == "bf16" else torch.uint8
    caches = [torch.zeros(n // 8, 8, 2, 64, device="cuda").to(_dtype(kv_type)) for _ in range(2)]
    slots = torch.randperm(n, device="cuda")
    pkv.norm_rope_append(None, v.cuda(), v.cuda(), slots=slots, k_cache=caches[0], v_cache=caches[1], k_scale=scale,
                         v_scale=scale)
    nan = torch.isnan(want.float())
    for cache in caches:
        got = cache.view(raw).view(-1, 2, 64)[slots].cpu()
        assert torch.equal(torch.isnan(got.view(_dtype(kv_type)).float()), nan)
        off = (got != want.view(raw)) & ~nan
        assert not off.any(), (int(off.sum()), v[off][:3], got.view(_dtype(kv_type)).float()[off][:3], want.float()[off][:3])


def test_bad_slots_and_positions_are_recorded(pkv):
    for name, value in (("slots", 10 ** 9), ("slots", 1 << 40), ("positions", 500), ("positions", -1)):
        s = _inputs(20, 4, 2, 128, 16, 128, "bf16", seed=6)
        s[name][11] = value
        k0, v0 = s["k_cache"].clone(), s["v_cache"].clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full((20, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        for st in (status, None):
            pkv.norm_rope_append(s["q"], s["k"], s["v"], positions=s["positions"], cos_sin=s["cos_sin"], slots=s["slots"],
                                 k_cache=s["k_cache"], v_cache=s["v_cache"], q_out=q_out, status=st)
        torch.cuda.synchronize()
        assert status.item() == pkv.PKV_ERR_DEVICE_BOUNDS, name
        assert (q_out[11] == 9.0).all() and not (q_out[10] == 9.0).all()
        wrote = (s["k_cache"] != k0).any(-1).any(-1).sum()
        assert wrote == 19 and (s["v_cache"] != v0).any(-1).any(-1).sum() == 19


def test_a_cache_of_more_than_2_31_elements(pkv):
    """Slots whose element offset passes 32 bits."""
    hkv, d, P = 4, 256, 64
    pages = (1 << 31) // (P * hkv * d) + 40
    k_cache = torch.zeros(pages, P, hkv, d, dtype=torch.float8_e4m3fn, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    s = _inputs(3, 4, hkv, d, P, d, "e4m3", seed=7)
    s["k_cache"], s["v_cache"] = k_cache, v_cache
    s["slots"][:] = torch.tensor([pages * P - 1, (1 << 31) // (hkv * d) + 5, 0], device="cuda")
    _check(pkv, s, "e4m3", what="far slots")


def test_captured_and_replayed_on_another_stream(pkv):
    s = _inputs(64, 8, 2, 128, 16, 128, "bf16", seed=8)
    args = dict(positions=s["positions"], cos_sin=s["cos_sin"], slots=s["slots"], k_cache=s["k_cache"],
                v_cache=s["v_cache"], q_weight=s["wq"], k_weight=s["wk"], q_out=torch.zeros(64, 8, 128,
                                                                                            dtype=torch.bfloat16, device="cuda"))
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.norm_rope_append(s["q"], s["k"], s["v"], **args)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.norm_rope_append(s["q"], s["k"], s["v"], **args)
        pkv.norm_rope_append(args["q_out"], None, q_out=args["q_out"])  # and a second one behind it
    other = _inputs(64, 8, 2, 128, 16, 128, "bf16", seed=9, pad=(60, 61, 62, 63))
    for name in ("q", "k", "v", "positions", "slots"):
        s[name].copy_(other[name])
    args["q_out"].zero_()
    s["k_cache"].zero_()
    g.replay()
    torch.cuda.synchronize()
    want = pkv.norm_rope_append(s["q"], s["k"], s["v"], **dict(args, q_out=torch.zeros_like(args["q_out"])))
    assert torch.equal(args["q_out"], want)
    assert int((s["k_cache"] != 0).any(-1).any(-1).sum()) == 60


def test_refusals_of_the_binding(pkv):
    s = _inputs(4, 4, 2, 128, 16, 128, "bf16")
    ok = dict(positions=s["positions"], cos_sin=s["cos_sin"], slots=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    for bad in (dict(slots=s["slots"].int()), dict(positions=s["positions"][:3]), dict(positions=None),
                dict(cos_sin=s["cos_sin"].double()), dict(v_cache=None), dict(slots=None),
                dict(k_cache=s["k_cache"][..., :64]), dict(v_cache=s["v_cache"][1:]),
                dict(q_weight=s["wq"].float()), dict(q_out=torch.empty(3, 4, 128, dtype=torch.bfloat16, device="cuda")),
                dict(k_cache=s["k_cache"].float(), v_cache=s["v_cache"].float())):
        with pytest.raises(ValueError):
            pkv.norm_rope_append(s["q"], s["k"], s["v"], **dict(ok, **bad))
    with pytest.raises(ValueError):
        pkv.norm_rope_append(s["q"], s["k"], s["v"][:, :1], **ok)
    with pytest.raises(ValueError):
        pkv.norm_rope_append(s["q"].transpose(1, 2), s["k"], s["v"], **ok)
    with pytest.raises(ValueError):
        pkv.norm_rope_append(None, None)
    with pytest.raises(pkv.PkvError):  # k without a cache or k_out
        pkv.norm_rope_append(s["q"], s["k"], positions=s["positions"], cos_sin=s["cos_sin"])
