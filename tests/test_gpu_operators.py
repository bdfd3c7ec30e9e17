"""perf/operators.py: the library's calls against the plain forms on the same inputs, over the
listed cases and a few drawn ones.

Tolerances: page operations and stored bits are equal. Attention: the probabilities are
rounded to bf16 (2^-8; f16 over 8-bit caches) before the product with V, so that an output
is off by 2^-8 sum p |v|, which the plain form gives for |V|, and each side rounds its result
once (2^-8); fp32 work in between adds less than 2^-12 of the same sum. The logits' fp32
sums of d products are off by d 2^-24 sum |q k| scale, 1e-3 at most here. Append: two fp32
computations of the same value, each rounded once: a step of the stored type, and
2^-17 (|a| + |b|) of a pair, which is below the row's largest value."""
from __future__ import annotations

import random

import pytest
import torch

from perf import operators

pytestmark = pytest.mark.gpu

CASES = {c["name"]: c for c in operators.listed()}
for _seed in range(40, 52):
    CASES[f"drawn {_seed}"] = operators.draw(random.Random(_seed))
STEP = {"bf16": (2.0 ** -7, 0.0), "e4m3": (2.0 ** -3, 2.0 ** -9), "e5m2": (2.0 ** -2, 2.0 ** -16)}


def _run(case, own, **over):
    operators.own = own
    try:
        state = operators.prepare(case, 5) | over
        out = operators.run(state)
        torch.cuda.synchronize()
        return out
    finally:
        operators.own = False


def _within(got, want, tol, what):
    off = (got.double() - want.double()).abs()
    assert not (off > tol).any() and torch.equal(torch.isnan(got), torch.isnan(want)), \
        f"{what}: {float((off / tol.clamp(min=1e-30)).max()):.2f} of the tolerance"


@pytest.mark.parametrize("name", CASES)
def test_the_librarys_calls_match_the_plain_forms(name):
    case = CASES[name]
    got, want = _run(case, True), _run(case, False)
    if case["op"] == "attend":
        v = operators.prepare(case, 5)["v"]
        weight = _run(case, False, v=v.float().abs().to(v.dtype))["out"].double()
        _within(got["out"], want["out"], (2.0 ** -8 + 2.0 ** -12) * weight + 2.0 ** -7 * want["out"].double().abs() + 1e-30,
                name)
        finite = torch.isfinite(want["lse"])
        assert torch.equal(finite, torch.isfinite(got["lse"]))
        assert float((got["lse"] - want["lse"])[finite].abs().max()) <= 1e-3
    elif case["op"] == "append":
        for key in ("q", "k", "v"):
            rel, low = STEP["bf16" if key == "q" else case["kv_type"]]
            x, y = got[key].double(), want[key].double()
            tol = rel * torch.maximum(x.abs(), y.abs()) + low + 2.0 ** -17 * y.abs().amax(-1, keepdim=True)
            _within(got[key], want[key], tol, f"{name} {key}")
    else:
        got, want = ({"slots": x} if torch.is_tensor(x) else x for x in (got, want))
        assert got.keys() == want.keys()
        for key in want:
            n = int(want["count"]) if case["op"] == "compact" and key in ("src", "dst") else None
            assert torch.equal(got[key][:n], want[key][:n]), f"{name}: {key}"
