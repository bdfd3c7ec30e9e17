"""The binding's own work on the host, without a GPU: tensors that report a CUDA device over
host memory, and a library that notes the calls it gets."""
from __future__ import annotations


import pytest
import torch

from paged_kv_sliding_gb300 import pkv


class OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def _dev(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


class Library:
    """Stands in for libpkv: every call succeeds and is noted in `calls`."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return pkv.PKV_OK
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(pkv, "_lib", lib)
    monkeypatch.setattr(pkv, "_append_descs", {})
    monkeypatch.setattr(pkv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


def _append(**over):
    k = _dev(4, 2, 64)
    pkv.norm_rope_append(None, k, k, slots=_dev(4, dtype=torch.int64), k_cache=_dev(3, 4, 2, 64), v_cache=_dev(3, 4, 2, 64),
                         **over)


@pytest.mark.parametrize("name", ["k_scale", "v_scale", "eps", "weight_offset"])
def test_an_append_takes_the_value_that_a_scalar_has_now(lib, name):
    """A scale kept in a tensor of one number and changed in place."""
    x = torch.tensor(0.5)
    for value in (0.5, 2.0, 0.25):
        x.fill_(value)
        _append(**{name: x})
        desc = lib.calls[-1][1][0]
        assert isinstance(desc, pkv.AppendDesc) and getattr(desc, name) == value


def test_an_append_takes_the_truth_that_a_flag_has_now(lib):
    x = torch.tensor(False)
    for value in (False, True, False):
        x.fill_(value)
        _append(interleaved=x)
        assert lib.calls[-1][1][0].interleaved == int(value)


def test_an_append_refuses_what_is_no_number(lib):
    for bad in ("half", None, torch.zeros(2)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            _append(k_scale=bad)
    assert not lib.calls
