"""The current device as the native calls ask for it, with PyTorch's raw
functions and without them.  CPU only: a tensor that says it is on a device."""
import pytest
import torch

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build


class Rows:
    """What the calls read of a device tensor of rows."""

    dtype, shape = torch.bfloat16, (3, 64)

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def stride(self):
        return (64, 1)

    def data_ptr(self):
        return 0x7F0000000004      # misaligned: refused by the library before anything is launched


@pytest.mark.parametrize("raw", [False, True])
def test_tensors_elsewhere_are_refused(monkeypatch, raw):
    dg_build.build()
    monkeypatch.setattr(dg, "_native", None)
    monkeypatch.setattr(dg, "_raw_stream", (lambda d: 0) if raw else None)
    monkeypatch.setattr(dg, "_current_device", (lambda: 2) if raw else None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("Stream", (), {"cuda_stream": 0}))
    with pytest.raises(ValueError, match="on the current device"):
        dg.dg_activate(Rows(0), dg.DG_ACT_RELU, y=Rows(0))
    with pytest.raises(ValueError, match="on the current device"):
        dg.dg_activate(Rows(2), dg.DG_ACT_RELU, y=Rows(1))
    with pytest.raises(dg.DgError, match="MISALIGNED"):
        dg.dg_activate(Rows(2), dg.DG_ACT_RELU, y=Rows(2))


@pytest.fixture(autouse=True)
def _again():
    yield
    dg._native = None
    dg._load_native()       # PyTorch's own functions bound again
