"""What the Python serving calls refuse before anything reaches the library.
CPU only: the tensors' shapes and types are looked at first, then that they
are on a device."""
import ctypes

import pytest
import torch

import fp16_tensor_core_gb300 as dg
from fp16_tensor_core_gb300 import build as dg_build

BF, I32 = torch.bfloat16, torch.int32


class Handle:
    """A cache or rotary handle as the calls see it, over host memory."""

    def __init__(self, c, name):
        self.c = c
        setattr(self, name, ctypes.addressof(c))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dg_build.build()


def heads(tokens=3, n=4, dim=64, dtype=BF):
    return torch.zeros(tokens, n, dim, dtype=dtype)


CACHE = Handle(dg._KvCache(0, 0, 0, 0, 10, 2, 16, 64), "cache_address")
ROTARY = Handle(dg._Rotary(0, 100, 64, 0), "rotary_address")
SHAPE = r"x must be BF16 or FP16 \[tokens, heads, head_dim\] with contiguous heads"


@pytest.mark.parametrize("x,match", [
    (heads(dtype=torch.float32), SHAPE), (torch.zeros(3, 64, dtype=BF), SHAPE),
    (torch.zeros(2, 3, 4, 64, dtype=BF), SHAPE), (heads(dim=128)[..., ::2], SHAPE),
    (heads(), "CUDA device memory"), (heads(dtype=torch.float16), "CUDA device memory"),
])
def test_heads(x, match):
    with pytest.raises(ValueError, match=match):
        dg.dg_rope(x, x, torch.zeros(3, dtype=I32), ROTARY)


def test_what_is_no_tensor():
    with pytest.raises(AttributeError):
        dg.dg_rope(None, None, None, ROTARY)
    with pytest.raises(AttributeError):
        dg.dg_kv_read(CACHE, torch.zeros(3, dtype=I32), k=[1.0])
    with pytest.raises(AttributeError):
        dg.dg_kv_append("k", "v", "slots", CACHE)
    with pytest.raises((AttributeError, ValueError)):
        dg.dg_attn_decode(1, 2, 3, 4, 5, 6)


def test_the_other_kind_of_handle():
    """A rotary table is no cache: nothing is read from it as one."""
    with pytest.raises(AttributeError, match="cache_address"):
        dg.dg_kv_append(FakeHeads(), FakeHeads(), torch.zeros(3, dtype=I32), ROTARY)


class FakeHeads:
    """What the calls read of a device tensor of heads."""

    dtype, shape, is_cuda = BF, (3, 2, 64), True

    def stride(self):
        return (128, 64, 1)

    def data_ptr(self):
        return 0x7F0000000000


def test_calls_with_host_tensors():
    k, slots = heads(n=2), torch.zeros(3, dtype=I32)
    for call in (lambda: dg.dg_kv_append(k, k, slots, CACHE), lambda: dg.dg_kv_read(CACHE, slots, v=k),
                 lambda: dg.dg_attn_decode(k, k, CACHE, slots[:, None], slots, slots)):
        with pytest.raises(ValueError, match="CUDA device memory"):
            call()
    assert dg.dg_kv_read(CACHE, slots) is None


def test_the_native_functions_count_their_arguments():
    native = dg._load_native()
    for f in (native.rope, native.kv_append, native.kv_read, native.attn_decode, native.bind):
        with pytest.raises(TypeError, match="arguments wanted"):
            f()
        with pytest.raises(TypeError, match="arguments wanted"):
            f(*range(20))
