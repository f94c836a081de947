"""CPU-side checks of pkv_pages_copy: page tensors whose bytes the call could not tell."""
import ctypes

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from paged_kv_cache_30_gb300 import build as pkv_build
from tests.test_abi import _t


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def copy(lib, t):
    one = (ctypes.POINTER(pkv.PkvTensor) * 1)(ctypes.pointer(t))
    a, b = (_t([0], pkv.DTYPE_I32, None, p) for p in (0x20000000, 0x30000000))
    return lib.pkv_pages_copy(ctypes.cast(one, ctypes.c_void_p), 1, ctypes.byref(a), ctypes.byref(b), None)


@pytest.mark.parametrize("dtype", [pkv.DTYPE_BF16, pkv.DTYPE_F32, pkv.DTYPE_I32, pkv.DTYPE_FP8])
def test_the_dtypes_of_the_library_are_taken(lib, dtype):
    assert copy(lib, _t([8, 4, 4], dtype, None, 0x10000000)) == 0


@pytest.mark.parametrize("dtype", [0, 5, -1, 1 << 20])
def test_other_dtypes_are_refused(lib, dtype):
    assert copy(lib, _t([8, 4, 4], dtype, None, 0x10000000)) == -1
    assert "dtype" in pkv.last_error()


def test_other_torch_dtypes_are_refused():
    lists = torch.zeros(1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for dtype in (torch.float16, torch.uint8, torch.int64):
        with pytest.raises(pkv.PkvError, match="dtype"):
            pkv.pages_copy(torch.zeros(4, 8, dtype=dtype), *lists)


@pytest.mark.parametrize("shape,stride,code", [
    ([8, 4, 4], [16, 1, 4], 0), ([8, 3, 1, 2], [6, 2, 99, 1], 0), ([8, 2, 3], [8, 1, 2], 0),
    ([8, 3, 3], [20, 2, 2], -1),        # as many elements as the span has, but not all of them
    ([8, 2, 2, 2], [20, 1, 1, 5], -1), ([8, 4, 2], [8, 0, 7], -1), ([8, 5, 3], [40, 3, 1], 0),
])
def test_pages_with_gaps_and_repeats_are_refused(lib, shape, stride, code):
    assert copy(lib, _t(shape, pkv.DTYPE_F32, stride, 0x10000000)) == code
