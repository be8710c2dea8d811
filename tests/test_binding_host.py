"""What the binding takes for a pointer (no GPU): None, an address, or an object with data_ptr().  Anything else is refused
before the library is called; ctypes alone would hand bytes, strings and arrays on as host addresses."""

import ctypes

import pytest

import mxfp8_weight_repack_amd as sh
from mxfp8_weight_repack_amd._lib import _ptr

FOREIGN = [b"bytes", "text", bytearray(64), ctypes.create_string_buffer(64), (ctypes.c_int32 * 4)(), 1.5, [1], object()]


@pytest.mark.parametrize("x", FOREIGN, ids=lambda x: type(x).__name__)
def test_only_pointers_pass(x):
    with pytest.raises(AttributeError):
        _ptr(x)
    # nothing would be launched if the object got through: a plan without a device, sizes of nothing
    plan = sh.Plan([dict(parent=-1, offset=0, rows=32, cols=64, row_stride=64, is_unit=True, optimizer="muon",
                         quantize=True)], 2048, host_only=True)
    for call in (lambda: sh.requant_mxfp8(plan, x, 4096, 4096), lambda: sh.cast_bf16(plan, 4096, x),
                 lambda: sh.moe_combine(x, None, None, 0, 1, 0, 32),
                 lambda: sh.quant_mxfp8(x, "fp32", 0, 32), lambda: sh.mx_matrix(x, None, 0, 32),
                 lambda: sh.swiglu_backward_mxfp8(None, x, None, 0, 32)):
        with pytest.raises(AttributeError):
            call()


def test_pointers_pass():
    class Tensor:
        def data_ptr(self):
            return 4096
    assert _ptr(None) is None and _ptr(4096) == 4096 and _ptr(0) == 0 and _ptr(Tensor()) == 4096
    sh.moe_combine(4096, 4096, Tensor(), 0, 1, 0, 32)
