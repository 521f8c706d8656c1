"""Widths of FP4 rows at the edge of what the calls take, on CPU: refused, or passed on whole."""
import ctypes

import pytest

from fp4_compressed_sparse_02_gb300 import csa2
from test_devices import B16, OnDevice, fp4, machine  # noqa: F401  (a fixture)
from test_rows_validation import L, SHAPE, linear, quant  # noqa: F401


@pytest.mark.parametrize("rows,cols", [(4, 33), (4, 31), (4, 48), (5, 32)])
def test_fp4_quant_refuses_an_out_of_another_shape(machine, rows, cols):  # noqa: F811
    with pytest.raises(ValueError, match="x's shape"):
        csa2.fp4_quant(OnDevice(0, B16, rows, cols), out=fp4(0, 4, 32))
    assert machine == []
    csa2.fp4_quant(OnDevice(0, B16, 4, 32), out=fp4(0, 4, 32))
    assert len(machine) == 1


# the last widths whose offsets, and the whole steps rounded up from them, stay in 32 bits, and the next
@pytest.mark.parametrize("fn,args,most", [
    ("csa2_fp4_quant", lambda n, rows: quant(o_cols=n, x_stride=n, o_rows=rows), 1 << 30),
    ("csa2_fp4_linear", lambda n, rows: linear(x_cols=n, w_cols=n, x_rows=rows), 1 << 26)])
def test_widths_that_leave_32_bits_are_refused(L, fn, args, most):  # noqa: F811
    for n in (most + 32, 2 ** 31 - 32):
        for rows in (0, 4):
            assert getattr(L, fn)(ctypes.byref(args(n, rows)), None) == SHAPE
            assert b"cols must be at most" in L.csa2_last_error_message()
    assert getattr(L, fn)(ctypes.byref(args(most, 0)), None) == 0
