"""Widths of FP4 rows at the edge of what the calls take, on CPU: refused, or passed on whole."""
import pytest

from fp4_compressed_sparse_02_gb300 import csa2
from test_devices import B16, OnDevice, fp4, machine  # noqa: F401  (a fixture)


@pytest.mark.parametrize("rows,cols", [(4, 33), (4, 31), (4, 48), (5, 32)])
def test_fp4_quant_refuses_an_out_of_another_shape(machine, rows, cols):  # noqa: F811
    with pytest.raises(ValueError, match="x's shape"):
        csa2.fp4_quant(OnDevice(0, B16, rows, cols), out=fp4(0, 4, 32))
    assert machine == []
    csa2.fp4_quant(OnDevice(0, B16, 4, 32), out=fp4(0, 4, 32))
    assert len(machine) == 1
