"""A list of no pages is refused: the address of an empty tensor is 0, which the library takes for no list at all, and the call
would attend to the whole context."""
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from test_devices import OnDevice, machine  # noqa: F401
from test_kv8_validation import cache, ws

B16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Empty(OnDevice):
    def data_ptr(self):
        return 0


@pytest.mark.parametrize("T", [0, 5])
def test_a_list_without_pages_is_refused(machine, T):  # noqa: F811
    t = lambda name, dtype, *shape: OnDevice(0, dtype, *shape)
    call = lambda n: csa2.kv8_attn(cache(t), t("q", B16, T, 6, 64), t("start", I32, 4), t("length", I32, 3), max_new=1,
                                   pages=(OnDevice if n and T else Empty)(0, I32, T, 2, n), out=t("out", B16, T, 6, 64), lse=t("lse", F32, T, 6), ws=ws(t))
    with pytest.raises(ValueError, match="at least one page"):
        call(0)
    assert machine == []
    call(3)
    assert len(machine) == 1
