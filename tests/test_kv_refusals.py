"""More refusals of the tpla_kv_* entry points before a GPU is touched:
results whose rows would lie over one another.  CPU only."""
import pytest

import mla_latent_kv_dim_b200 as tp
from test_kv_abi import F32, INVALID, _decode, _prefill, _t


@pytest.mark.parametrize("stride", [(0, 1, 1), (8, 0, 1)])
def test_broadcast_lse(stride):
    assert _decode(lse=_t((4, 8, 1), F32, stride=stride)) == INVALID
    assert _prefill(lse=_t((30, 8, 1), F32, stride=stride)) == INVALID
    assert tp.launch_count() == 0
