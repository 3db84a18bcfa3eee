"""Python calls of the tpla_kv_* operators that the binding answers itself:
numbers past a C int, results too large for the GPU."""
import pytest
import torch

import mla_latent_kv_dim_b200 as tp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["rope_offset", "q_rope_offset"])
@pytest.mark.parametrize("value", [1 << 32, -(1 << 32), (1 << 32) + 8])
def test_offsets_past_an_int_are_refused(cuda_dev, name, value):
    """Not taken modulo 2^32, which would be a column of the row."""
    k = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=cuda_dev)
    cache = torch.zeros((1, 64, 1, 64), dtype=torch.bfloat16, device=cuda_dev)
    at = torch.zeros((1,), dtype=torch.int32, device=cuda_dev)
    table = torch.zeros((1, 1), dtype=torch.int32, device=cuda_dev)
    cs = torch.ones((4, 32), device=cuda_dev)
    before = tp.launch_count()
    with pytest.raises(tp.TplaError) as e:
        tp.kv_append(k, k, at, table, cache, cache.clone(), cos_sin=cs, q=k,
                     **{"rope_offset": 0, "q_rope_offset": 0, name: value})
    assert e.value.status == -1 and tp.launch_count() == before
    assert not cache.any()


def test_results_that_do_not_fit(cuda_dev):
    """torch's own error where the GPU has no room for what a call allocates
    (here an output of 2 TB), as the latent calls raise it."""
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=cuda_dev).expand(1 << 20, 8192, 64)
    kv = torch.zeros((1, 64, 1, 64), dtype=torch.bfloat16, device=cuda_dev)
    n = torch.zeros((1,), dtype=torch.int32, device=cuda_dev)
    with pytest.raises(torch.OutOfMemoryError):
        tp.kv_decode(q, kv, kv, n, n[None], scale=0.1)
    with pytest.raises(torch.OutOfMemoryError):
        tp.kv_prefill(q, kv[0], kv[0], n, scale=0.1)
