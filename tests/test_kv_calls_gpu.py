"""Python calls of the tpla_kv_* operators that the binding answers itself:
results too large for the GPU."""
import pytest
import torch

import mla_latent_kv_dim_b200 as tp

pytestmark = pytest.mark.gpu


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
