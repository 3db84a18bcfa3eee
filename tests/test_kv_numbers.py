"""Numbers that the tpla_kv_* calls refuse before a GPU is touched.  CPU only:
the descriptors of test_kv_abi, whose addresses are never read."""
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from test_kv_abi import INVALID, _decode, _prefill


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_scales_whose_log2_form_is_no_f32(scale):
    """scale log2(e), by which the kernels multiply, would be infinite, and
    every score of 0 no number."""
    before = tp.launch_count()
    assert _decode(scale=scale) == INVALID
    assert _prefill(scale=scale) == INVALID
    assert tp.launch_count() == before


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 1e-45, 0.0])
def test_scales_that_are_taken(scale):
    """They get past the check: refused for the workspace (given, too small)
    or, without a GPU, as unsupported."""
    assert _decode(scale=scale, ws=0x10000, bytes=16) not in (0, INVALID)
    if not torch.cuda.is_available():
        assert _prefill(scale=scale) == -2


@pytest.mark.parametrize("out_dtype", [torch.int32, torch.float64, torch.int8, None])
def test_output_types(out_dtype):
    """Refused by name, whatever else is given; not answered with f32."""
    b = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 64, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1,), dtype=torch.int32)
    with pytest.raises(TypeError, match="out_dtype"):
        tp.kv_decode(b, c, c, i, i[None], scale=0.1, out_dtype=out_dtype)
    with pytest.raises(TypeError, match="out_dtype"):
        tp.kv_prefill(b, b, b, i, scale=0.1, out_dtype=out_dtype)
