"""tpla_kv_prefill within the bound of its own roundings.  kv_cases.check_attention
allows what kv_decode needs, which divides by the sum of the rounded weights."""
import numpy as np
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import EPS, attend64, paged_cache, rows_of

pytestmark = pytest.mark.gpu


def _check(out, lse, ref, dtype, out_dtype):
    """out: a weight is rounded once to 16 bits (EPS) in the numerator, and the
    divisor is the f32 sum of the weights before that: EPS sum_j p_j |v_j|.  In
    fp16 weights are stored times 2^9, those below 2^-14 then with the absolute
    half step 2^-25, against a sum of at least 2^9 (some key's weight is the
    reference's, or larger): 2^-34 sum_j |v_j|.  EPS of the value for the output
    (fp16: 2^-25 at least).  f32: scores of |q . k| < 1000 are off by 2^-23 * 1000
    * scale (<= 1/8) = 1.5e-5 in natural log units at most, in the weights and
    in their sum: 3e-5 sum_j p_j |v_j|, which covers the sums' 2^-20.
    lse: 1.5e-5, 2^-20 of the sum and 2^-22 of the value."""
    want, want_lse, mag, vsum = ref
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()[..., 0]
    tol = (EPS[dtype] + 3e-5) * mag + EPS[out_dtype] * np.abs(want) + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -34 * vsum
    if out_dtype == torch.float16:
        tol = tol + 2.0 ** -25
    worst = (np.abs(out - want) / tol).max()
    lse_worst = (np.abs(lse - want_lse) / (1.6e-5 + 2.0 ** -22 * np.abs(want_lse))).max()
    assert worst <= 1.0 and lse_worst <= 1.0


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_packed_prompts(cuda_dev, Dk, Dv, dtype):
    gen = torch.Generator().manual_seed(Dk)
    new = [1, 200, 129, 600]
    T, scale = sum(new), Dk ** -0.5
    q = (1.5 * torch.randn((T, 6, Dk), generator=gen)).to(dtype)
    k = torch.randn((T, 2, Dk), generator=gen).to(dtype)
    v = torch.randn((T, 2, Dv), generator=gen).to(dtype)
    cu = np.cumsum([0] + new)
    ref = [np.concatenate(x) for x in zip(*[
        attend64(q[a:z], k[a:z], v[a:z], scale, range(1, z - a + 1)) for a, z in zip(cu, cu[1:])])]
    d = [x.to(cuda_dev) for x in (q, k, v, torch.tensor(cu, dtype=torch.int32))]
    for out_dtype in (dtype, torch.float32):
        out, lse = tp.kv_prefill(*d, scale=scale, out_dtype=out_dtype)
        _check(out, lse, ref, dtype, out_dtype)
    assert tp.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_pieces(cuda_dev, dtype):
    gen = torch.Generator().manual_seed(7)
    L, T = 5000, 40
    kc, pt = paged_cache([L], 2, 128, dtype, gen)
    vc = torch.randn(kc.shape, generator=gen).to(dtype)
    q = (1.5 * torch.randn((T, 6, 128), generator=gen)).to(dtype)
    ref = attend64(q, rows_of(kc, pt, 0, L), rows_of(vc, pt, 0, L), 0.088, range(L - T + 1, L + 1))
    d = [x.to(cuda_dev) for x in (q, kc, vc, torch.tensor([0, T], dtype=torch.int32))]
    out, lse = tp.kv_prefill(*d, seq_lens=torch.tensor([L], dtype=torch.int32, device=cuda_dev),
                             page_table=pt.to(cuda_dev), scale=0.088)
    _check(out, lse, ref, dtype, torch.float32)
    assert tp.device_status() == 0
