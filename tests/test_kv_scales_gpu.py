"""Very small and very large softmax scales of tpla_kv_decode and
tpla_kv_prefill."""
import pytest
import torch

import mla_latent_kv_dim_b200 as tp

pytestmark = pytest.mark.gpu


def _calls(dev, gain, scale):
    """Decode and prefill of the same values times `gain`."""
    gen = torch.Generator().manual_seed(8)
    T = 150
    q, k, v = ((0.5 * torch.randn((T, h, 64), generator=gen)).bfloat16() for h in (4, 2, 2))
    q, k, v = (q * gain).to(dev), (k * gain).to(dev), v.to(dev)
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    n = torch.tensor([T], dtype=torch.int32, device=dev)
    return (*tp.kv_prefill(q, k, v, cu, scale=scale),
            *tp.kv_decode(q[-1:], k[None], v[None], n, None, scale=scale))


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [-40, -20, 20, 59])
def test_a_power_of_two_moved_into_the_scale(cuda_dev, power, sign):
    """q and k times 2^p and the scale by 2^-2p: every product, sum and score
    is the same number up to its exponent (|q . k| < 2^8, so nothing leaves
    f32's range: 2^(8 + 118), and 0.125 log2(e) 2^-118 is a normal number), so
    the results are the same bits."""
    want = _calls(cuda_dev, 1.0, sign * 0.125)
    got = _calls(cuda_dev, 2.0 ** power, sign * 0.125 * 2.0 ** (-2 * power))
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert same == [True] * 4
    assert tp.device_status() == 0


def test_zero_scale_over_large_products(cuda_dev):
    """A scale of 0 weighs every key alike, however large the products: out is
    the mean of the values.  2^-8 of it for the weights' and 2^-18 for the
    f32 sums' rounding; lse = ln n, an f32 of at most 5.02."""
    gen = torch.Generator().manual_seed(8)
    T = 150
    k = (0.5 * torch.randn((T, 2, 64), generator=gen)).bfloat16() * 2.0 ** 59
    q = (0.5 * torch.randn((T, 4, 64), generator=gen)).bfloat16() * 2.0 ** 59
    v = torch.randn((T, 2, 64), generator=gen).abs().bfloat16()
    mean = v.double().cumsum(0) / torch.arange(1, T + 1)[:, None, None]
    mean = mean.repeat_interleave(2, 1).to(cuda_dev)
    ln = torch.arange(1, T + 1, device=cuda_dev).double().log()[:, None, None]
    q, k, v = (x.to(cuda_dev) for x in (q, k, v))
    cu = torch.tensor([0, T], dtype=torch.int32, device=cuda_dev)
    n = torch.tensor([T], dtype=torch.int32, device=cuda_dev)
    out, lse = tp.kv_prefill(q, k, v, cu, scale=0.0)
    one, one_lse = tp.kv_decode(q[-1:], k[None], v[None], n, None, scale=0.0)
    for o, l, m, z in ((out, lse, mean, ln), (one, one_lse, mean[-1:], ln[-1:])):
        error, lse_error = ((o - m).abs() / m).max().item(), (l - z).abs().max().item()
        assert error <= 2.0 ** -8 + 2.0 ** -18 and lse_error <= 2.0 ** -20
    assert tp.device_status() == 0
