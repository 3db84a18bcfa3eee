"""Weights far below the largest one in the fp16 form of tpla_kv_decode and
tpla_kv_prefill: a first token that draws nearly all of the attention, as many
models' first tokens do, and very many others whose weights together are what
the output consists of."""
import math

import pytest
import torch

import mla_latent_kv_dim_b200 as tp

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -11
# The first key is (SCORE / 8) in each of 64 columns, the queries are 1, the
# scale is 1/8 and the other keys are 0: scores SCORE and 0, exact in fp16 and
# f32.  The others' weight is e^-17.75 = 2^-25.61 of the first's.
SCORE = 17.75


def _cache(dev, L):
    k = torch.zeros((L // 64, 64, 1, 64), dtype=torch.float16, device=dev)
    k[0, 0] = SCORE / 8
    v = torch.ones((L // 64, 64, 1, 64), dtype=torch.float16, device=dev)
    v[0, 0] = 0
    return k, v


def _check(out, lse, n, rounding):
    """A row over n keys: (n - 1) w / (1 + (n - 1) w), lse = SCORE +
    ln(1 + (n - 1) w), w = e^-SCORE.

    out: `rounding` is the relative half step of the others' weights (all the
    same number) in fp16; the f32 products add at most 2^10 of them a row or
    piece one step after another, each with at most 2^-23 of the sum: 2^-13 +
    2^-13 for the sum of the weights; the exponential's argument (25.6 in log2
    units) and value are good to 2^-19.
    lse: the running sum starts with the first key's weight, and each later
    addition may be off by 2^-24 of it.  There are 2^8 in prefill (one a key
    tile) and at most 2^10 in decode: with 64 heads a warp has half of each of
    the 2^8 pages, so a lane 8 of its tokens, which it adds two at a time.
    Together 2^-14; 2^-18 for the roundings of a maximum of 25.6 log2 units, of
    the logarithm and of the result."""
    w = math.exp(-SCORE)
    z = 1 + (n - 1) * w
    want = (n - 1) * w / z
    error = ((out.double() - want).abs().max() / want).item()
    lse_error = (lse.double() - SCORE - math.log(z)).abs().max().item()
    assert error <= rounding + 2.0 ** -12 + 2.0 ** -18
    assert lse_error <= 2.0 ** -14 + 2.0 ** -18


# prefill stores the largest weight at 2^9 or above: the others at 2^-16.61,
# where fp16 has steps of 2^-24.  Decode stores it at 2^15: a normal number.
PREFILL, DECODE = 2.0 ** -8.39, EPS


@pytest.mark.parametrize("B,T", [(200, 64), (400, 256)])
def test_prefill_over_a_dominant_first_token(cuda_dev, B, T):
    """Two hundred items in two pieces each; and enough that none is cut."""
    L = 1 << 14
    k, v = _cache(cuda_dev, L)
    q = torch.ones((T * B, 1, 64), dtype=torch.float16, device=cuda_dev)
    pt = torch.arange(L // 64, dtype=torch.int32, device=cuda_dev)[None].repeat(B, 1)
    cu = torch.arange(0, T * B + 1, T, dtype=torch.int32, device=cuda_dev)
    n = torch.full((B,), L, dtype=torch.int32, device=cuda_dev)
    out, lse = tp.kv_prefill(q, k, v, cu, seq_lens=n, page_table=pt, scale=0.125, causal=False)
    _check(out, lse, L, PREFILL)
    assert tp.device_status() == 0


@pytest.mark.parametrize("Hq", [1, 20, 64])
def test_decode_over_a_dominant_first_token(cuda_dev, Hq):
    """Enough requests that every one lies in a slice or two."""
    L, B = 1 << 14, 300
    k, v = _cache(cuda_dev, L)
    q = torch.ones((B, Hq, 64), dtype=torch.float16, device=cuda_dev)
    pt = torch.arange(L // 64, dtype=torch.int32, device=cuda_dev)[None].repeat(B, 1)
    n = torch.full((B,), L, dtype=torch.int32, device=cuda_dev)
    out, lse = tp.kv_decode(q, k, v, n, pt, scale=0.125)
    _check(out, lse, L, DECODE)
    assert tp.device_status() == 0


@pytest.mark.parametrize("dtype,step", [(torch.float16, 5.9), (torch.float16, 6.1),
                                        (torch.bfloat16, 7.9), (torch.bfloat16, 8.1)])
def test_maxima_that_climb_by_nearly_the_lag(cuda_dev, dtype, step):
    """Scores that climb by `step` log2 units from a key tile of 64 to the next,
    just below and above what prefill lets weights grow by before it rescales:
    none overflows, and the last tile, which has nearly all of the weight, gives
    the result.  Tile j's scores are all s_j (k is s_j in one column and 0 in
    the others, q 1, the scale 1), its values j: out is a mean of whole numbers."""
    tiles = 12
    s = (torch.arange(tiles) * step * math.log(2)).to(dtype)
    k = torch.zeros((64 * tiles, 1, 64), dtype=dtype)
    k[:, 0, 0] = s.repeat_interleave(64)
    v = torch.arange(tiles).repeat_interleave(64).to(dtype)[:, None, None].expand(-1, 1, 64).contiguous()
    q = torch.zeros((256, 1, 64), dtype=dtype)
    q[..., 0] = 1
    cq = torch.tensor([0, 256], dtype=torch.int32, device=cuda_dev)
    ck = torch.tensor([0, 64 * tiles], dtype=torch.int32, device=cuda_dev)
    out, lse = tp.kv_prefill(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), cq, ck, scale=1.0,
                             causal=False)
    p = torch.softmax(s.double(), 0)
    want, want_lse = (p * torch.arange(tiles)).sum().item(), torch.logsumexp(s.double(), 0).item() + math.log(64)
    # one rounding a weight; arguments below 2^7 log2 units in f32: 2^-17 of a weight
    eps = torch.finfo(dtype).eps / 2
    error, lse_error = (out.double() - want).abs().max().item(), (lse.double() - want_lse).abs().max().item()
    assert error <= (eps + 2.0 ** -16) * want and lse_error <= 2.0 ** -16
    assert tp.device_status() == 0
