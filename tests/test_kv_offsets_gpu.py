"""Offsets of tpla_kv_prefill that fall: recorded, and never more work than the
call has room for.  The bounds on the list of items are checked on the CPU by
test_kv_plan."""
import numpy as np
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import attend64, check_attention, paged_cache, rows_of

pytestmark = pytest.mark.gpu


def _inputs(T, Hq, Hkv, seed):
    gen = torch.Generator().manual_seed(seed)
    return [(1.2 * torch.randn((T, h, 64), generator=gen)).bfloat16() for h in (Hq, Hkv, Hkv)]


def test_rows_claimed_twice(cuda_dev):
    """[0, 70), [70, 60) and [60, 100): the second has no rows, the others
    keep theirs, and rows 60 to 69 hold values of one or the other (two blocks
    store them, in pieces of a row)."""
    q, k, v = _inputs(120, 4, 2, 1)
    cu = torch.tensor([0, 70, 60, 100], dtype=torch.int32)
    res = torch.full((120, 4, 64), 3.0, device=cuda_dev)
    lse = torch.full((120, 4, 1), 3.0, device=cuda_dev)
    tp.kv_prefill(*(x.to(cuda_dev) for x in (q, k, v, cu)), scale=0.125, out=res, lse=lse)
    assert tp.device_status() == -6 and tp.device_status() == 0
    refs = [attend64(q[a:z], k[a:z], v[a:z], 0.125, range(1, z - a + 1)) for a, z in ((0, 70), (60, 100))]
    check_attention(res[:60], lse[:60], [x[:60] for x in refs[0]], torch.bfloat16, torch.float32, "first")
    check_attention(res[70:100], lse[70:100], [x[10:] for x in refs[1]], torch.bfloat16, torch.float32, "third")
    shared = res[60:70].double().cpu().numpy()
    error = np.minimum(*(np.abs(shared - r) for r in (refs[0][0][60:], refs[1][0][:10])))
    assert error.max() <= (2 * 2.0 ** -8 + 3e-5) * np.abs(v.double().numpy()).max()
    assert (res[100:] == 3).all().item() and (lse[100:] == 3).all().item()


def test_offsets_that_end_in_zeros(cuda_dev):
    """A batch padded with zeros behind its last request: that request and the
    ones before it keep their rows."""
    q, k, v = _inputs(100, 2, 2, 2)
    d = [x.to(cuda_dev) for x in (q, k, v)]
    good = torch.tensor([0, 30, 100], dtype=torch.int32, device=cuda_dev)
    want, want_lse = tp.kv_prefill(*d, good, scale=0.125)
    out, lse = tp.kv_prefill(*d, torch.tensor([0, 30, 100, 0, 0], dtype=torch.int32, device=cuda_dev),
                             scale=0.125)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert tp.device_status() == -6


@pytest.mark.parametrize("Hq,times", [(2, 40), (2, 3000), (128, 9)])
def test_more_rows_than_the_call_has_room_for(cuda_dev, Hq, times):
    """All rows claimed `times` times over packed keys: nothing is written."""
    T = 3000
    q, k, v = (x.to(cuda_dev) for x in _inputs(T, Hq, 1, 3))
    cu = torch.tensor([0, T] * times, dtype=torch.int32, device=cuda_dev)
    res = torch.full((T, Hq, 64), 3.0, device=cuda_dev)
    lse = torch.full((T, Hq, 1), 3.0, device=cuda_dev)
    tp.kv_prefill(q, k, v, cu, scale=0.125, out=res, lse=lse)
    assert tp.device_status() == -6 and tp.device_status() == 0
    assert (res == 3).all().item() and (lse == 3).all().item()


@pytest.mark.parametrize("T,times", [(100, 2), (100, 40), (600, 40)])
def test_items_in_pieces(cuda_dev, T, times):
    """The same over long paged keys, whose items are cut.  100 tokens are one
    item (of 128): a claim by each of the 2 times - 1 requests fits, and every
    claim gives the same values.  600 are five: 200 items where 83 fit."""
    L, Hq = 6000, 2
    gen = torch.Generator().manual_seed(4)
    lens = [L] * (2 * times - 1)
    kc, pt = paged_cache([L], 1, 64, torch.bfloat16, gen)
    vc = torch.randn(kc.shape, generator=gen).bfloat16()
    q = torch.randn((T, Hq, 64), generator=gen).bfloat16()
    cu = torch.tensor([0, T] * times, dtype=torch.int32, device=cuda_dev)
    res = torch.full((T, Hq, 64), 3.0, device=cuda_dev)
    lse = torch.full((T, Hq, 1), 3.0, device=cuda_dev)
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device=cuda_dev)  # every word negative
    tp.kv_prefill(q.to(cuda_dev), kc.to(cuda_dev), vc.to(cuda_dev), cu,
                  seq_lens=torch.tensor(lens, dtype=torch.int32, device=cuda_dev),
                  page_table=pt.repeat(len(lens), 1).to(cuda_dev), scale=0.125, out=res, lse=lse,
                  workspace=ws)
    assert tp.device_status() == -6 and tp.device_status() == 0
    if T == 100:
        ref = attend64(q, rows_of(kc, pt, 0, L), rows_of(vc, pt, 0, L), 0.125, range(L - T + 1, L + 1))
        check_attention(res, lse, ref, torch.bfloat16, torch.float32, "twice")
    else:
        assert (res == 3).all().item() and (lse == 3).all().item()
