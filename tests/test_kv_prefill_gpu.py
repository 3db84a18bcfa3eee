"""GPU parity of tpla_kv_prefill (packed prompts over packed or paged keys and
values) against attention in 64 bits; the bounds are derived in
kv_cases.check_attention."""
import numpy as np
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import attend64, check_attention, paged_cache, rows_of

pytestmark = pytest.mark.gpu


def _cu(lens, first=0):
    return torch.tensor(np.cumsum([first] + list(lens)), dtype=torch.int32)


def _limits(T, L, causal):
    return [max(0, min(L, L - T + i + 1)) if causal else L for i in range(T)]


def _join(parts):
    return [np.concatenate(x) for x in zip(*parts)]


def _packed(new, held, Hq, Hkv, Dk, Dv, dtype, seed, causal, scale):
    """Packed inputs and their reference."""
    gen = torch.Generator().manual_seed(seed)
    T, L = sum(new), sum(held)
    q = (1.5 * torch.randn((T, Hq, Dk), generator=gen)).to(dtype)
    k = torch.randn((L, Hkv, Dk), generator=gen).to(dtype)
    v = torch.randn((L, Hkv, Dv), generator=gen).to(dtype)
    cq, ck = _cu(new), _cu(held)
    parts = []
    for b, (n, m) in enumerate(zip(new, held)):
        rows, keys = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        parts.append(attend64(q[rows], k[keys], v[keys], scale, _limits(n, m, causal)))
    return q, k, v, cq, ck, _join(parts)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("Hq,Hkv,dtype", [(1, 1, torch.bfloat16), (4, 4, torch.float16),
                                          (8, 2, torch.bfloat16), (7, 1, torch.float16),
                                          (48, 1, torch.bfloat16), (129, 1, torch.bfloat16)])
def test_packed_causal(cuda_dev, Dk, Dv, Hq, Hkv, dtype):
    new = [1, 127, 128, 129, 0, 300, 5, 64] if Hq < 40 else [1, 70, 0, 130]
    scale = Dk ** -0.5
    q, k, v, cq, _, ref = _packed(new, new, Hq, Hkv, Dk, Dv, dtype, Hq + Dk, True, scale)
    d = [t.to(cuda_dev) for t in (q, k, v, cq)]
    out, lse = tp.kv_prefill(*d, scale=scale, out_dtype=dtype)
    assert tp.device_status() == 0
    check_attention(out, lse, ref, dtype, dtype, "packed")


@pytest.mark.parametrize("T", [1, 2, 33, 255, 256, 257, 700])
def test_one_prompt(cuda_dev, T):
    """One request: no sorted list of items."""
    q, k, v, cq, _, ref = _packed([T], [T], 4, 2, 128, 128, torch.bfloat16, T, True, 0.088)
    d = [t.to(cuda_dev) for t in (q, k, v, cq)]
    out, lse = tp.kv_prefill(*d, scale=0.088, out_dtype=torch.bfloat16)
    assert tp.device_status() == 0
    check_attention(out, lse, ref, torch.bfloat16, torch.bfloat16, "one")


@pytest.mark.parametrize("causal", [True, False])
def test_other_key_lengths(cuda_dev, causal):
    """Keys of their own lengths: more than tokens (a prefix), fewer (causal
    rows that see nothing), none at all."""
    new, held = [40, 130, 20, 3, 200], [400, 129, 0, 300, 60]
    q, k, v, cq, ck, ref = _packed(new, held, 6, 2, 64, 64, torch.bfloat16, 3, causal, 0.125)
    d = [t.to(cuda_dev) for t in (q, k, v, cq, ck)]
    out, lse = tp.kv_prefill(*d, scale=0.125, causal=causal, out_dtype=torch.float32)
    assert tp.device_status() == 0
    check_attention(out, lse, ref, torch.bfloat16, torch.float32, "lengths")
    if causal:  # 130 tokens against 129 keys, 200 against 60
        assert torch.all(torch.isneginf(lse[40])) and torch.all(torch.isneginf(lse[193:193 + 140]))


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,hf", [
    (torch.bfloat16, 8, 2, 128, 128, False), (torch.float16, 5, 5, 64, 64, True),
    (torch.bfloat16, 16, 1, 192, 128, False)])
def test_paged_chunks_after_a_prefix(cuda_dev, dtype, Hq, Hkv, Dk, Dv, hf):
    gen = torch.Generator().manual_seed(Dk)
    new, held = [17, 64, 1, 200, 90], [17, 264, 500, 201, 128]
    kc, pt = paged_cache(held, Hkv, Dk, dtype, gen, heads_first=hf)
    vc = torch.randn(kc.shape[:3] + (Dv,), generator=gen).to(dtype)
    q = (1.5 * torch.randn((sum(new), Hq, Dk), generator=gen)).to(dtype)
    cq, scale = _cu(new), Dk ** -0.5
    ref = _join([attend64(q[cq[b]:cq[b + 1]], rows_of(kc, pt, b, m), rows_of(vc, pt, b, m), scale,
                          _limits(n, m, True)) for b, (n, m) in enumerate(zip(new, held))])
    # everything that no token owns is NaN
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, n in enumerate(held):
        for t in range(n):
            used[pt[b, t // 64], t % 64] = True
    kc[~used] = float("nan")
    vc[~used] = float("nan")
    dk = torch.empty_strided(kc.shape, kc.stride(), dtype=dtype, device=cuda_dev).copy_(kc)
    seq = torch.tensor(held, dtype=torch.int32)
    out, lse = tp.kv_prefill(q.to(cuda_dev), dk, vc.to(cuda_dev), cq.to(cuda_dev),
                             seq_lens=seq.to(cuda_dev), page_table=pt.to(cuda_dev), scale=scale,
                             out_dtype=dtype)
    assert tp.device_status() == 0
    check_attention(out, lse, ref, dtype, dtype, "paged")


@pytest.mark.parametrize("new,held,Hq,Hkv,causal", [
    ([1], [5000], 4, 2, True), ([7, 1, 0, 30], [3000, 9000, 700, 2000], 8, 1, True),
    ([200], [4300], 2, 2, True), ([40, 3], [1500, 1], 40, 1, False),
    ([3000, 2], [2500, 1025], 2, 1, True)])
def test_few_items_with_many_keys(cuda_dev, new, held, Hq, Hkv, causal):
    """Too few items for the GPU: their keys are cut into pieces and joined.
    (The last case has rows that see nothing in some pieces, or in none.)"""
    gen = torch.Generator().manual_seed(sum(held))
    kc, pt = paged_cache(held, Hkv, 64, torch.bfloat16, gen, spare_pages=5)
    vc = torch.randn(kc.shape, generator=gen).to(torch.bfloat16)
    q = (1.5 * torch.randn((sum(new), Hq, 64), generator=gen)).to(torch.bfloat16)
    cq = _cu(new)
    ref = _join([attend64(q[cq[b]:cq[b + 1]], rows_of(kc, pt, b, m), rows_of(vc, pt, b, m), 0.125,
                          _limits(n, m, causal)) for b, (n, m) in enumerate(zip(new, held))])
    d = [t.to(cuda_dev) for t in (q, kc, vc, cq)]
    seq = torch.tensor(held, dtype=torch.int32, device=cuda_dev)
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = tp.kv_prefill(*d, seq_lens=seq, page_table=pt.to(cuda_dev), scale=0.125,
                                 causal=causal, out_dtype=dtype)
        assert tp.device_status() == 0
        check_attention(out, lse, ref, torch.bfloat16, dtype, "pieces")


def test_a_neighbours_rows_are_not_used(cuda_dev):
    """Packed: a request's last tile holds its neighbour's first rows; what
    stands there (NaN, infinities) does not reach it."""
    new = [70, 64, 200]
    q, k, v, cq, _, ref = _packed(new, new, 4, 2, 64, 64, torch.bfloat16, 2, True, 0.125)
    k[70:134] = float("nan")
    v[70:134] = float("inf")
    d = [t.to(cuda_dev) for t in (q, k, v, cq)]
    out, lse = tp.kv_prefill(*d, scale=0.125, out_dtype=torch.bfloat16)
    rows = list(range(70)) + list(range(134, 334))
    check_attention(out[rows], lse[rows], [x[rows] for x in ref], torch.bfloat16, torch.bfloat16,
                    "neighbour")


def test_rows_of_no_request_and_strided_views(cuda_dev):
    """Rows before the first and behind the last request stay as they were;
    q, k, v as slices of one projection; out as a slice."""
    gen = torch.Generator().manual_seed(5)
    new, T = [60, 90], 200
    qkv = (1.2 * torch.randn((T, 12, 64), generator=gen)).to(torch.bfloat16)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    cq = _cu(new, first=10)
    ref = _join([attend64(q[cq[b]:cq[b + 1]], k[cq[b]:cq[b + 1]], v[cq[b]:cq[b + 1]], 0.125,
                          _limits(n, n, True)) for b, n in enumerate(new)])
    d = qkv.to(cuda_dev)
    res = torch.full((T, 9, 64), 3.0, dtype=torch.bfloat16, device=cuda_dev)
    lse = torch.full((T, 8, 1), 3.0, device=cuda_dev)
    tp.kv_prefill(d[:, :8], d[:, 8:10], d[:, 10:], cq.to(cuda_dev), scale=0.125, out=res[:, 1:],
                  lse=lse)
    assert tp.device_status() == 0
    check_attention(res[10:160, 1:], lse[10:160], ref, torch.bfloat16, torch.bfloat16, "views")
    assert torch.all(res[:, 0] == 3) and torch.all(res[:10] == 3) and torch.all(res[160:] == 3)
    assert torch.all(lse[:10] == 3) and torch.all(lse[160:] == 3)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.7])
def test_scales_and_growing_maxima(cuda_dev, scale):
    """Keys that grow along the prompt make the running maximum climb (the
    accumulator is rescaled); a negative and a zero scale."""
    gen = torch.Generator().manual_seed(9)
    T = 640
    q = torch.randn((T, 2, 64), generator=gen).abs().to(torch.bfloat16)
    k = (torch.randn((T, 2, 64), generator=gen).abs() * torch.linspace(0, 1, T)[:, None, None])
    k, v = k.to(torch.bfloat16), torch.randn((T, 2, 64), generator=gen).to(torch.bfloat16)
    ref = attend64(q, k, v, scale, _limits(T, T, True))
    d = [t.to(cuda_dev) for t in (q, k, v, _cu([T]))]
    out, lse = tp.kv_prefill(*d, scale=scale, out_dtype=torch.bfloat16)
    check_attention(out, lse, ref, torch.bfloat16, torch.bfloat16, "scale")


def test_bad_lengths_and_pages_are_recorded(cuda_dev):
    gen = torch.Generator().manual_seed(6)
    held, new = [200, 128], [10, 20]
    kc, pt = paged_cache(held, 2, 64, torch.bfloat16, gen)
    vc = torch.randn(kc.shape, generator=gen).to(torch.bfloat16)
    q = torch.randn((30, 4, 64), generator=gen).to(torch.bfloat16)
    good = pt.clone()
    pt[0, 1] = kc.shape[0] + 7
    seq = torch.tensor(held, dtype=torch.int32)
    d = [t.to(cuda_dev) for t in (q, kc, vc, _cu(new))]
    out, lse = tp.kv_prefill(*d, seq_lens=seq.to(cuda_dev), page_table=pt.to(cuda_dev),
                             scale=0.125, out_dtype=torch.bfloat16)
    assert tp.device_status() == -6 and tp.device_status() == 0
    keep = [t for t in range(200) if not 64 <= t < 128]
    lim = [sum(t < 190 + i + 1 for t in keep) for i in range(10)]
    ref = _join([attend64(q[:10], rows_of(kc, good, 0, 200)[keep], rows_of(vc, good, 0, 200)[keep],
                          0.125, lim),
                 attend64(q[10:], rows_of(kc, good, 1, 128), rows_of(vc, good, 1, 128), 0.125,
                          _limits(20, 128, True))])
    check_attention(out, lse, ref, torch.bfloat16, torch.bfloat16, "bad page")
    # offsets past the tensor are clipped: the second request keeps its 20 rows
    cq = torch.tensor([0, 10, 31], dtype=torch.int32, device=cuda_dev)
    out2, _ = tp.kv_prefill(d[0], d[1], d[2], cq, seq_lens=seq.to(cuda_dev),
                            page_table=good.to(cuda_dev), scale=0.125, out_dtype=torch.bfloat16)
    assert tp.device_status() == -6
    assert torch.equal(out2[10:], out[10:])


def test_capture_and_streams(cuda_dev):
    new = [100, 300]
    q, k, v, cq, _, ref = _packed(new, new, 4, 2, 128, 128, torch.bfloat16, 1, True, 0.1)
    d = [t.to(cuda_dev) for t in (q, k, v, cq)]
    want, want_lse = tp.kv_prefill(*d, scale=0.1)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tp.kv_prefill(*d, scale=0.1, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tp.kv_prefill(*d, scale=0.1, out=out, lse=lse, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert tp.device_status() == 0
