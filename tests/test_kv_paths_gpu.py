"""GPU tests of the kv calls as a caller may combine them: rows on 16-byte
boundaries only, caches whose offsets pass 32 bits, very many requests, two
calls at once, library-managed workspaces, equal results of equal calls.
Bounds are those of kv_cases.check_attention."""
import ctypes

import numpy as np
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import attend64, check_attention, paged_cache, rows_of
from mla_latent_kv_dim_b200 import _native as N

pytestmark = pytest.mark.gpu


def _rows(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32)


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16),
                                             (torch.float16, torch.float32)])
def test_rows_on_16_byte_boundaries(cuda_dev, dtype, out_dtype):
    """Every tensor is a view whose rows begin 16 bytes behind a 32-byte
    boundary; what lies between the rows keeps its values."""
    gen = torch.Generator().manual_seed(1)
    lens, Hq, Hkv, D, scale = [70, 1, 200], 4, 2, 64, 0.125
    T = sum(lens)

    def view(heads, type_=dtype):
        pad = 8 if type_ != torch.float32 else 4
        whole = torch.randn((T, heads, D + 2 * pad), generator=gen).to(type_).to(cuda_dev)
        part = whole[:, :, pad:pad + D]
        assert part.data_ptr() % 32 == 16
        return whole, part

    (_, q), (_, k), (_, v) = view(Hq), view(Hkv), view(Hkv)
    whole, out = view(Hq, out_dtype)
    before = whole.clone()
    cu = _rows(lens)
    _, lse = tp.kv_prefill(q, k, v, cu.to(cuda_dev), scale=scale, out=out)
    parts = [attend64(q[a:z].cpu(), k[a:z].cpu(), v[a:z].cpu(), scale, range(1, z - a + 1))
             for a, z in zip(cu[:-1], cu[1:])]
    ref = [np.concatenate(x) for x in zip(*parts)]
    check_attention(out, lse, ref, dtype, out_dtype, "prefill")
    pad = (whole.shape[2] - D) // 2
    assert torch.equal(whole[:, :, :pad], before[:, :, :pad])
    assert torch.equal(whole[:, :, pad + D:], before[:, :, pad + D:])

    kc, pt = paged_cache(lens, Hkv, D, dtype, gen)
    vc = torch.randn(kc.shape, generator=gen).to(dtype)
    B = len(lens)
    _, lse = tp.kv_decode(q[:B], kc.to(cuda_dev), vc.to(cuda_dev),
                          torch.tensor(lens, dtype=torch.int32, device=cuda_dev),
                          pt.to(cuda_dev), scale, out[:B])
    parts = [attend64(q[b:b + 1].cpu(), rows_of(kc, pt, b, n), rows_of(vc, pt, b, n), scale, [n])
             for b, n in enumerate(lens)]
    check_attention(out[:B], lse, [np.concatenate(x) for x in zip(*parts)], dtype, out_dtype,
                    "decode")
    assert tp.device_status() == 0


def test_offsets_past_32_bits(cuda_dev):
    """A pool of 2^32 + values: the request's pages are its first and last,
    and lie over 2^31 values (2^32 bytes) apart."""
    Hkv, D, scale = 4, 64, 0.125
    blocks = (1 << 32) // (64 * Hkv * D) + 8
    kc = torch.empty((blocks, 64, Hkv, D), dtype=torch.bfloat16, device=cuda_dev)
    vc = torch.empty_like(kc)
    pages = [blocks - 1, 0, blocks // 2 + 3, blocks - 2]
    gen = torch.Generator().manual_seed(2)
    T, Hq = 200, 8
    k, v = (torch.randn((T, Hkv, D), generator=gen).bfloat16() for _ in range(2))
    q = torch.randn((T, Hq, D), generator=gen).bfloat16()
    pt = torch.tensor([pages], dtype=torch.int32, device=cuda_dev)
    dq, dk, dv = (t.to(cuda_dev) for t in (q, k, v))
    tp.kv_append(dk, dv, torch.arange(T, dtype=torch.int32, device=cuda_dev), pt, kc, vc,
                 requests=torch.zeros(T, dtype=torch.int32, device=cuda_dev))
    for cache, rows in ((kc, dk), (vc, dv)):
        assert torch.equal(cache[pages].reshape(-1, Hkv, D)[:T], rows)
    n = torch.tensor([T], dtype=torch.int32, device=cuda_dev)
    ref = attend64(q, k, v, scale, range(1, T + 1))
    out, lse = tp.kv_prefill(dq, kc, vc, _rows([T]).to(cuda_dev), seq_lens=n, page_table=pt,
                             scale=scale)
    check_attention(out, lse, ref, torch.bfloat16, torch.float32, "prefill")
    out, lse = tp.kv_decode(dq[-1:], kc, vc, n, pt, scale)
    check_attention(out, lse, [x[-1:] for x in ref], torch.bfloat16, torch.float32, "decode")
    # a contiguous cache whose second request begins past 2^31 values
    rows = (1 << 31) // (Hkv * D) + 64
    flat = kc.view(-1, Hkv, D)[:2 * rows].view(2, rows, Hkv, D)
    flat_v = vc.view(-1, Hkv, D)[:2 * rows].view(2, rows, Hkv, D)
    tp.kv_append(dk, dv, torch.arange(T, dtype=torch.int32, device=cuda_dev), None, flat, flat_v,
                 requests=torch.ones(T, dtype=torch.int32, device=cuda_dev))
    out, lse = tp.kv_decode(dq[-2:], flat, flat_v,
                            torch.tensor([0, T], dtype=torch.int32, device=cuda_dev), None, scale)
    check_attention(out[1:], lse[1:], [x[-1:] for x in ref], torch.bfloat16, torch.float32, "flat")
    assert not out[0].any() and tp.device_status() == 0


def test_very_many_requests(cuda_dev):
    """More requests than threads of a block or slices of the work, a third of
    them empty, all on the same few pages."""
    gen = torch.Generator().manual_seed(3)
    B, Hq, Hkv, D, scale = 4099, 2, 1, 64, 0.2
    kc = torch.randn((7, 64, Hkv, D), generator=gen).half()
    vc = torch.randn((7, 64, Hkv, D), generator=gen).half()
    lens = (torch.arange(B, dtype=torch.int32) * 37 % 150 - 50).clamp(min=0)
    pt = torch.stack([(torch.arange(B) + i) % 7 for i in range(2)], 1).int()
    q = torch.randn((B, Hq, D), generator=gen).half()
    out, lse = tp.kv_decode(*(t.to(cuda_dev) for t in (q, kc, vc, lens, pt)), scale)
    parts = [attend64(q[b:b + 1], rows_of(kc, pt, b, n), rows_of(vc, pt, b, n), scale, [n])
             for b, n in enumerate(lens.tolist())]
    check_attention(out, lse, [np.concatenate(x) for x in zip(*parts)], torch.float16,
                    torch.float32, "decode")
    assert tp.device_status() == 0


def test_two_calls_at_once_and_equal_results(cuda_dev):
    """Calls on two streams, each with workspaces of its own, and repeated
    calls give the same bits."""
    gen = torch.Generator().manual_seed(4)
    lens, Hq, Hkv, D, scale = [900, 17, 2500, 0, 640], 16, 2, 128, 0.09
    kc, pt = paged_cache(lens, Hkv, D, torch.bfloat16, gen)
    vc = torch.randn(kc.shape, generator=gen).bfloat16()
    new = [50, 17, 300, 0, 1]
    T = sum(new)
    q = torch.randn((T, Hq, D), generator=gen).bfloat16().to(cuda_dev)
    kc, vc, pt = kc.to(cuda_dev), vc.to(cuda_dev), pt.to(cuda_dev)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    cu = _rows(new).to(cuda_dev)

    def both():
        return (*tp.kv_prefill(q, kc, vc, cu, seq_lens=n, page_table=pt, scale=scale),
                *tp.kv_decode(q[:5], kc, vc, n, pt, scale))

    want = both()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(both())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert tp.device_status() == 0


def test_library_managed_workspaces(cuda_dev):
    """Through the C entry points without a workspace, on a stream."""
    gen = torch.Generator().manual_seed(5)
    lens, Hq, Hkv, D, scale = [3000, 5], 4, 1, 64, 0.125
    kc, pt = paged_cache(lens, Hkv, D, torch.float16, gen)
    vc = torch.randn(kc.shape, generator=gen).half()
    q = torch.randn((40, Hq, D), generator=gen).half().to(cuda_dev)
    kc, vc, pt = kc.to(cuda_dev), vc.to(cuda_dev), pt.to(cuda_dev)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    cu = _rows([36, 4]).to(cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def p(t):
        return None if t is None else ctypes.byref(N.desc(t))

    out = torch.empty((40, Hq, D), device=cuda_dev)
    lse = torch.empty((40, Hq, 1), device=cuda_dev)
    handle = ctypes.c_void_p(side.cuda_stream)
    assert tp.lib().tpla_kv_prefill(p(q), p(kc), p(vc), p(cu), None, p(n), p(pt), 1, scale, p(out),
                                    p(lse), None, 0, handle) == 0
    one, one_lse = torch.empty((2, Hq, D), device=cuda_dev), torch.empty((2, Hq, 1), device=cuda_dev)
    assert tp.lib().tpla_kv_decode(p(q[:2]), p(kc), p(vc), p(n), p(pt), scale, p(one), p(one_lse),
                                   None, 0, handle) == 0
    side.synchronize()
    a, b = tp.kv_prefill(q, kc, vc, cu, seq_lens=n, page_table=pt, scale=scale)
    assert torch.equal(out, a) and torch.equal(lse, b)
    a, b = tp.kv_decode(q[:2], kc, vc, n, pt, scale)
    assert torch.equal(one, a) and torch.equal(one_lse, b)
    # too short or misaligned: refused before a launch
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=cuda_dev)
    before = tp.launch_count()
    for at, size in ((ws.data_ptr(), 16), (ws.data_ptr() + 8, 1 << 23)):
        assert tp.lib().tpla_kv_decode(p(q[:2]), p(kc), p(vc), p(n), p(pt), scale, p(one),
                                       p(one_lse), at, size, handle) == -4
    # a workspace that is no plain run of memory is not used
    sparse = ws[:1].expand(1 << 24)
    a2, _ = tp.kv_decode(q[:2], kc, vc, n, pt, scale, workspace=sparse)
    assert tp.launch_count() == before + 2 and torch.equal(a, a2)
    assert tp.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_of_either_exponential(cuda_dev, dtype):
    """A row whose sum is one key of score 0 and 16 r keys of score s, these in
    every column of a key tile in turn: its log-sum-exp is
    ln(1 + 16 r e^s).  Of the weights' relative error (2.2e-7, 2 ulp of the
    exponential unit being 2.4e-7) and that of s / ln 2 in f32, |s| 2^-23 (two
    roundings), the logarithm keeps at most the same absolute error; its own
    rounding is a few 2^-24 of 1 + |lse|."""
    r, D = 40, 64
    scores = [-0.25 * i for i in range(60)] + [0.0, -40.0, -80.0]
    far = -256.0  # e^-256 is 0 beside any of them
    q = torch.zeros((1, 1, D), dtype=dtype)
    q[..., 0] = 1
    for column in range(8):
        rows = []
        for s in scores:
            k = torch.full((64 * (r + 1),), far)
            k[0] = 0
            k[64:].view(-1, 64)[:, [column + 8 * i for i in range(8)]] = s
            k[64:].view(-1, 64)[:, [(column + 1) % 8 + 8 * i for i in range(8)]] = s
            rows.append(k)
        B, L = len(scores), 64 * (r + 1)
        k = torch.zeros((B * L, 1, D), dtype=dtype)
        k[:, 0, 0] = torch.cat(rows).to(dtype)
        v = torch.ones((B * L, 1, D), dtype=dtype)
        out, lse = tp.kv_prefill(q.expand(B, 1, D).contiguous().to(cuda_dev), k.to(cuda_dev),
                                 v.to(cuda_dev), _rows([1] * B).to(cuda_dev),
                                 _rows([L] * B).to(cuda_dev), scale=1.0)
        s = torch.tensor(scores, dtype=torch.float64)
        want = torch.log1p(16 * r * s.exp())
        err = (lse[:, 0, 0].double().cpu() - want).abs()
        tol = 2.4e-7 + s.abs() * 2.0 ** -23 + (1 + want) * 2.0 ** -22
        assert (err <= tol).all(), (column, (err / tol).max())
        # values of 1: what the rounding of the weights leaves of the sum
        half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
        share = 1 - torch.exp(-want)  # what the rounded weights have of the sum
        # (half a step each, in fp16 below 2^-14 the absolute 2^-25), and less
        # than a unit in the last place, 2^-23 of a sum near 1, that each of the
        # 4 (r + 1) matrix products of 16 keys drops as it adds into f32
        tol = half * share + 4 * (r + 1) * 2.0 ** -23 + 1e-6
        if dtype == torch.float16:
            tol = tol + 16 * r * 2.0 ** -25
        assert ((out.double().cpu()[:, 0] - 1).abs() <= tol[:, None]).all()
    assert tp.device_status() == 0


@pytest.mark.parametrize("T", [2700, 2900])
def test_one_prompt_of_many_heads(cuda_dev, T):
    """Keys and values beyond the L2: heads one after another, tiles in pairs
    (an odd and an even number of them).  Some rows of some heads against 64
    bits, and every row of every head against the same call for those heads
    alone, bit by bit."""
    gen = torch.Generator(device=cuda_dev).manual_seed(6)
    H, D, scale = 148, 64, 0.125
    q, k, v = (torch.randn((T, H, D), generator=gen, device=cuda_dev).bfloat16() for _ in range(3))
    cu = _rows([T]).to(cuda_dev)
    out, lse = tp.kv_prefill(q, k, v, cu, scale=scale)
    rows, heads = list(range(0, T, 97)) + [T - 1], [0, 1, 73, 146, 147]
    ref = attend64(q[rows][:, heads].cpu(), k[:, heads].cpu(), v[:, heads].cpu(), scale,
                   [r + 1 for r in rows])
    check_attention(out[rows][:, heads], lse[rows][:, heads], ref, torch.bfloat16, torch.float32,
                    "sample")
    for h in range(0, H, 37):
        part = slice(h, h + 37)
        a, b = tp.kv_prefill(q[:, part], k[:, part], v[:, part], cu, scale=scale)
        assert torch.equal(a, out[:, part]) and torch.equal(b, lse[:, part])
    assert tp.device_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_no_number(cuda_dev, bad):
    """Its own rows are NaN, every other row keeps its bits: in a prompt, in a
    prompt cut along its keys, and in a decode step split over the GPU."""
    gen = torch.Generator().manual_seed(8)
    lens, Hq, Hkv, D, scale = [5000, 300], 8, 2, 128, 0.09
    kc, pt = paged_cache(lens, Hkv, D, torch.bfloat16, gen)
    vc = torch.randn(kc.shape, generator=gen).bfloat16()
    kc, vc, pt = kc.to(cuda_dev), vc.to(cuda_dev), pt.to(cuda_dev)
    q = torch.randn((90, Hq, D), generator=gen).bfloat16().to(cuda_dev)
    worse = q.clone()
    worse[0, 3, 5] = worse[77, 0, 100] = bad
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    cu = _rows([60, 30]).to(cuda_dev)
    for call in (lambda x: tp.kv_prefill(x, kc, vc, cu, seq_lens=n, page_table=pt, scale=scale),
                 lambda x: tp.kv_prefill(x[:30], kc[0], vc[0], _rows([30]).to(cuda_dev),
                                         _rows([64]).to(cuda_dev), scale=scale),
                 lambda x: tp.kv_decode(x[:2], kc, vc, n, pt, scale)):
        want, want_lse = call(q)
        out, lse = call(worse)
        hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=cuda_dev)
        hit[0, 3] = True
        if out.shape[0] > 77:
            hit[77, 0] = True
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    assert tp.device_status() == 0
