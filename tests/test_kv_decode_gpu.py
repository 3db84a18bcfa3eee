"""GPU parity of tpla_kv_decode (one new token per request over the
uncompressed cache) against attention in 64 bits; the bounds are derived in
kv_cases.check_attention."""
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import attend64, check_attention, paged_cache, rows_of

pytestmark = pytest.mark.gpu


def _reference(q, kc, vc, pt, lens, scale):
    parts = [attend64(q[b:b + 1], rows_of(kc, pt, b, n), rows_of(vc, pt, b, n), scale, [n])
             for b, n in enumerate(lens)]
    return [__import__("numpy").concatenate(x) for x in zip(*parts)]


def _case(lens, Hq, Hkv, Dk, Dv, dtype, seed, paged=True, heads_first=False, gain=1.5):
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    if paged:
        kc, pt = paged_cache(lens, Hkv, Dk, dtype, gen, heads_first=heads_first)
        vc = torch.randn(kc.shape[:3] + (Dv,), generator=gen).to(dtype)
    else:
        kc = torch.randn((B, max(lens) + 3, Hkv, Dk), generator=gen).to(dtype)
        vc = torch.randn((B, max(lens) + 3, Hkv, Dv), generator=gen).to(dtype)
        pt = None
    q = (gain * torch.randn((B, Hq, Dk), generator=gen)).to(dtype)
    return q, kc, vc, pt


def _on(dev, *ts):
    return [None if t is None else
            torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=dev).copy_(t) for t in ts]


RAGGED = [0, 1, 63, 64, 65, 300, 129, 1000]


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("Hq,Hkv,dtype", [
    (1, 1, torch.bfloat16), (3, 3, torch.float16), (8, 2, torch.bfloat16), (14, 2, torch.float16),
    (16, 1, torch.bfloat16), (40, 2, torch.bfloat16), (64, 1, torch.float16),
    (100, 1, torch.bfloat16), (260, 2, torch.bfloat16)])
def test_ragged(cuda_dev, Dk, Dv, Hq, Hkv, dtype):
    lens = RAGGED if Hq < 64 else [0, 1, 65, 300]
    q, kc, vc, pt = _case(lens, Hq, Hkv, Dk, Dv, dtype, seed=Hq + Dk)
    seq = torch.tensor(lens, dtype=torch.int32)
    scale = Dk ** -0.5
    out, lse = tp.kv_decode(*_on(cuda_dev, q, kc, vc, seq, pt), scale=scale, out_dtype=dtype)
    assert tp.device_status() == 0
    check_attention(out, lse, _reference(q, kc, vc, pt, lens, scale), dtype, dtype, "ragged")
    assert not out[0].any()


@pytest.mark.parametrize("paged,heads_first", [(True, True), (False, False)])
def test_layouts_and_f32_output(cuda_dev, paged, heads_first):
    lens = [5, 64, 200, 1]
    q, kc, vc, pt = _case(lens, 8, 4, 128, 128, torch.bfloat16, 5, paged, heads_first)
    # queries and results as slices of wider rows
    wide = torch.zeros((4, 8, 200), dtype=torch.bfloat16)
    wide[..., 16:144] = q
    dq = wide.to(cuda_dev)[..., 16:144]
    res = torch.full((4, 10, 136), 3.0, device=cuda_dev)
    seq = torch.tensor(lens, dtype=torch.int32)
    ds = _on(cuda_dev, kc, vc, seq, pt)
    out, lse = tp.kv_decode(dq, *ds, scale=0.1, out=res[:, 1:9, :128])
    assert tp.device_status() == 0
    check_attention(out, lse, _reference(q, kc, vc, pt, lens, 0.1), torch.bfloat16, torch.float32,
                    "layout")
    assert torch.all(res[:, 0] == 3) and torch.all(res[:, 9] == 3) and torch.all(res[..., 128:] == 3)


@pytest.mark.parametrize("lens,Hq,Hkv", [([20000], 4, 2), ([9000, 1, 3, 0, 5000], 16, 2),
                                         ([64] * 300, 2, 1), ([1] * 70, 4, 4)])
def test_split_and_join(cuda_dev, lens, Hq, Hkv):
    """Long requests over many SMs, many short ones in one SM's slice."""
    q, kc, vc, pt = _case(lens, Hq, Hkv, 64, 64, torch.bfloat16, 11)
    seq = torch.tensor(lens, dtype=torch.int32)
    out, lse = tp.kv_decode(*_on(cuda_dev, q, kc, vc, seq, pt), scale=0.125,
                            out_dtype=torch.bfloat16)
    assert tp.device_status() == 0
    check_attention(out, lse, _reference(q, kc, vc, pt, lens, 0.125), torch.bfloat16,
                    torch.bfloat16, "split")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(cuda_dev, scale):
    lens = [77, 130]
    q, kc, vc, pt = _case(lens, 6, 2, 64, 64, torch.bfloat16, 4, gain=0.5)
    seq = torch.tensor(lens, dtype=torch.int32)
    out, lse = tp.kv_decode(*_on(cuda_dev, q, kc, vc, seq, pt), scale=scale,
                            out_dtype=torch.bfloat16)
    check_attention(out, lse, _reference(q, kc, vc, pt, lens, scale), torch.bfloat16,
                    torch.bfloat16, "scale")


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq", [4, 40, 64])
def test_rows_behind_the_last_token_are_not_used(cuda_dev, junk, Hq):
    lens = [1, 70, 128, 16]
    q, kc, vc, pt = _case(lens, Hq, 1, 64, 64, torch.bfloat16, 6)
    seq = torch.tensor(lens, dtype=torch.int32)
    ref = _reference(q, kc, vc, pt, lens, 0.125)
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[pt[b, t // 64], t % 64] = True
    kc[~used] = junk
    vc[~used] = junk
    out, lse = tp.kv_decode(*_on(cuda_dev, q, kc, vc, seq, pt), scale=0.125,
                            out_dtype=torch.bfloat16)
    check_attention(out, lse, ref, torch.bfloat16, torch.bfloat16, "junk")


def test_bad_pages_and_lengths_count_as_absent(cuda_dev):
    """A page id outside the pool: its tokens are absent.  A length beyond the
    table: clipped.  Both are recorded; the other requests are unaffected."""
    lens = [200, 100, 128]
    q, kc, vc, pt = _case(lens, 4, 2, 64, 64, torch.bfloat16, 9)
    good = pt.clone()
    pt[0, 1] = kc.shape[0]
    pt[1, 0] = -5
    seq = torch.tensor([200, 100, 64 * pt.shape[1] + 1], dtype=torch.int32)
    pt[2, 2:] = -1
    out, lse = tp.kv_decode(*_on(cuda_dev, q, kc, vc, seq, pt), scale=0.125,
                            out_dtype=torch.bfloat16)
    assert tp.device_status() == -6 and tp.device_status() == 0
    keep = [[t for t in range(200) if not 64 <= t < 128], list(range(64, 100)), list(range(128))]
    for b in range(3):
        k = rows_of(kc, good, b, lens[b])[keep[b]]
        v = rows_of(vc, good, b, lens[b])[keep[b]]
        ref = attend64(q[b:b + 1], k, v, 0.125, [len(keep[b])])
        check_attention(out[b:b + 1], lse[b:b + 1], ref, torch.bfloat16, torch.bfloat16, f"b{b}")


def test_streams_capture_and_workspaces(cuda_dev):
    """On a stream of its own, captured and replayed on new inputs, with the
    caller's workspace; library-managed and caller workspaces agree."""
    lens = [700, 64, 1]
    q, kc, vc, pt = _case(lens, 8, 2, 128, 128, torch.bfloat16, 12)
    seq = torch.tensor(lens, dtype=torch.int32)
    dq, dk, dv, ds, dp = _on(cuda_dev, q, kc, vc, seq, pt)
    want, want_lse = tp.kv_decode(dq, dk, dv, ds, dp, scale=0.1)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    tp.kv_decode(dq, dk, dv, ds, dp, scale=0.1, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tp.kv_decode(dq, dk, dv, ds, dp, scale=0.1, out=out, lse=lse, workspace=ws)
    out.zero_()
    ds.copy_(torch.tensor([64, 1, 0], dtype=torch.int32))
    g.replay()
    again, again_lse = tp.kv_decode(dq, dk, dv, ds, dp, scale=0.1)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, again_lse) and not torch.equal(out, want)
    assert tp.device_status() == 0
