"""GPU parity of tpla_kv_append: keys and values stored in the cache with the
position rotation on the way, against the rotation in 64 bits.

The kernel turns a pair in f32 (two products and a sum: at most 1.5 * 2^-23 of
|a| + |b|, with |cos|, |sin| <= 1) and rounds once to the cache's type (half a
step of the value).  Columns that are not rotated are rounded only, so they
are equal.  What the call does not store is bit-identical."""
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import EPS, paged_cache, rope64, rope_table

pytestmark = pytest.mark.gpu


def _close(got, want, src, dtype, rot_cols):
    """got: stored rows; want: 64-bit rows; src: what went in (64 bits)."""
    got = got.double().cpu()
    plain = [c for c in range(want.shape[-1]) if c not in rot_cols]
    assert torch.equal(got[..., plain], want[..., plain].to(dtype).double())
    size = src.abs().amax(-1, keepdim=True) * 2
    tol = EPS[dtype] * want.abs() + 1.5 * 2.0 ** -23 * size * (1 + EPS[dtype])
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert torch.all((got - want).abs() <= tol), ((got - want).abs() / tol).max()


CASES = [
    # dtype, source, Hkv, Hq, Dk, Dv, rot, off, interleaved, paged, heads_first
    (torch.bfloat16, torch.bfloat16, 2, 6, 128, 128, 128, 0, False, True, False),
    (torch.bfloat16, torch.float32, 3, 3, 64, 64, 32, 32, True, True, True),
    (torch.float16, torch.float16, 1, 7, 192, 128, 64, 128, True, True, False),
    (torch.float16, torch.float32, 5, 5, 128, 64, 64, 0, False, False, False),
    (torch.bfloat16, torch.bfloat16, 1, 4, 576, 0, 64, 512, True, True, False),
    (torch.bfloat16, torch.bfloat16, 4, 4, 40, 24, 16, 8, False, True, False),
]


@pytest.mark.parametrize("case", CASES)
def test_rows_and_queries(cuda_dev, case):
    dtype, src, Hkv, Hq, Dk, Dv, rot, off, inter, paged, hf = case
    gen = torch.Generator().manual_seed(Hkv * 100 + Dk)
    lens = [1, 130, 64, 257]
    new = [1, 3, 64, 2]  # the last tokens of each request
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).to(torch.int32)
    req = torch.repeat_interleave(torch.arange(4), torch.tensor(new)).to(torch.int32)
    T = len(pos)
    # a permutation: tokens of a call may come in any order
    order = torch.randperm(T, generator=gen)
    pos, req = pos[order], req[order]
    if paged:
        kc, pt = paged_cache(lens, Hkv, Dk, dtype, gen, heads_first=hf)
        vc = torch.randn((kc.shape[0], 64, Hkv, Dv), generator=gen).to(dtype) if Dv else None
    else:
        kc, pt = torch.randn((4, 257, Hkv, Dk), generator=gen).to(dtype), None
        vc = torch.randn((4, 257, Hkv, Dv), generator=gen).to(dtype)
    k = torch.randn((T, Hkv, Dk), generator=gen).to(src)
    v = torch.randn((T, Hkv, Dv), generator=gen).to(src) if Dv else None
    q = torch.randn((T, Hq, Dk), generator=gen).to(dtype)
    table = rope_table(300, rot)
    d = lambda t: None if t is None else t.to(cuda_dev)  # noqa: E731
    dk = torch.empty_strided(kc.shape, kc.stride(), dtype=dtype, device=cuda_dev).copy_(kc)
    dv = d(vc)
    out = tp.kv_append(d(k), d(v), d(pos), d(pt), dk, dv, requests=d(req), cos_sin=d(table),
                       rope_offset=off, interleaved=inter, q=d(q))
    torch.cuda.synchronize()
    assert tp.device_status() == 0
    cols = range(off, off + rot)
    wk = rope64(k, table, pos.tolist(), off, inter)
    wq = rope64(q, table, pos.tolist(), off, inter)
    block = torch.tensor([int(pt[r, p // 64]) if paged else int(r) for r, p in zip(req, pos)])
    row = pos.long() % 64 if paged else pos.long()
    _close(dk.cpu()[block, row], wk, k.double(), dtype, cols)
    _close(out, wq, q.double(), dtype, cols)
    if Dv:
        assert torch.equal(dv.cpu()[block, row], v.to(dtype))
    for got, was in ((dk, kc), (dv, vc)):
        if was is not None:
            got, was = got.cpu().clone(), was.clone()
            got[block, row] = 0
            was[block, row] = 0
            assert torch.equal(got, was), "rows that no token names changed"


def test_in_place_queries_strided_views_and_no_rotation(cuda_dev):
    """q rotated in place; rope columns of wider queries into those of another
    buffer; and an append without a table."""
    gen = torch.Generator().manual_seed(3)
    kc, pt = paged_cache([65, 10], 2, 64, torch.bfloat16, gen)
    vc = kc.clone()
    k = torch.randn((2, 2, 64), generator=gen).to(torch.bfloat16)
    pos = torch.tensor([64, 9], dtype=torch.int32)
    table = rope_table(80, 64)
    q = torch.randn((2, 4, 64), generator=gen).to(torch.bfloat16)
    args = [t.to(cuda_dev) for t in (k, k, pos, pt, kc, vc)]
    dq = q.to(cuda_dev)
    far = tp.kv_append(*args, cos_sin=table.to(cuda_dev), q=dq)
    near = tp.kv_append(*args, cos_sin=table.to(cuda_dev), q=dq, q_out=dq)
    assert near.data_ptr() == dq.data_ptr() and torch.equal(far, near)
    # q's columns 64..127 of 128 into columns 512..575 of 576
    wide = torch.randn((2, 4, 128), generator=gen).to(torch.bfloat16)
    wide[..., 64:] = q
    to = torch.full((2, 4, 576), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    tp.kv_append(*args, cos_sin=table.to(cuda_dev), q=wide.to(cuda_dev)[..., 64:],
                 q_out=to[..., 512:])
    assert torch.equal(to[..., 512:], far) and torch.all(to[..., :512] == 7)
    tp.kv_append(*args)
    torch.cuda.synchronize()
    blocks = [int(pt[0, 1]), int(pt[1, 0])]
    assert torch.equal(args[4].cpu()[blocks, [0, 9]], k)
    assert tp.device_status() == 0


@pytest.mark.parametrize("bad", ["position", "page", "request", "table"])
def test_padding_and_bad_rows(cuda_dev, bad):
    """Padding rows are skipped in silence; a row that cannot be stored leaves
    everything of its own as it was and is recorded; the others are stored."""
    gen = torch.Generator().manual_seed(8)
    kc, pt = paged_cache([64, 128], 2, 64, torch.bfloat16, gen)
    vc = kc.clone()
    pos = torch.tensor([10, -1, 100], dtype=torch.int32)
    req = torch.tensor([0, 0, 1], dtype=torch.int32)
    table = rope_table(128, 64)
    k = torch.randn((3, 2, 64), generator=gen).to(torch.bfloat16)
    q_out = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device=cuda_dev)

    def run():
        a, b = kc.to(cuda_dev), vc.to(cuda_dev)
        tp.kv_append(k.to(cuda_dev), k.to(cuda_dev), pos.to(cuda_dev), pt.to(cuda_dev), a, b,
                     requests=req.to(cuda_dev), cos_sin=table.to(cuda_dev), q=k.to(cuda_dev),
                     q_out=q_out)
        torch.cuda.synchronize()
        return a.cpu(), b.cpu()

    a, b = run()
    assert tp.device_status() == 0
    assert torch.all(q_out[1] == 5) and not torch.all(q_out[2] == 5)
    first = int(pt[0, 0])
    assert torch.equal(b[first, 10], k[0])
    q_out.fill_(5.0)
    if bad == "position":
        pos[2] = 128
    elif bad == "page":
        pt[1, 1] = kc.shape[0]
    elif bad == "request":
        req[2] = 2
    else:
        table = table[:100]
    a, b = run()
    assert tp.device_status() == -6 and tp.device_status() == 0
    assert torch.equal(b[first, 10], k[0]) and torch.all(q_out[2] == 5)
    b[first, 10] = vc[first, 10]
    assert torch.equal(b, vc)


def test_no_tokens(cuda_dev):
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=cuda_dev)
    c = torch.zeros((1, 64, 2, 64), dtype=torch.bfloat16, device=cuda_dev)
    n = torch.empty((0,), dtype=torch.int32, device=cuda_dev)
    pt = torch.zeros((0, 1), dtype=torch.int32, device=cuda_dev)
    tp.kv_append(e, e, n, pt, c, c.clone())
    assert tp.device_status() == 0 and not c.any()
