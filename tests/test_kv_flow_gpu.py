"""The uncompressed key/value operators together, as a serving loop uses them,
and next to the latent ones."""
import numpy as np
import pytest
import torch

import mla_latent_kv_dim_b200 as tp
from kv_cases import attend64, check_attention, rope64, rope_table, rows_of
from mla_latent_kv_dim_b200.workloads import as_f64
from oracle import tpla_oracle as O
from parity import assert_lse_close, assert_out_close, to_np

pytestmark = pytest.mark.gpu


def test_prompts_then_decode_steps(cuda_dev):
    """Packed prompts are appended (rotated) and attended over the paged cache;
    then decode steps append one token per request and attend.  Requests of
    different lengths, one prompt in two chunks.  Every result is compared with
    attention in 64 bits over the rows that the cache holds."""
    gen = torch.Generator().manual_seed(21)
    Hq, Hkv, D, dt = 8, 2, 128, torch.bfloat16
    scale, table = D ** -0.5, rope_table(512, D)
    B, held = 3, [0, 0, 0]
    pt = torch.randperm(3 * 6 + 2, generator=gen)[:18].reshape(3, 6).to(torch.int32)
    kc = torch.full((20, 64, Hkv, D), float("nan"), dtype=dt, device=cuda_dev)
    vc = torch.full((20, 64, Hkv, D), float("nan"), dtype=dt, device=cuda_dev)
    d_pt, d_table = pt.to(cuda_dev), table.to(cuda_dev)
    stored = 0
    for new in ([70, 1, 130], [60, 0, 0], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        q = (1.5 * torch.randn((T, Hq, D), generator=gen)).to(dt)
        k = torch.randn((T, Hkv, D), generator=gen).to(dt)
        v = torch.randn((T, Hkv, D), generator=gen).to(dt)
        req = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(torch.int32)
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)]).to(torch.int32)
        qr = tp.kv_append(k.to(cuda_dev), v.to(cuda_dev), pos.to(cuda_dev), d_pt, kc, vc,
                          requests=req.to(cuda_dev), cos_sin=d_table, q=q.to(cuda_dev))
        held = [h + n for h, n in zip(held, new)]
        seq = torch.tensor(held, dtype=torch.int32, device=cuda_dev)
        cq = torch.tensor(np.cumsum([0] + new), dtype=torch.int32)
        if new == [1, 1, 1]:
            out, lse = tp.kv_decode(qr, kc, vc, seq, d_pt, scale=scale, out_dtype=dt)
            # one token a prompt is the same attention
            two, two_lse = tp.kv_prefill(qr, kc, vc, cq.to(cuda_dev), seq_lens=seq,
                                         page_table=d_pt, scale=scale, out_dtype=dt)
        else:
            out, lse = tp.kv_prefill(qr, kc, vc, cq.to(cuda_dev), seq_lens=seq, page_table=d_pt,
                                     scale=scale, out_dtype=dt)
            two = None
        assert tp.device_status() == 0
        hk, hv, hq = kc.cpu(), vc.cpu(), qr.cpu()
        # what was stored is the rotated key (f32 arithmetic, one rounding)
        wk = rope64(k, table, pos.tolist(), 0, False)
        got = torch.stack([hk[pt[r, p // 64], p % 64] for r, p in zip(req, pos)]).double()
        assert torch.all((got - wk).abs() <= 2.0 ** -8 * wk.abs() + 2.0 ** -20)
        stored += T
        assert int((~torch.isnan(hk[..., 0, 0])).sum()) == stored
        parts = [attend64(hq[cq[b]:cq[b + 1]], rows_of(hk, pt, b, held[b]),
                          rows_of(hv, pt, b, held[b]), scale,
                          [held[b] - new[b] + i + 1 for i in range(new[b])]) for b in range(B)]
        ref = [np.concatenate(x) for x in zip(*parts)]
        check_attention(out, lse, ref, dt, dt, f"{new}")
        if two is not None:
            check_attention(two, two_lse, ref, dt, dt, f"{new} as prompts")


def test_a_captured_decode_step(cuda_dev):
    """Append and attention of a step in one graph, replayed with new tokens,
    positions and lengths; a padding row leaves everything as it was."""
    gen = torch.Generator().manual_seed(4)
    B, Hq, Hkv, D, dt = 4, 4, 1, 64, torch.float16
    pt = torch.arange(8, dtype=torch.int32).reshape(4, 2).to(cuda_dev)
    kc = torch.randn((8, 64, Hkv, D), generator=gen).to(dt).to(cuda_dev)
    vc = torch.randn((8, 64, Hkv, D), generator=gen).to(dt).to(cuda_dev)
    table = rope_table(128, D).to(cuda_dev)
    new = lambda: [torch.randn((B, h, D), generator=gen).to(dt).to(cuda_dev)  # noqa: E731
                   for h in (Hq, Hkv, Hkv)]
    q, k, v = new()
    pos = torch.tensor([5, 63, 64, -1], dtype=torch.int32, device=cuda_dev)
    seq = torch.tensor([6, 64, 65, 0], dtype=torch.int32, device=cuda_dev)
    qr, out = torch.empty_like(q), torch.empty((B, Hq, D), dtype=dt, device=cuda_dev)
    lse = torch.empty((B, Hq, 1), device=cuda_dev)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=cuda_dev)

    def step():
        tp.kv_append(k, v, pos, pt, kc, vc, cos_sin=table, q=q, q_out=qr)
        tp.kv_decode(qr, kc, vc, seq, pt, scale=0.125, out=out, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for add in (1, 2):
        for t, n in zip((q, k, v), new()):
            t.copy_(n)
        pos[:3] += 1
        seq[:3] += 1
        was_q, was_k, was_v = qr[3].clone(), kc.clone(), vc.clone()
        g.replay()
        got, got_lse = out.clone(), lse.clone()
        a_k, a_v, a_q = was_k, was_v, torch.empty_like(q)
        tp.kv_append(k, v, pos, pt, a_k, a_v, cos_sin=table, q=q, q_out=a_q)
        want, want_lse = tp.kv_decode(a_q, a_k, a_v, seq, pt, scale=0.125, out_dtype=dt)
        torch.cuda.synchronize()
        assert torch.equal(kc, a_k) and torch.equal(vc, a_v)
        assert torch.equal(got[:3], want[:3]) and torch.equal(got_lse[:3], want_lse[:3])
        assert not got[3].any() and torch.all(torch.isneginf(got_lse[3]))
        # bit by bit: the row was never written and may hold NaN, unequal to itself
        assert torch.equal(qr[3].view(torch.int16), was_q.view(torch.int16))
    assert tp.device_status() == 0


def test_latent_rows_with_rotated_rope_columns(cuda_dev):
    """The latent cache as a cache of one tensor: rows [512 latent | 64 rope]
    appended with their rope columns rotated, the queries' rope columns turned
    into the absorbed query, and exact MLA decode over it."""
    gen = torch.Generator().manual_seed(6)
    H, lens, scale = 16, [130, 64, 1], 192 ** -0.5
    T = sum(lens)
    rows = torch.randn((T, 1, 576), generator=gen)
    rows[..., :512] *= torch.exp(-torch.arange(512) / 128.0)
    rows = rows.to(torch.bfloat16)
    req = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).to(torch.int32)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    pt = torch.randperm(9, generator=gen)[:9].reshape(3, 3).to(torch.int32)
    table = rope_table(200, 64)
    cache = torch.zeros((9, 64, 576), dtype=torch.bfloat16, device=cuda_dev)
    tp.kv_append(rows.to(cuda_dev), None, pos.to(cuda_dev), pt.to(cuda_dev), cache.unsqueeze(2),
                 None, requests=req.to(cuda_dev), cos_sin=table.to(cuda_dev), rope_offset=512,
                 interleaved=True)
    # the last tokens' queries: latent part given, rope part turned into place
    qa = torch.randn((3, H, 576), generator=gen).to(torch.bfloat16).to(cuda_dev)
    q_rope = torch.randn((3, H, 192), generator=gen).to(torch.bfloat16)
    last = torch.tensor([n - 1 for n in lens], dtype=torch.int32)
    tp.kv_append(rows[[129, 193, 194]].to(cuda_dev), None, last.to(cuda_dev), pt.to(cuda_dev),
                 cache.unsqueeze(2), None, cos_sin=table.to(cuda_dev), rope_offset=512,
                 interleaved=True, q=q_rope.to(cuda_dev)[..., 128:], q_out=qa[..., 512:],
                 q_rope_offset=0)
    seq = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    out, lse = tp.decode(qa, cache, seq, pt.to(cuda_dev), 1, "replicate", scale)
    torch.cuda.synchronize()
    assert tp.device_status() == 0
    want_rows = rope64(rows, table, pos.tolist(), 512, True).to(torch.bfloat16)[:, 0]
    want_q = rope64(q_rope[..., 128:], table, last.tolist(), 0, True).to(torch.bfloat16)
    per = [as_f64(r) for r in want_rows.split(lens)]
    hq = qa.cpu()
    # a rounding to the other neighbour where f32 and 64 bits part
    assert torch.all((hq[..., 512:].double() - want_q.double()).abs()
                     <= 2.0 ** -7 * want_q.double().abs() + 2.0 ** -20)
    ro, rl = O.tpla_decode_ref(as_f64(hq), per, 1, "replicate", np.float32(scale))
    assert_out_close(to_np(out), ro, what="latent")
    assert_lse_close(to_np(lse), rl)


def test_per_head_form_of_a_latent_prompt(cuda_dev):
    """MLA's prompt attention in its two forms: absorbed over the latent rows
    (tpla_prefill, then the V up-projection), and per head over the projected
    keys and values (tpla_kv_prefill, 128 + 64 and 128 columns).  In exact
    arithmetic they are the same function; keys, values and absorbed queries
    are each rounded once to bf16, so twice the parity bar."""
    gen = torch.Generator().manual_seed(13)
    T, H, scale = 150, 16, 192 ** -0.5
    c = torch.randn((T, 512), generator=gen, dtype=torch.float64)
    c = (c / c.pow(2).mean(1, keepdim=True).sqrt()).to(torch.bfloat16).double()
    rope = torch.randn((T, 64), generator=gen).to(torch.bfloat16).double()
    wk = (torch.randn((H, 512, 128), generator=gen, dtype=torch.float64) * 0.04).to(torch.bfloat16).double()
    wv = (torch.randn((H, 512, 128), generator=gen, dtype=torch.float64) * 0.04).to(torch.bfloat16)
    qn = torch.randn((T, H, 128), generator=gen).to(torch.bfloat16).double()
    qr = torch.randn((T, H, 64), generator=gen).to(torch.bfloat16).double()
    bf = lambda t: t.to(torch.bfloat16).to(cuda_dev)  # noqa: E731
    # absorbed
    qa = torch.cat([torch.einsum("thd,hjd->thj", qn, wk), qr], -1)
    cache = torch.zeros((3, 64, 576), dtype=torch.bfloat16, device=cuda_dev)
    row = torch.tensor([2, 0, 1], dtype=torch.int32, device=cuda_dev)
    lat, lse_a = tp.prefill(bf(qa), torch.cat([c, rope], -1).float().to(cuda_dev), 0, row, cache,
                            eps=0.0, scale=scale)
    y_a = tp.vup_combine(lat, wv.to(cuda_dev))
    # per head
    k = torch.cat([torch.einsum("tj,hjd->thd", c, wk), rope[:, None].expand(T, H, 64)], -1)
    v = torch.einsum("tj,hjd->thd", c, wv.double())
    cu = torch.tensor([0, T], dtype=torch.int32, device=cuda_dev)
    y_p, lse_p = tp.kv_prefill(bf(torch.cat([qn, qr], -1)), bf(k), bf(v), cu, scale=scale)
    torch.cuda.synchronize()
    assert tp.device_status() == 0
    assert_out_close(to_np(y_p), to_np(y_a), factor=2.0, what="two forms")
    assert_lse_close(to_np(lse_p), to_np(lse_a), factor=2.0)
