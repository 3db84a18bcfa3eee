"""Shared pieces of the tests of the uncompressed key/value operators: cache
layouts and plain implementations in 64 bits (no code of the package)."""
from __future__ import annotations

import math

import numpy as np
import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def paged_cache(lens, Hkv, D, dtype, gen, extra=3, heads_first=False, spare_pages=0):
    """A pool of 64-token pages in random order and each request's rows:
    (cache [blocks, 64, Hkv, D], page table [B, max_pages] with -1 where a
    request has no page)."""
    pages = [(n + 63) // 64 for n in lens]
    total = sum(pages) + extra
    shape = (total, Hkv, 64, D) if heads_first else (total, 64, Hkv, D)
    cache = torch.randn(shape, generator=gen).to(dtype)
    if heads_first:
        cache = cache.transpose(1, 2)
    order = torch.randperm(total, generator=gen)
    table = torch.full((len(lens), max(1, max(pages) + spare_pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return cache, table


def rows_of(cache, table, b, n):
    """Request b's first n rows [n, Hkv, D] in 64 bits."""
    if table is None:
        return cache[b, :n].double()
    pages = table[b, :(n + 63) // 64].long()
    return cache[pages].reshape(-1, *cache.shape[2:])[:n].double()


def attend64(q, k, v, scale, limit):
    """Attention of q [T, Hq, Dk] over k, v [L, Hkv, D] in 64 bits, token i
    over its first limit[i] keys: (out, lse, sum_j p_j |v_j|, sum_j |v_j|);
    errors of the weights scale with the last two."""
    T, Hq, _ = q.shape
    g = Hq // k.shape[1]
    out = np.zeros((T, Hq, v.shape[2]))
    mag, vsum = np.zeros_like(out), np.zeros_like(out)
    lse = np.full((T, Hq), -np.inf)
    q, k, v = (x.double().numpy() for x in (q, k, v))
    for h in range(Hq):
        s = scale * (q[:, h] @ k[:, h // g].T)
        for i in range(T):
            n = int(limit[i])
            if n <= 0:
                continue
            x = s[i, :n]
            m = x.max()
            e = np.exp(x - m)
            z = e.sum()
            lse[i, h] = m + math.log(z)
            out[i, h] = (e / z) @ v[:n, h // g]
            mag[i, h] = (e / z) @ np.abs(v[:n, h // g])
            vsum[i, h] = np.abs(v[:n, h // g]).sum(0)
    return out, lse, mag, vsum


def check_attention(out, lse, ref, dtype, out_dtype, what):
    """Bounds from the roundings alone.

    out: each weight is rounded once to the input type (half a step, EPS) in
    the numerator and in the sum that divides it, so the error is at most
    2 EPS sum_j p_j |v_j|; the result is rounded to the output type (EPS of
    its value).  fp16 weights below 2^-14 have the absolute half step 2^-25:
    2^-25 sum_j |v_j| against a sum of weights of at least 1/256 (the running
    maximum may lag by 2^8 and then weights are larger, never smaller).
    Scores are f32 sums of exact products: with |q_i k_i| summing to less than
    1000 on these inputs, 2^-23 * 1000 * scale (<= 1/8) is 1.5e-5 in natural
    log units, which moves a weight by that much: 2 * 1.5e-5 of the same sum.
    lse: the same 1.5e-5, the f32 exponentials' and sum's few 2^-22, and the
    rounding of its value."""
    want, want_lse, mag, vsum = ref
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()[..., 0]
    tol = (2 * EPS[dtype] + 3e-5) * mag + EPS[out_dtype] * np.abs(want) + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * vsum
    if out_dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(out - want)
    assert np.all(np.isfinite(out)), f"{what}: non-finite output"
    worst = (err / tol).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: output error is {worst:.2f} of the bound"
    assert np.array_equal(np.isneginf(lse), np.isneginf(want_lse)), f"{what}: empty rows"
    fin = np.isfinite(want_lse)
    if fin.any():
        e = np.abs(lse[fin] - want_lse[fin])
        assert np.all(e <= 1.7e-5 + 2.0 ** -22 * np.abs(want_lse[fin])), f"{what}: lse {e.max():.2e}"


def rope64(x, cos_sin, positions, off, interleaved):
    """x [T, H, D] with the pairs of its rotated columns turned, in 64 bits."""
    y = x.double().clone()
    n = cos_sin.shape[1] // 2
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for j in range(n):
            a, b = (off + 2 * j, off + 2 * j + 1) if interleaved else (off + j, off + n + j)
            c, s = float(cos_sin[p, j]), float(cos_sin[p, n + j])
            xa, xb = x[t, :, a].double(), x[t, :, b].double()
            y[t, :, a] = xa * c - xb * s
            y[t, :, b] = xb * c + xa * s
    return y


def rope_table(rows, rot, base=10000.0):
    rate = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * rate
    return torch.cat([ang.cos(), ang.sin()], 1).float()
