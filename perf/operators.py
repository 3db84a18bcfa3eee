"""Cases that measure attention over uncompressed keys and values: the paged
key and value cache that grouped-head and per-head models keep where latent
attention keeps one compressed row.

Three operators, each with its plain form and the framework's call:

* ``append``: the new tokens' keys and values are stored in the paged cache
  and the keys (and queries) get their position rotation on the way;
* ``decode``: attention of one new token per request over the paged cache;
* ``prompt``: causal attention of packed prompts of different lengths, over
  packed keys and values or over the paged cache (a chunk after a prefix).

``run`` takes the plain form where ``own`` is false and the framework's
kernels where it is true.
"""
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HEADS = [(64, 64), (128, 128), (192, 128)]  # widths of a key head and of a value head
SCORES = 1 << 31  # the most scores that a prompt's plain form holds at a time


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of 64 requests: a row of 8 heads each, latency counts
        dict(name="append step", op="append", dtype="bf16", src="bf16", b=64, lo=200, hi=1000,
             new_lo=1, new_hi=1, hq=32, hkv=8, dk=128, dv=128, rot=128, off=0, inter=False, lens=1),
        # packed prompts of 16 requests, some after cached tokens; f32 keys and values as a
        # projection with f32 sums leaves them
        dict(name="append prompts", op="append", dtype="f16", src="f32", b=16, lo=0, hi=500,
             new_lo=300, new_hi=1700, hq=64, hkv=8, dk=128, dv=128, rot=64, off=0, inter=False,
             lens=2),
        # latent rows (512 latent and 64 rope values, one shared head, no values of their own)
        # of a prompt, and the rope columns of 128 query heads into the absorbed query
        dict(name="append latent rows", op="append", dtype="bf16", src="bf16", b=2, lo=0, hi=0,
             new_lo=2048, new_hi=2048, hq=128, hkv=1, dk=576, dv=0, rot=64, off=512, inter=True,
             lens=3),
        # one short request of a small model: latency
        dict(name="decode tiny", op="decode", dtype="bf16", b=1, lo=256, hi=256, hq=16, hkv=4,
             dk=64, dv=64, lens=0),
        # an ordinary serving batch of mixed lengths, four query heads to a key head
        dict(name="decode batch", op="decode", dtype="bf16", b=32, lo=2048, hi=4096, hq=32, hkv=8,
             dk=128, dv=128, lens=4),
        # heads of their own (128 + 64 rope columns of keys, 128 of values), fp16, ragged
        dict(name="decode per head", op="decode", dtype="f16", b=13, lo=1, hi=5001, hq=16, hkv=16,
             dk=192, dv=128, lens=5),
        # four long contexts, eight query heads to a key head: the split over the length
        dict(name="decode long", op="decode", dtype="bf16", b=4, lo=131072, hi=131072, hq=64,
             hkv=8, dk=128, dv=128, lens=6),
        # one short prompt of a small model: latency
        dict(name="prompt tiny", op="prompt", dtype="bf16", b=1, lo=77, hi=77, pre_lo=0, pre_hi=0,
             paged=False, hq=16, hkv=4, dk=64, dv=64, lens=0),
        # packed prompts of different lengths
        dict(name="prompt packed", op="prompt", dtype="bf16", b=12, lo=33, hi=1500, pre_lo=0,
             pre_hi=0, paged=False, hq=32, hkv=8, dk=128, dv=128, lens=7),
        # chunks of four long prompts after what the paged cache holds already
        dict(name="prompt chunk paged", op="prompt", dtype="f16", b=4, lo=300, hi=512,
             pre_lo=4000, pre_hi=8000, paged=True, hq=32, hkv=4, dk=128, dv=128, lens=8),
        # one prompt of latent attention in its per-head form: 128 heads of 192 and 128
        dict(name="prompt per head", op="prompt", dtype="bf16", b=1, lo=4096, hi=4096, pre_lo=0,
             pre_hi=0, paged=False, hq=128, hkv=128, dk=192, dv=128, lens=0),
        # a long prompt on one tensor-parallel rank: eight query heads, one key head
        dict(name="prompt long", op="prompt", dtype="bf16", b=1, lo=16384, hi=16384, pre_lo=0,
             pre_hi=0, paged=False, hq=8, hkv=1, dk=128, dv=128, lens=0),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    dk, dv = rng.choice(HEADS)
    lens = rng.randrange(1 << 30)
    hkv = _between(rng, 1, 16)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "append":
        latent = rng.random() < 0.3
        if latent:
            hkv, dk, dv = 1, 576, 0
        rot = 64 if latent else rng.choice([r for r in (32, 64, 128) if r <= dk])
        new = _between(rng, 1, 2048)
        b = _between(rng, 1, max(1, min(64, 8192 // new)))
        return dict(op=op, dtype=dtype, src=rng.choice([dtype, "f32"]), b=b, lo=0,
                    hi=rng.choice([0, 63, 1000]), new_lo=max(1, new // 2), new_hi=new,
                    hq=hkv * group, hkv=hkv, dk=dk, dv=dv, rot=rot,
                    off=dk - rot if latent or rng.random() < 0.5 else 0,
                    inter=rng.random() < 0.5, lens=lens)
    if op == "decode":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 32, 64])
        hi = _between(rng, 1, 65536)
        room = (1 << 30) // (hi * hkv * (dk + dv))  # values of the cache
        return dict(op=op, dtype=dtype, b=_between(rng, 1, max(1, min(64, room))),
                    lo=rng.randint(1, hi), hi=hi, hq=min(128, hkv * group) // hkv * hkv, hkv=hkv,
                    dk=dk, dv=dv, lens=lens)
    paged = rng.random() < 0.5
    pre = _between(rng, 1, 8192) if paged and rng.random() < 0.7 else 0
    hi = _between(rng, 1, 4096)
    hkv = _between(rng, 1, 8)
    room = SCORES // 4 // (hi * (hi + pre) * hkv * group)
    while room < 1:
        hi, pre = (hi + 1) // 2, pre // 2
        room = SCORES // 4 // (hi * (hi + pre) * hkv * group)
    return dict(op=op, dtype=dtype, b=_between(rng, 1, min(24, room)), lo=max(1, hi // 8), hi=hi,
                pre_lo=pre // 2, pre_hi=pre, paged=paged, hq=hkv * group, hkv=hkv, dk=dk, dv=dv,
                lens=lens)


def _lengths(case, lo, hi, salt):
    """The requests' lengths: the case's own, whatever the inputs' seed."""
    rng = random.Random(2 * case["lens"] + salt)
    return [rng.randint(lo, hi) for _ in range(case["b"])]


def _plan(case):
    """Each request's cached tokens before the call and tokens of the call."""
    if case["op"] == "decode":
        return [n - 1 for n in _lengths(case, case["lo"], case["hi"], 0)], [1] * case["b"]
    if case["op"] == "append":
        return (_lengths(case, case["lo"], case["hi"], 0),
                _lengths(case, case["new_lo"], case["new_hi"], 1))
    return (_lengths(case, case["pre_lo"], case["pre_hi"], 0),
            _lengths(case, case["lo"], case["hi"], 1))


def work(case):
    before, new = _plan(case)
    tokens = sum(new)
    held = sum(before) + tokens
    hq, hkv, dk, dv = case["hq"], case["hkv"], case["dk"], case["dv"]
    pages = 4 * sum((a + n + PAGE - 1) // PAGE for a, n in zip(before, new))
    if case["op"] == "append":
        src = 4 if case["src"] == "f32" else 2
        longest = max(a + n for a, n in zip(before, new))
        rows = tokens * hkv * (dk + dv) * (src + 2)
        queries = tokens * hq * (case["rot"] if dv == 0 else dk) * (2 + 2)
        table = min(tokens, longest) * case["rot"] * 4
        return {"bytes": rows + queries + table + 8 * tokens + pages,
                "flops": tokens * (hq + hkv) * case["rot"] // 2 * 6}
    pairs = sum(n * a + n * (n + 1) // 2 for a, n in zip(before, new))
    rows = held * hkv * (dk + dv) * 2
    heads = tokens * hq * ((dk + dv) * 2 + 4)
    paged = case["op"] == "decode" or case["paged"]
    return {"bytes": rows + heads + 4 * case["b"] + (pages if paged else 0),
            "flops": 2 * pairs * hq * (dk + dv)}


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, dk, dv, b = case["hq"], case["hkv"], case["dk"], case["dv"], case["b"]

    def rand(*shape, dtype=dt, gain=1.0):
        return (torch.randn(shape, generator=gen, device=dev, dtype=dtype) * gain)

    before, new = _plan(case)
    tokens, ends = sum(new), [a + n for a, n in zip(before, new)]
    of = torch.repeat_interleave(torch.arange(b), torch.tensor(new))
    cu = torch.zeros(b + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(new).cumsum(0)
    s = {"case": case, "longest": max(ends), "widest": max(new),
         "requests": of.to(dev, torch.int32), "cu": cu.to(dev, torch.int32),
         "positions": (torch.arange(tokens) - cu[of] + torch.tensor(before)[of]).to(dev, torch.int32),
         "seq_lens": torch.tensor(ends, dtype=torch.int32, device=dev)}
    if case["op"] != "prompt" or case["paged"]:
        # a pool of pages in random order; the table's unused entries are zeros
        pages = [(n + PAGE - 1) // PAGE for n in ends]
        order = torch.randperm(sum(pages) + 3, generator=gen, device=dev)
        table = torch.zeros((b, max(pages)), dtype=torch.int64, device=dev)
        first = torch.tensor([0] + pages, device=dev).cumsum(0)
        col = torch.arange(max(pages), device=dev)[None]
        live = col < torch.tensor(pages, device=dev)[:, None]
        table[live] = order[(first[:-1, None] + col)[live]]
        s["page_table"] = table.to(torch.int32)
        s["k_cache"] = rand(order.numel(), PAGE, hkv, dk)
        s["v_cache"] = rand(order.numel(), PAGE, hkv, dv) if dv else None
    if case["op"] == "append":
        src = DTYPES[case["src"]]
        s["k"] = rand(tokens, hkv, dk, dtype=src)
        s["v"] = rand(tokens, hkv, dv, dtype=src) if dv else None
        rate = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
        angle = torch.arange(max(ends), dtype=torch.float64, device=dev)[:, None] * rate
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if dv:
            s["q"], s["q_off"] = rand(tokens, hq, dk), case["off"]
            s["q_out"] = torch.empty_like(s["q"])
        else:  # the rope columns of [128 | 64] queries, into those of the absorbed [512 | 64]
            s["q"], s["q_off"] = rand(tokens, hq, 128 + case["rot"])[..., 128:], 0
            s["q_out"] = rand(tokens, hq, dk)[..., case["off"]:]
        return s
    s["q"] = rand(tokens, hq, dk, gain=1.5)
    if case["op"] == "prompt" and not case["paged"]:
        s["k"], s["v"] = rand(tokens, hkv, dk), rand(tokens, hkv, dv)
    s["scale"] = dk ** -0.5
    return s


# ------------------------------------------------------------------ a pass
def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _run_append(state)
    return _run_decode(state) if op == "decode" else _run_prompt(state)


def _rotated(x, cos, sin, off, inter):
    """x in 32 bits with the pairs of its columns [off, off + 2 n) turned by their angles."""
    x = x.float()
    n = cos.shape[-1]
    part = x[..., off:off + 2 * n]
    if inter:
        a, c = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
    else:
        a, c = part[..., :n], part[..., n:]
        turned = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    return torch.cat([x[..., :off], turned, x[..., off + 2 * n:]], -1)


def _run_append(s):
    c = s["case"]
    if own:
        import mla_latent_kv_dim_b200 as tp
        tp.kv_append(s["k"], s["v"], s["positions"], s["page_table"], s["k_cache"], s["v_cache"],
                     requests=s["requests"], cos_sin=s["cos_sin"], rope_offset=c["off"],
                     interleaved=c["inter"], q=s["q"], q_out=s["q_out"], q_rope_offset=s["q_off"])
        return _stored(s)
    pos = s["positions"].long()
    cos, sin = s["cos_sin"][pos][:, None].chunk(2, -1)
    page = s["page_table"][s["requests"].long(), pos // PAGE].long()
    s["k_cache"][page, pos % PAGE] = _rotated(s["k"], cos, sin, c["off"], c["inter"]).to(s["k_cache"].dtype)
    if s["v"] is not None:
        s["v_cache"][page, pos % PAGE] = s["v"].to(s["v_cache"].dtype)
    s["q_out"].copy_(_rotated(s["q"], cos, sin, s["q_off"], c["inter"]))
    return _stored(s)


def _stored(s):
    return [s[x] for x in ("k_cache", "v_cache", "q_out") if s[x] is not None]


def _attend(q, k, v, scale, held, limit):
    """Plain attention in 32 bits of q [B, T, Hq, Dk] over k, v [B, L, Hkv, D]: key j of request b
    counts for query i where j < limit[b, i]; values behind held[b] are not read."""
    B, T, Hq, _ = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    at = torch.arange(L, device=q.device)
    v = v.float().masked_fill((at >= held[:, None])[:, :, None, None], 0)
    qg = q.float().view(B, T, Hkv, Hq // Hkv, -1).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(qg, k.float().permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, T, L).mul_(scale)
    x.masked_fill_((at >= limit[..., None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, T, -1)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + total.log())[..., 0]
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)


def _paged(cache, table, longest):
    return cache[table.long()].flatten(1, 2)[:, :longest]


def _run_decode(s):
    q = s["q"]
    if own:
        import mla_latent_kv_dim_b200 as tp
        return tp.kv_decode(q, s["k_cache"], s["v_cache"], s["seq_lens"], s["page_table"],
                            scale=s["scale"], out_dtype=q.dtype)
    k = _paged(s["k_cache"], s["page_table"], s["longest"])
    v = _paged(s["v_cache"], s["page_table"], s["longest"])
    held = s["seq_lens"].long()
    out, lse = _attend(q[:, None], k, v, s["scale"], held, held[:, None])
    return out[:, 0].to(q.dtype), lse[:, 0, :, None]


def _run_prompt(s):
    q, paged = s["q"], s["case"]["paged"]
    if own:
        import mla_latent_kv_dim_b200 as tp
        if paged:
            return tp.kv_prefill(q, s["k_cache"], s["v_cache"], s["cu"], seq_lens=s["seq_lens"],
                                 page_table=s["page_table"], scale=s["scale"], out_dtype=q.dtype)
        return tp.kv_prefill(q, s["k"], s["v"], s["cu"], scale=s["scale"], out_dtype=q.dtype)
    cu, held = s["cu"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.arange(s["widest"], device=q.device)).clamp_(max=q.shape[0] - 1)
    limit = (held - new)[:, None] + torch.arange(1, s["widest"] + 1, device=q.device)
    if paged:
        k = _paged(s["k_cache"], s["page_table"], s["longest"])
        v = _paged(s["v_cache"], s["page_table"], s["longest"])
    else:
        k, v = s["k"][at], s["v"][at]
    out, lse = _attend(q[at], k, v, s["scale"], held, torch.minimum(limit, held[:, None]))
    of = s["requests"].long()
    row = torch.arange(q.shape[0], device=q.device) - cu[of]
    return out[of, row].to(q.dtype), lse[of, row][..., None]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definitions, request by request and head by head, in 64 bits."""
    s = prepare(case, seed)
    before, new = _plan(case)
    hq, hkv, dk, dv = case["hq"], case["hkv"], case["dk"], case["dv"]
    group, first = hq // hkv, 0
    table = s["page_table"].tolist() if "page_table" in s else None
    if case["op"] == "append":
        kc = s["k_cache"].double()
        vc = None if dv == 0 else s["v_cache"].double()
        qo = s["q"].double()
        n = case["rot"] // 2
        j = torch.arange(n, device=kc.device)
        lower, upper = (2 * j, 2 * j + 1) if case["inter"] else (j, j + n)
        for b in range(case["b"]):
            rows = slice(first, first + new[b])
            ang = s["cos_sin"][before[b]:before[b] + new[b]].double()
            co, si = ang[:, None, :n], ang[:, None, n:]
            kb = s["k"][rows].double()
            for x, off in ((kb, case["off"]), (qo[rows], s["q_off"])):
                lo, up = x[..., off + lower], x[..., off + upper]
                x[..., off + lower] = lo * co - up * si
                x[..., off + upper] = lo * si + up * co
            at = torch.arange(before[b], before[b] + new[b], device=kc.device)
            page = s["page_table"][b].long()[at // PAGE]
            kc[page, at % PAGE] = kb
            if vc is not None:
                vc[page, at % PAGE] = s["v"][rows].double()
            first += new[b]
        return [kc, qo] if vc is None else [kc, vc, qo]
    outs = torch.empty((sum(new), hq, dv), dtype=torch.float64, device=s["q"].device)
    lses = torch.empty((sum(new), hq, 1), dtype=torch.float64, device=s["q"].device)
    for b in range(case["b"]):
        total = before[b] + new[b]
        if table is None:
            kb, vb = s["k"][first:first + total], s["v"][first:first + total]
        else:
            own_pages = torch.tensor(table[b][:(total + PAGE - 1) // PAGE], device=outs.device)
            kb = s["k_cache"][own_pages].reshape(-1, hkv, dk)[:total]
            vb = s["v_cache"][own_pages].reshape(-1, hkv, dv)[:total]
        for h in range(hq):
            kh, vh = kb[:, h // group].double(), vb[:, h // group].double()
            for i in range(0, new[b], 2048):
                m = min(2048, new[b] - i)
                seen = before[b] + i + m
                rows = slice(first + i, first + i + m)
                x = s["scale"] * (s["q"][rows, h].double() @ kh[:seen].T)
                last = before[b] + i + torch.arange(m, device=x.device)
                x[torch.arange(seen, device=x.device)[None] > last[:, None]] = -math.inf
                z = torch.logsumexp(x, -1, keepdim=True)
                outs[rows, h] = torch.exp(x - z) @ vh[:seen]
                lses[rows, h] = z
        first += new[b]
    return outs, lses
