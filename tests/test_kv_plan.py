"""The list of items that tpla_kv_prefill's plan kernel makes, restated: its
entries and the pieces' slots are as many as the workspace has room for, and
every entry up to the count is written whole, for offsets that rise and for
offsets that fall and claim rows again.  CPU only."""
import random

import pytest

KEYS, ROWS, MIN_PIECE = 64, 128, 8


def shape(T, B, heads, gg, cap_rows, sms):
    """What the launcher sizes the workspace by."""
    tpt = ROWS // gg
    entries = T // (2 * tpt) + B
    cut = T // (2 * tpt) * heads < 2 * sms and cap_rows >= 2 * MIN_PIECE * KEYS
    slots = -(-4 * sms // heads) if cut else 0
    return tpt, entries, cut, slots, entries + (2 * sms if cut else 0)


def plan(cu, lens, T, heads, gg, cap_rows, causal, sms):
    """(entries as (request, t0, j0, j1, slot), items in pieces, slots), or
    None where the requests claim too many items."""
    tpt, room, cut, slots, _ = shape(T, len(lens), heads, gg, cap_rows, sms)
    tb = 2 * tpt
    items = []
    for b, held in enumerate(lens):
        lo = max(0, min(cu[b], T))
        n = max(lo, min(cu[b + 1], T)) - lo
        if len(items) > room:
            break
        for t0 in range(0, n, tb):
            last = min(t0 + tb, n) - 1
            limit = max(0, min(held, held - n + last + 1)) if causal else held
            items.append((b, t0, -(-limit // KEYS)))
    if len(items) > room:
        return None
    longest = max(MIN_PIECE, -(-sum(i[2] for i in items) * heads // (2 * sms)))
    listed, joins, used = [], 0, 0
    for b, t0, tiles in items:
        k = max(1, -(-tiles // longest)) if cut else 1
        length = -(-tiles // k)
        slot = used
        if k > 1:
            joins, used = joins + 1, used + k
        for i in range(k):
            listed.append((b, t0, i * length, min(tiles, (i + 1) * length), slot + i if k > 1 else -1))
    return listed, joins, used


@pytest.mark.parametrize("seed", range(60))
def test_room_for_every_entry(seed):
    rng = random.Random(seed)
    for _ in range(20):
        sms = rng.choice([1, 20, 132, 148])
        gg, heads = rng.choice([1, 3, 8, 100, 128]), rng.choice([1, 2, 5, 16, 700])
        B, T = rng.randint(1, 60), int(10 ** rng.uniform(0, 4))
        paged = rng.random() < 0.6
        cap = int(10 ** rng.uniform(1, 6)) if paged else T
        kind = rng.choice(["rising", "falling", "twice", "any"])
        if kind == "rising":
            cu = sorted(rng.randint(0, T) for _ in range(B + 1))
        elif kind == "falling":
            cu = sorted((rng.randint(0, T) for _ in range(B + 1)), reverse=True)
        elif kind == "twice":
            cu = [T * (i & 1) for i in range(B + 1)]
        else:
            cu = [rng.randint(-5, T + 5) for _ in range(B + 1)]
        lens = [rng.randint(0, cap) if paged else max(0, min(z, T) - max(0, min(a, T)))
                for a, z in zip(cu, cu[1:])]
        _, entries, cut, slots, capacity = shape(T, B, heads, gg, cap, sms)
        made = plan(cu, lens, T, heads, gg, cap, rng.random() < 0.7, sms)
        if made is None:
            assert kind in ("twice", "any")
            continue
        listed, joins, used = made
        assert len(listed) <= capacity and used <= slots and joins <= slots
        assert all(0 <= j0 <= j1 and t0 >= 0 for _, t0, j0, j1, _ in listed)
        taken = sorted(s for *_, s in listed if s >= 0)
        assert taken == list(range(used))  # no slot twice


def test_rising_offsets_are_never_too_many():
    """One more row than a whole number of tiles in each request."""
    for gg in (1, 3, 128):
        tb = 2 * (ROWS // gg)
        for B in (1, 7, 500):
            cu = [b * (tb + 1) for b in range(B + 1)]
            assert plan(cu, [9] * B, cu[-1], 1, gg, 9, True, 148) is not None
