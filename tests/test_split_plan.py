"""The cuts of the split attention (pa_split_attention.cu), restated on the CPU: every unit of
every item goes to one CTA, a cut item's pieces sit on consecutive CTAs in the slots where the join
looks for them, and the first one counts the others right."""
import random

import pytest

ITEM_COST, LEAST_PIECE = 3, 2


def place(x, seqs, hkv, cut):
    """(sequence, item of it, key tile, units of the item before the cut) of unit x."""
    at = 0
    for s, (blocks, tiles) in enumerate(seqs):
        cost = tiles + ITEM_COST
        span = cost * blocks * hkv
        if at <= x < at + span:
            i, off = divmod(x - at, cost)
            tile = max(0, off - ITEM_COST)
            if tile < LEAST_PIECE and (cut or off <= 0):
                tile = 0
            elif not cut or tiles - tile < LEAST_PIECE:
                tile, i = 0, i + 1
            return s, i, tile, off
        at += span
    return len(seqs), 0, 0, 0


def shares(seqs, hkv, grid, cut):
    total = sum(b * hkv * (t + ITEM_COST) for b, t in seqs)
    share = max(-(-total // grid), LEAST_PIECE if cut else 1)
    ends = [place(c * share, seqs, hkv, cut) if c * share < total else (len(seqs), 0, 0, 0)
            for c in range(grid + 1)]
    return share, ends


def walk(seqs, hkv, ends, c):
    """The pieces of CTA c as K's loader announces them: (s, i, first tile, end, slot)."""
    s, i, tile, _ = ends[c]
    es, ei, et, _ = ends[c + 1]
    while True:
        if s < len(seqs) and i >= seqs[s][0] * hkv:
            i = tile = 0
            s += 1
            while s < len(seqs) and seqs[s][0] == 0:
                s += 1
        if not (s < len(seqs) and (s, i, tile) < (es, ei, et)):
            return
        end = et if (s, i) == (es, ei) else seqs[s][1]
        yield s, i, tile, end, (0 if tile > 0 else (1 if end < seqs[s][1] else -1))
        i, tile = i + 1, 0


def check(seqs, hkv, grid, cut):
    share, ends = shares(seqs, hkv, grid, cut)
    pieces = {}
    for c in range(grid):
        used = set()
        for s, i, t0, t1, slot in walk(seqs, hkv, ends, c):
            assert 0 <= t0 <= t1 <= seqs[s][1]
            assert slot < 0 or slot not in used
            used.add(slot)
            pieces.setdefault((s, i), []).append((c, t0, t1, slot))
    want = {(s, i) for s, (b, _) in enumerate(seqs) for i in range(b * hkv)}
    assert set(pieces) == want
    for (s, i), got in pieces.items():
        tiles = seqs[s][1]
        assert got[0][1] == 0 and got[-1][2] == tiles
        if len(got) == 1:
            assert got[0][3] == -1
        else:
            assert cut and got[0][3] == 1 and all(g[3] == 0 for g in got[1:])
            assert all(a[2] == b[1] and a[0] + 1 == b[0] for a, b in zip(got, got[1:]))
            assert all(t1 - t0 >= min(LEAST_PIECE, share) for _, t0, t1, _ in got)
    # the joins: written by the CTA whose share's end cuts an item that it holds the start of
    joins = {}
    for c in range(grid):
        es, ei, et, off = ends[c + 1]
        if et > 0:
            fs, fi, ft, _ = ends[c]
            if fs < es or fi < ei or ft == 0:
                joins[(es, ei)] = (c, 1 + (seqs[es][1] - LEAST_PIECE + ITEM_COST - off) // share)
    assert joins == {k: (g[0][0], len(g) - 1) for k, g in pieces.items() if len(g) > 1}


@pytest.mark.parametrize("seed", range(40))
def test_every_unit_once_and_joins_consecutive(seed):
    rng = random.Random(seed)
    for _ in range(60):
        n = rng.choice([1, 1, 2, 3, 7, 20, 70])
        top = rng.choice([1, 3, 8, 9, 20, 100, 600])
        seqs = [(rng.choice([0, 1, 1, 1, 2, 5]), rng.randint(0, top)) for _ in range(n)]
        seqs = [(b, t) if b else (0, 0) for b, t in seqs]
        check(seqs, rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 5, 16, 148, 152]),
              rng.random() < 0.8)


def test_one_long_sequence_uses_every_sm():
    share, ends = shares([(1, 16384)], 1, 152, True)
    assert len({e[:3] for e in ends}) == 153
