"""The packed attention's division of work, restated: ranges of half blocks that cut pairs of tiles at key blocks, the
slots of the parts, and the combination's view of them.  For random lengths every block of every pair and head belongs to
exactly one CTA, no part is shorter than the least, no two parts share a slot, and the combination adds exactly a pair's
parts, in their order, wherever the pair was cut."""
import random

import pytest

MIN_PART, ITEM_COST, SMS = 4, 3, 152


def cut_at(off, eh):
    e = (eh + 1) // 2
    b = off // 2 if off < eh else e
    return 0 if b < MIN_PART else e if e - b < MIN_PART else b


def groups_of(hkv):
    abreast = max(d for d in range(1, 9) if hkv % d == 0)
    return abreast, hkv // abreast, SMS // abreast


def pairs_of(seqs, tokens, subgroups):
    """(half blocks of the pair, of its two tiles, begin) of every pair of tiles."""
    out, at = [], 0
    for q, k in seqs:
        for t in range(0, q, 2 * tokens):
            last = [k - q + min(t + (x + 1) * tokens, q) - 1 for x in (0, 1)]
            tiles = [l // 64 + 1 if l >= 0 else 0 for l in last]
            if q - t <= tokens:
                tiles[1] = 0
            out.append((max(tiles), tiles, at))
            at += (max(tiles) + ITEM_COST) * subgroups
    return out, at


def check(seqs, hq, hkv):
    tokens = 128 // (hq // hkv)
    abreast, subgroups, groups = groups_of(hkv)
    pairs, work = pairs_of(seqs, tokens, subgroups)
    per = max(-(-work // groups), 2 * MIN_PART + ITEM_COST)
    start = [max([i for i, p in enumerate(pairs) if p[2] <= g * per], default=0) for g in range(groups)]
    parts = {}  # (pair, subgroup) -> [(first block, last, group, slot)]
    for g in range(groups):
        lo, hi = g * per, (g + 1) * per
        if lo >= work:
            continue
        for i in range(start[g], len(pairs)):
            eh, _, at = pairs[i]
            for sub in range(subgroups):
                begin, wide, e = at + sub * (eh + ITEM_COST), eh + ITEM_COST, (eh + 1) // 2
                if begin >= hi or begin + wide <= lo:
                    continue
                b0 = 0 if begin >= lo else cut_at(lo - begin, eh)
                b1 = e if begin + wide <= hi else cut_at(hi - begin, eh)
                if b0 >= b1 and (e > 0 or begin < lo):
                    continue
                slot = None if (b0, b1) == (0, e) else (g, 0 if b0 > 0 else 2)
                parts.setdefault((i, sub), []).append((b0, b1, g, slot))
    used = set()
    for i, (eh, tiles, at) in enumerate(pairs):
        for sub in range(subgroups):
            mine, e = parts[i, sub], (eh + 1) // 2
            assert [p[0] for p in mine] == [0, *[p[1] for p in mine[:-1]]] and mine[-1][1] == e
            assert len(mine) == 1 or all(p[1] - p[0] >= MIN_PART for p in mine)
            assert (len(mine) == 1) == (mine[0][3] is None)
            for p in mine:
                assert p[3] is None or p[3] not in used
                used.add(p[3]) if p[3] else None
    combined = {}
    for g in range(1, groups):
        if g * per >= work:
            continue
        eh, tiles, at = pairs[start[g]]
        wide, blocks = eh + ITEM_COST, (eh + 1) // 2
        sub = (g * per - at) // wide
        begin = at + sub * wide

        def border(k):
            return 0 if k * per <= begin else cut_at(k * per - begin, eh)

        if border(g) in (0, blocks) or border(g - 1) > 0:
            continue
        assert (start[g], sub) not in combined
        for x in (0, 1):
            e, n = (tiles[x] + 1) // 2, 0
            if e > 0:
                n = 1
                while border(g - 1 + n) < e:
                    n += 1
            combined[start[g], sub] = True
            slots = [(g - 1 + k, 2 if k == 0 else 0) for k in range(n)]
            assert slots == [p[3] for p in parts[start[g], sub] if p[0] < e]
    assert set(combined) == {key for key, p in parts.items() if len(p) > 1}


@pytest.mark.parametrize("seed", range(40))
def test_every_block_once_and_every_part_combined(seed):
    r = random.Random(seed)
    hkv = r.choice([1, 1, 2, 3, 7, 8, 11, 16, 24])
    hq = hkv * r.choice([1, 2, 4, 7, 128 if hkv == 1 else 8])
    longest = r.choice([60, 700, 9000, 100000])
    seqs = []
    for _ in range(r.choice([1, 2, 5, 40, 300])):
        k = r.randrange(longest)
        seqs.append((r.choice([0, 1, 1, 1, min(k, r.randrange(1, 400)), 5 if k < 5 else 1]), k))
    check(seqs, hq, hkv)


@pytest.mark.parametrize("seqs,hq,hkv", [([(1, 0)], 8, 2), ([(1, 1)], 1, 1), ([(1, 10 ** 6)], 8, 1), ([(3, 2)] * 5, 4, 1),
                                         ([(1, n) for n in range(900, 1400, 3)], 32, 8), ([(5000, 5000)], 32, 8)])
def test_edges(seqs, hq, hkv):
    check(seqs, hq, hkv)
