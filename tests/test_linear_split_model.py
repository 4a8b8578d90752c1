"""Model of how the linear layer's product is laid over CTA pairs (LinSplit and LinWork in
comm_overlap_gb300/csrc/linear.cu): every step of every tile is computed once, each pair publishes at most
one partial and does so first, and the pair that finishes a tile adds exactly the partials of the pairs
before it that hold a part of it."""
import random

import pytest

MIN_SHARE = 8


def split(tiles, kb, pairs):
    full, rest = divmod(tiles, pairs)
    q = max(-(-rest * kb // pairs), MIN_SHARE)
    if rest == 0 or q * 8 > kb * 7:
        q = kb
    parts = -(-rest * kb // q)
    return dict(units=pairs if full else parts, round=pairs, share=q, split=rest > 0 and q < kb)


def work(tiles, kb, s, unit):
    full, rest = divmod(tiles, s["round"])
    i0 = unit * s["share"]
    i1 = min(i0 + s["share"], rest * kb)
    pub = fin = None
    helpers = 0
    if i0 < i1:
        t = i0 // kb
        first = (full * s["round"] + t, i0 - t * kb, min(i1, (t + 1) * kb) - t * kb)
        if first[2] < kb:
            pub = first
        else:
            fin, helpers = first, unit - t * kb // s["share"]
            if i1 > (t + 1) * kb:
                pub = (first[0] + 1, 0, i1 - (t + 1) * kb)
    return pub, [(unit + i * s["units"], 0, kb) for i in range(full)], fin, helpers


def check(tiles, kb, pairs):
    s = split(tiles, kb, pairs)
    if tiles == 0:
        assert s["units"] == 0
        return
    assert 1 <= s["units"] <= pairs
    done, published = {}, {}
    for u in range(s["units"]):
        pub, whole, fin, helpers = work(tiles, kb, s, u)
        for seg in ([pub] if pub else []) + whole + ([fin] if fin else []):
            assert 0 <= seg[0] < tiles and 0 <= seg[1] < seg[2] <= kb
            for k in range(seg[1], seg[2]):
                assert (seg[0], k) not in done
                done[seg[0], k] = u
        if pub:
            assert s["split"] and pub[2] < kb  # the flags and slots were set up, and another pair finishes it
            published[u] = pub
        if fin:
            mine = [published[v] for v in range(u - helpers, u)]  # lower pairs only; each has published
            edges = [(0, 0)] + [p[1:] for p in mine] + [fin[1:]]
            assert all(p[0] == fin[0] for p in mine)
            assert edges[1][0] == 0 and all(a[1] == b[0] for a, b in zip(edges[1:], edges[2:])) and edges[-1][1] == kb
            for v in range(u - helpers, u):
                del published[v]
    assert not published, "a partial that nobody adds"
    assert len(done) == tiles * kb


@pytest.mark.parametrize("pairs", [1, 2, 7, 64, 76])
def test_every_step_once(pairs):
    for tiles in list(range(0, 2 * pairs + 3)) + [5 * pairs + 1, 40, 80, 128]:
        for kb in (1, 2, 8, 9, 10, 13, 40, 64, 161):
            check(tiles, kb, pairs)


def test_random_layouts():
    rng = random.Random(3)
    for _ in range(400):
        check(rng.randrange(1, 400), rng.randrange(1, 300), rng.randrange(1, 77))
