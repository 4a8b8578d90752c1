"""Model check of the cached attention kernel's barrier protocol (cached_attention.cu).

Roles, each in the program order of the kernel: the loading warp, the warp that issues the products, and four warps of keys for each
group of rows.  A TMA copy lands at an arbitrary later time; products complete in the order they were issued, each commit arriving
once all before it have.  Random interleavings of all of this, over items of few and of many tiles, prepared by the loading warp or by
the keys' warps, must

* never deadlock,
* pass every parity wait exactly when the phase that it means has completed,
* never overwrite a tile of the ring, Q, a buffer of scores or of weights, an item's rows, a list of exponents or O while somebody still
  reads it, and let each be read with the content that is meant."""
import random
from collections import deque

import pytest


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.arrived, self.done = name, count, 0, 0

    def arrive(self):
        self.arrived += 1
        assert self.arrived <= self.count, f"{self.name}: more arrivals than it counts"
        if self.arrived == self.count:
            self.arrived, self.done = 0, self.done + 1

    def passed(self, parity, phase):
        """A wait with this parity, which means phase `phase` (from 0)."""
        assert self.done <= phase + 1, f"{self.name}: {self.done} phases done, the waiter means {phase}"
        yes = (self.done & 1) != (parity & 1)
        assert yes == (self.done >= phase + 1), f"{self.name}: parity {parity} for phase {phase} with {self.done} done"
        return yes


class Model:
    exp_tiles, empty_wait, q_empty_wait, ready_look = 4, True, True, True

    def __init__(self, items, slots, groups, rng):
        """items: (tiles, whether the keys' warps prepare it) each."""
        self.items, self.slots, self.warps, self.groups, self.rng = items, slots, 4 * groups, groups, rng
        n = self.warps
        bar = lambda name, k, count: [Bar(f"{name}{i}", count) for i in range(k)]
        self.full, self.empty = bar("full", slots, 1), bar("empty", slots, 1)
        self.q_full, self.s_full, self.p_full = bar("q_full", 2, 1), bar("s_full", 2, 1), bar("p_full", 2, n)
        self.pv_done, self.exps, self.q_empty = bar("pv_done", 2, 1), bar("exps", 4, 1), bar("q_empty", 2, n + 1)
        self.ready = Bar("ready", n)
        self.copies, self.pipe = [], deque()
        self.content, self.readers, self.pieces, self.out = {}, {}, {}, []
        self.meeting = {}  # barriers of warps: [arrived, times]
        self.progress = [(-1, -1)] * n  # item and tile that each warp of keys has done with

    # ---- memory: named buffers with what they hold and who reads them
    def write(self, name, what, part=0, parts=1):
        assert not self.readers.get(name), f"{name} is overwritten while it is read"
        old = self.content.get(name)
        if parts == 1:
            self.content[name] = what
        else:
            have = old[1] if isinstance(old, tuple) and old[0] == ("partly", what) else frozenset()
            have = have | {part}
            self.content[name] = what if len(have) == parts else (("partly", what), have)

    def read(self, name, what):
        assert self.content.get(name) == what, f"{name} holds {self.content.get(name)}, meant is {what}"

    def land(self):
        name, what, slot = self.copies.pop(self.rng.randrange(len(self.copies)))
        self.content[name] = what
        self.full[slot].arrive()

    def complete(self):
        kind, x = self.pipe.popleft()
        if kind == "commit":
            x.arrive()
        else:
            reads, name, what = x
            for r in reads:
                self.readers[r] -= 1
            self.content[name] = what

    def product(self, reads, name, what):
        for r, held in reads:
            self.read(r, held)
            self.readers[r] = self.readers.get(r, 0) + 1
        self.pipe.append(("product", ([r for r, _ in reads], name, what)))

    def meet(self, name, count):
        m = self.meeting.setdefault(name, [0, 0])
        mine = m[1]
        m[0] += 1
        if m[0] == count:
            m[0], m[1] = 0, mine + 1
        while m[1] == mine:
            yield lambda: m[1] != mine

    def wait(self, bar, parity, phase):
        yield lambda: bar.passed(parity, phase)

    # ---- the loading warp
    def loader(self):
        slot = rnd = made = item = tile_of_all = 0

        def store():
            t = made - 1
            if t >= self.exp_tiles:
                assert all(done >= t - self.exp_tiles for _, done in self.progress), "exponents are overwritten before they are read"
            self.write(f"exps{t % self.exp_tiles}", t)
            self.exps[t % self.exp_tiles].arrive()

        while True:
            there = item < len(self.items)
            tiles = self.items[item][0] if there else 0
            for tile in range(tiles + 1):
                if tile < tiles:
                    if made > 0:
                        store()
                        yield None
                    for what in "KV":
                        if rnd > 0 and self.empty_wait:
                            yield from self.wait(self.empty[slot], rnd - 1, rnd - 1)
                        name = f"ring{slot}"
                        assert not self.readers.get(name), f"{name} is overwritten while it is read"
                        self.content.pop(name, None)
                        self.copies.append((name, (what, tile_of_all), slot))
                        yield None
                        slot += 1
                        if slot == self.slots:
                            slot, rnd = 0, rnd + 1
                    made += 1
                    tile_of_all += 1
                if tile == 0 and item > 0:
                    if item >= 2 and self.q_empty_wait:
                        yield from self.wait(self.q_empty[item & 1], (item >> 1) + 1, (item >> 1) - 1)
                    assert all(done >= item - 2 for done, _ in self.progress), "a piece is overwritten before its item's end"
                    self.pieces[item & 1] = item
                    yield None
                    if there and not self.items[item][1]:
                        self.write(f"q{item & 1}", item)
                        self.write(f"rows{item & 1}", item)
                    yield None
                    self.q_full[item & 1].arrive()
                if not there:
                    break
            if not there:
                break
            item += 1
        if made > 0:
            store()

    # ---- the products
    def products(self):
        s = dict(tile=0, tiles=0, item=0, made=0, slot_k=0, round_k=0, readied=0, more=False)
        of = {}  # tile of all -> (item, whether it is the item's first)

        def enter():
            i = s["item"]
            yield from self.wait(self.q_full[i & 1], i >> 1, i >> 1)
            s["tile"], s["tiles"] = 0, self.items[i][0] if i < len(self.items) else 0
            assert i == 0 or self.pieces[i & 1] == i
            s["more"] = s["tiles"] > 0
            if s["more"] and i > 0 and self.items[i][1]:
                yield from self.wait(self.ready, s["readied"], s["readied"])
                s["readied"] += 1

        def next_ready():
            i = s["item"] + 1
            if not self.q_full[i & 1].passed(i >> 1, i >> 1):
                return False
            return not (self.ready_look and i < len(self.items) and self.items[i][1])

        def scores():
            k = s["made"]
            yield from self.wait(self.full[s["slot_k"]], s["round_k"], s["round_k"])
            if k >= 2:
                assert all(done >= k - 2 for _, done in self.progress), "scores are overwritten before they are read"
            i = s["item"]
            self.product([(f"ring{s['slot_k']}", ("K", k)), (f"q{i & 1}", i)], f"s{k & 1}", k)
            of[k] = i, s["tile"] == 0
            self.pipe.append(("commit", self.s_full[k & 1]))
            self.pipe.append(("commit", self.empty[s["slot_k"]]))
            s["tile"] += 1
            if s["tile"] == s["tiles"]:
                self.pipe.append(("commit", self.q_empty[i & 1]))
            s["slot_k"] += 2
            if s["slot_k"] >= self.slots:
                s["slot_k"], s["round_k"] = s["slot_k"] - self.slots, s["round_k"] + 1
            s["made"] += 1
            yield None

        yield from enter()
        if s["more"]:
            yield from scores()
        j, slot_v, round_v = 0, 1, 0
        while j < s["made"]:
            last = s["tile"] == s["tiles"]
            if last and next_ready():
                s["item"] += 1
                yield from enter()
                last = False
            if not last and s["more"]:
                yield from scores()
            yield from self.wait(self.p_full[j & 1], j >> 1, j >> 1)
            yield from self.wait(self.full[slot_v], round_v, round_v)
            i, first = of[j]
            if first:
                assert i == 0 or all(done >= i - 1 for done, _ in self.progress), "O is overwritten before it is read"
            self.product([(f"ring{slot_v}", ("V", j)), (f"p{j & 1}", j)], "o", (i, j))
            self.pipe.append(("commit", self.pv_done[j & 1]))
            self.pipe.append(("commit", self.empty[slot_v]))
            yield None
            slot_v += 2
            if slot_v >= self.slots:
                slot_v, round_v = slot_v - self.slots, round_v + 1
            if last:
                s["item"] += 1
                yield from enter()
                if s["more"]:
                    yield from scores()
            j += 1

    # ---- a warp of keys
    def keys(self, w):
        group = w // 4
        self.write("q0", 0, w, self.warps)
        self.write("rows0", 0, w, self.warps)
        yield from self.meet("all", self.warps)
        if w == 0:
            self.q_full[0].arrive()
        j, slot_v, round_v, readied, item = 0, 1, 0, 0, 0
        while True:
            yield from self.wait(self.q_full[item & 1], item >> 1, item >> 1)
            there = item < len(self.items)
            assert item == 0 or self.pieces[item & 1] == item
            yield from self.meet("all", self.warps)
            if not there:
                return
            tiles, by_keys = self.items[item]
            if item > 0 and by_keys:
                self.write(f"q{item & 1}", item, w, self.warps)
                self.write(f"rows{item & 1}", item, w, self.warps)
                yield None
                self.ready.arrive()
                yield from self.wait(self.ready, readied, readied)
                readied += 1
            for tile in range(tiles):
                yield from self.wait(self.exps[j % 4], j // 4, j // 4)
                self.read(f"exps{j % self.exp_tiles}", j)
                yield from self.wait(self.s_full[j & 1], j >> 1, j >> 1)
                self.read(f"s{j & 1}", j)
                self.read(f"rows{item & 1}", item)
                yield from self.meet(f"group{group}", 4)
                if tile > 0 and random.Random(j * 7 + group).random() < 0.3:  # a row's reference moves, and O with it
                    yield from self.wait(self.pv_done[(j - 1) & 1], (j - 1) >> 1, (j - 1) >> 1)
                    self.read("o", (item, j - 1))
                if j >= 2:
                    yield from self.wait(self.pv_done[j & 1], (j - 2) >> 1, (j - 2) >> 1)
                self.write(f"p{j & 1}", j, w, self.warps)
                if tile == tiles - 1 and group == 0:  # values past the keys are cleared
                    yield from self.wait(self.full[slot_v], round_v, round_v)
                    self.read(f"ring{slot_v}", ("V", j))
                    assert not self.readers.get(f"ring{slot_v}"), "values are cleared while they are read"
                yield None
                self.progress[w] = self.progress[w][0], j  # (of scores and exponents; the weights are written)
                self.p_full[j & 1].arrive()
                j += 1
                slot_v += 2
                if slot_v >= self.slots:
                    slot_v, round_v = slot_v - self.slots, round_v + 1
                yield None
            yield from self.meet(f"group{group}", 4)
            yield from self.wait(self.pv_done[(j - 1) & 1], (j - 1) >> 1, (j - 1) >> 1)
            yield from self.meet(f"group{group}", 4)
            self.read("o", (item, j - 1))
            self.read(f"rows{item & 1}", item)
            self.out.append((item, w))
            yield None
            self.progress[w] = item, self.progress[w][1]
            self.q_empty[item & 1].arrive()
            item += 1

    def run(self):
        agents = {name: (gen, None) for name, gen in [("loader", self.loader()), ("products", self.products()),
                                                     *((f"keys{w}", self.keys(w)) for w in range(self.warps))]}
        # some are slow for a while, so that others get as far ahead as they can
        weight = {name: self.rng.choice([1, 1, 5, 25]) for name in (*agents, "copies", "pipe")}
        while agents:
            able = [name for name, (_, ready) in agents.items() if ready is None or ready()]
            able += ["copies"] * bool(self.copies) + ["pipe"] * bool(self.pipe)
            assert able, f"deadlock of {sorted(agents)}"
            name = self.rng.choices(able, [weight[a] for a in able])[0]
            if name == "copies":
                self.land()
            elif name == "pipe":
                self.complete()
            else:
                gen, _ = agents[name]
                try:
                    agents[name] = gen, next(gen)
                except StopIteration:
                    del agents[name]
        while self.pipe:
            self.complete()
        assert sorted(self.out) == [(i, w) for i in range(len(self.items)) for w in range(self.warps)]
        assert not self.copies and not any(self.readers.values())


def lists(rng, by_keys):
    n = rng.randint(1, 7)
    return [(rng.choice([1, 1, 2, 3, 5, 9]), by_keys and rng.random() < 0.5) for _ in range(n)]


@pytest.mark.parametrize("slots,groups", [(6, 1), (5, 1), (4, 2)])
def test_protocol(slots, groups):
    for seed in range(150):
        rng = random.Random(seed)
        Model(lists(rng, slots != 6), slots, groups, rng).run()


@pytest.mark.parametrize("mistake", ["empty_wait", "q_empty_wait", "ready_look", "exp_tiles"])
def test_planted_mistakes_are_found(mistake):
    """A ring's place taken again without a wait, an item's memory too, the next item entered before the last product although the keys'
    warps prepare it, exponents of two tiles only."""
    class Wrong(Model):
        pass

    setattr(Wrong, mistake, 2 if mistake == "exp_tiles" else False)
    found = 0
    for seed in range(150):
        rng = random.Random(seed)
        try:
            Wrong(lists(rng, True), 4, 2, rng).run()
        except AssertionError:
            found += 1
    assert found > 0
