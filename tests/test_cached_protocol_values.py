"""Model check of the cached attention kernel's barrier protocol where the keys' warps look at a tile's values before they weigh it, in tiles in
which a row's reference moves (its first ones, and any later one)."""
import random

import pytest

from test_cached_protocol_model import Model, lists


class Looking(Model):
    just, place = None, 0  # the tile whose scores a warp has just read; where it looks for the values, off the right place

    def read(self, name, what):
        super().read(name, what)
        if name in ("s0", "s1"):
            self.just = what  # (the same warp goes on to its group's meeting without a pause)

    def meet(self, name, count):
        tile, self.just = self.just, None
        yield from super().meet(name, count)
        if tile is not None and random.Random(f"{tile} {name}").random() < 0.5:
            at = 2 * tile + 1
            yield from self.wait(self.full[at % self.slots], at // self.slots, at // self.slots)
            self.read(f"ring{(at + self.place) % self.slots}", ("V", tile))
            yield None
            self.read(f"ring{(at + self.place) % self.slots}", ("V", tile))  # (still there)


@pytest.mark.parametrize("slots,groups", [(5, 1), (4, 2)])
def test_values_are_there_while_they_are_looked_at(slots, groups):
    for seed in range(120):
        rng = random.Random(seed)
        Looking(lists(rng, True), slots, groups, rng).run()


def test_another_place_is_found():
    class Wrong(Looking):
        place = 1

    with pytest.raises(AssertionError):
        for seed in range(20):
            rng = random.Random(seed)
            Wrong(lists(rng, True), 5, 1, rng).run()
