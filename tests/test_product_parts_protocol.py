"""The grouped product's tiles of a long k, checked on the CPU: such a tile is computed in parts, each
summed by the MMAs in an accumulator of its own, and the storing warps add the parts up.

The first part goes to the accumulator that the tile before did not begin with and stays there; the
others go to the other one, one after the other, each of which is added to the first and given back.
The model is that of the hand-off (test_product_protocol), in which a part is a tile that is told like
others; it asserts, beside what that asserts, that each storing warp of each block adds and stores whole
parts, all of them, and in their order.
"""
import random

import pytest

from test_product_protocol import STORERS, Cluster, Plain, depths, plain_depths


def flat(tiles):
    """[(depth, number of the tile, is it its first part, is it its last)]"""
    return [(d, i, p == 0, p == len(t) - 1) for i, t in enumerate(tiles) for p, d in enumerate(t)]


class Parts(Cluster):
    def __init__(self, tiles, weight, seed, planted=None):
        self.parts = flat(tiles)
        super().__init__(2, [p[0] for p in self.parts], weight, seed)
        self.planted = planted
        # what a storing warp's share of an accumulator holds: the turns summed up there
        self.held = {(c, s): [[], []] for c in range(2) for s in range(STORERS)}
        self.names = {c: iter(range(STORERS)) for c in range(2)}

    def accumulators(self):
        """For each turn (first, the one that the part goes to), or None without anything to sum."""
        first = 1
        for depth, _, begins, _ in self.parts:
            if depth:
                first ^= begins
            yield (first, first if begins else first ^ 1) if depth else None

    def mma(self, c):
        it, b = 0, self.bars[c]
        uses = {"full": [0] * self.depth, "ready": [0] * self.depth}
        taken = [0, 0]
        for turn, (depth, to) in enumerate(zip(self.tiles, self.accumulators())):
            yield from self.next(c, turn)
            stages = self.stages(depth)
            if not stages:
                continue
            buf = to[1]
            if taken[buf]:
                yield from self.wait(b["acc_empty"][buf], taken[buf] - 1)
            taken[buf] += 1
            for i, (place, tail) in enumerate(stages):
                s = (it + place) % self.depth
                name = "ready" if tail else "full"
                yield from self.wait(b[name][s], uses[name][s])
                uses[name][s] += 1
                self.pipes[0].append(("sum", turn, buf, i == 0))
                self.pipes[0].append(("read", s, it + place, tail, buf))
                self.pipes[0].append(("empty", s))
                if i == len(stages) - 1:
                    self.pipes[0].append(("acc", buf))
            it += len(stages)
        yield from self.next(c, len(self.tiles))

    def mma_step(self, p):
        if self.pipes[p][0][0] != "sum":
            return super().mma_step(p)
        _, turn, buf, begins = self.pipes[p].pop(0)
        for held in self.held.values():
            if begins:
                held[buf] = [turn]
            elif held[buf] != [turn]:
                self.errors.append(f"accumulator {buf} holds {held[buf]} in turn {turn}")

    def release(self, c, buf):
        self.acc_unread[0][buf] -= 1
        self.bars[0]["acc_empty"][buf].arrive()

    def storer(self, c):
        b, taken, mine = self.bars[c], [0, 0], self.held[c, next(self.names[c])]
        whole = []
        for turn, ((depth, _, begins, ends), to) in enumerate(zip(self.parts, self.accumulators())):
            yield from self.next(c, turn)
            if depth == 0:
                continue
            first, buf = to
            yield from self.wait(b["acc_full"][buf], taken[buf])
            taken[buf] += 1
            whole = [turn] if begins else whole + [turn]
            yield None
            if not begins:
                if self.planted == "early":  # given back before it is added
                    self.release(c, buf)
                    yield None
                if mine[first] != whole[:-1] or mine[buf] != [turn]:
                    self.errors.append(f"block {c} adds {mine[buf]} to {mine[first]} in turn {turn}")
                mine[first] = mine[first] + mine[buf]
                if self.planted != "early":
                    yield None
                    self.release(c, buf)
            if not ends:
                continue
            yield None
            if mine[first] != whole:
                self.errors.append(f"block {c} stores {mine[first]} for {whole}")
            self.release(c, first)
        yield from self.next(c, len(self.tiles))


def long_tiles(rnd, weight):
    """Tiles of one to six parts, all of them whole stages but the last."""
    tiles = []
    for d in depths(rnd, weight):
        more = rnd.choice([0, 0, 1, 2, 5]) if d else 0
        tiles.append([rnd.choice([1, 2, 7])] * more + [d])
    return tiles


@pytest.mark.parametrize("weight", [False, True])
def test_parts(weight):
    for seed in range(250):
        tiles = long_tiles(random.Random(3000 + seed), weight)
        errors = Parts(tiles, weight, seed).run()
        assert not errors, (seed, tiles, errors[:3])


def test_a_part_given_back_before_it_is_added_is_found():
    found = 0
    for seed in range(100):
        try:
            found += bool(Parts([[2, 2, 1], [1, 1, 1, 3.5]], True, seed, planted="early").run())
        except AssertionError:
            found += 1
    assert found


class PlainParts(Plain):
    """The same roles in one block."""

    def __init__(self, tiles, seed):
        self.parts = flat(tiles)
        super().__init__([p[0] for p in self.parts], seed)
        self.held = [[[], []] for _ in range(STORERS)]
        self.names = iter(range(STORERS))
        self.unread = [0, 0]

    accumulators = Parts.accumulators

    def plain_mma(self):
        it, taken = 0, [0, 0]
        for turn, (depth, to) in enumerate(zip(self.tiles, self.accumulators())):
            yield from self.next(0, turn)
            if depth == 0:
                continue
            buf = to[1]
            if taken[buf]:
                yield from self.wait(self.b["acc_empty"][buf], taken[buf] - 1)
            taken[buf] += 1
            for i in range(int(depth)):
                yield from self.wait(self.b["full"][it % 2], it // 2)
                if self.unread[buf]:
                    self.errors.append(f"accumulator {buf} written before it was read")
                for h in self.held:
                    h[buf] = [turn]
                self.b["empty"][it % 2].arrive()
                it += 1
                yield None
            self.unread[buf] = STORERS
            self.b["acc_full"][buf].arrive()
        yield from self.next(0, len(self.tiles))

    def plain_storer(self):
        taken, mine, whole = [0, 0], self.held[next(self.names)], []
        for turn, ((depth, _, begins, ends), to) in enumerate(zip(self.parts, self.accumulators())):
            yield from self.next(0, turn)
            if depth == 0:
                continue
            first, buf = to
            yield from self.wait(self.b["acc_full"][buf], taken[buf])
            taken[buf] += 1
            whole = [turn] if begins else whole + [turn]
            yield None
            for add in [True] * (not begins) + [False] * ends:
                if add:
                    mine[first] = mine[first] + mine[buf]
                elif mine[first] != whole:
                    self.errors.append(f"stores {mine[first]} for {whole}")
                yield None
                self.unread[buf if add else first] -= 1
                self.b["acc_empty"][buf if add else first].arrive()
        yield from self.next(0, len(self.tiles))


def test_parts_by_plain_loads():
    for seed in range(250):
        rnd = random.Random(seed)
        tiles = [[rnd.choice([1, 3])] * (rnd.choice([0, 1, 4]) if d else 0) + [d] for d in plain_depths(rnd)]
        errors = PlainParts(tiles, seed).run()
        assert not errors, (seed, tiles, errors[:3])
