"""How a block of the grouped product ends, checked on the CPU.

An arrival that MMAs bring to a barrier (tcgen05.commit) comes when they are done, on its own: it is
no step of the thread that asked for it, so neither the block's barrier nor the cluster's orders it, and
of several any may come first.  Each has to be waited for, in every block that it goes to, before
that block ends, or it would reach shared memory that is another's.

The model is that of the hand-off (test_product_protocol) with such arrivals on their way for any
time.  Which of them a role waits for behind its last tile (`finish`) is taken from the kernel's
source.
"""
import os
import random
import re

import pytest

from test_product_protocol import Bar, Cluster, Plain, depths, plain_depths

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "hyper_connection_mix_gb300", "csrc", "hcmix_product.cuh")
ROLES = ["plain loads: rows", "producer\n", "the last stage of an expert", "MMA\n", "epilogue", "the tiles, in turn"]


def ends():
    """{role: the barriers of its own block that it waits for behind its last tile, in all blocks or
    (with `leader`) in a pair's first alone}"""
    text = open(SOURCE).read()
    text = text[text.index("hcmix_product_kernel(const"):text.index("// ---- host side")]
    at = [text.index("// ---- " + r) for r in ROLES] + [len(text)]
    role = {r.strip(): re.sub(r"//[^\n]*", "", text[a:b]) for r, a, b in zip(ROLES, at, at[1:])}
    return {r: set(re.findall(r"finish\(C\.(\w+)", role[r])) for r in ("producer", "MMA")}


class PairExit(Cluster):
    def __init__(self, tiles, weight, seed, waits):
        super().__init__(2, tiles, weight, seed)
        self.waits, self.live, self.seen = waits, 0, 0
        self.used = sum(len(self.stages(d)) for d in tiles)
        for c in range(2):
            self.bars[c]["drain"] = [Bar(1, f"drain of block {c}")]
        # a barrier whose arrivals take longer than the others'
        self.slow = self.rnd.choice([b.name for bars in self.bars for n in ("empty", "acc_full", "drain") for b in bars[n]])

    def send(self, bar):
        self.copies.append(bar)

    def land(self, copy):
        if not isinstance(copy, Bar):
            return super().land(copy)
        if copy.name == self.slow and self.rnd.random() < 0.95:
            return self.send(copy)
        if self.live == 0:
            self.errors.append(f"{copy.name}: an arrival behind the block's end")
        copy.arrive()

    def mma_step(self, p):
        if self.pipes[p][0][0] == "read":
            return super().mma_step(p)
        op = self.pipes[p].pop(0)
        if op[0] == "acc":
            self.acc_unread[p][op[1]] = 2 * 2
        for c in range(2):
            self.send(self.bars[c][{"empty": "empty", "acc": "acc_full", "drain": "drain"}[op[0]]][op[1]])

    def ending(self, role, *last):
        """The role, with what it waits for at its end; blocks end with the last role of the pair."""
        self.live += 1

        def steps():
            yield from role
            for bar, phase in last:
                yield from self.wait(bar, phase)
            self.live -= 1
        return steps()

    def last(self, c, names):
        b = self.bars[c]
        some = [(b["empty"][i % self.depth], i // self.depth) for i in range(max(0, self.used - self.depth), self.used)]
        return (some if "empty" in names else []) + ([(b["drain"][0], 0)] if "drain" in names else [])

    def scheduler(self, c):
        return self.ending(super().scheduler(c))

    def storer(self, c):
        return self.ending(super().storer(c))

    def tailer(self, c, which):
        return self.ending(super().tailer(c, which))

    def producer(self, c):
        return self.ending(super().producer(c), *self.last(c, self.waits["producer"]))

    def mma(self, c):
        def steps(role):
            yield from role
            self.pipes[0].append(("drain", 0))
        return self.ending(steps(super().mma(c)), *self.last(c, self.waits["MMA"]))


@pytest.mark.parametrize("weight", [False, True])
def test_pairs(weight):
    waits = ends()
    for seed in range(150):
        tiles = depths(random.Random(2000 + seed), weight)
        errors = PairExit(tiles, weight, seed, waits).run()
        assert not errors, (seed, tiles, errors[:3])


STORERS = 2


class PlainExit(Plain):
    def __init__(self, tiles, seed, waits):
        super().__init__(tiles, seed)
        self.waits, self.flying = waits, []
        self.used = sum(int(d) for d in tiles)
        self.b["drain"] = [Bar(1, "drain")]

    def plain_mma(self):
        it = acc = 0
        for turn, depth in enumerate(self.tiles):
            yield from self.next(0, turn)
            if depth == 0:
                continue
            if acc >= 2:
                yield from self.wait(self.b["acc_empty"][acc % 2], acc // 2 - 1)
            for _ in range(int(depth)):
                yield from self.wait(self.b["full"][it % 2], it // 2)
                self.flying.append(self.b["empty"][it % 2])
                it += 1
            self.flying.append(self.b["acc_full"][acc % 2])
            acc += 1
        yield from self.next(0, len(self.tiles))
        self.flying.append(self.b["drain"][0])
        if "empty" in self.waits["MMA"]:
            for i in range(max(0, self.used - 2), self.used):
                yield from self.wait(self.b["empty"][i % 2], i // 2)
        if "drain" in self.waits["MMA"]:
            yield from self.wait(self.b["drain"][0], 0)

    def run(self):
        at = [(r, None) for r in [self.scheduler(0), self.plain_mma()] + [self.plain_storer() for _ in range(STORERS)]
              + [self.plain_producer() for _ in range(self.WARPS)]]
        while at and not self.errors:
            ready = [("role", i) for i, (_, w) in enumerate(at) if w is None or (w[0].phase & 1) != (w[1] & 1)]
            moves = ready + [("arrival", i) for i in range(len(self.flying))]
            assert moves, "deadlock: " + ", ".join(f"{w[0].name} phase {w[1]}" for _, w in at)
            kind, i = self.rnd.choice(moves)
            if kind == "arrival":
                self.flying.pop(i).arrive()
                continue
            try:
                at[i] = (at[i][0], next(at[i][0]))
            except StopIteration:
                at.pop(i)
        return self.errors + [f"{b.name}: an arrival behind the block's end" for b in self.flying]


def test_plain_loads():
    waits = ends()
    for seed in range(200):
        tiles = plain_depths(random.Random(seed))
        errors = PlainExit(tiles, seed, waits).run()
        assert not errors, (seed, tiles, errors[:3])


@pytest.mark.parametrize("missing", ["empty", "drain"])
def test_an_end_that_does_not_wait_is_found(missing):
    """Planted in the model: a role that leaves one kind of arrivals unwaited for."""
    waits = {r: {"empty", "drain"} - {missing} for r in ("producer", "MMA")}
    tiles = [3, 1, 7]
    assert any(PairExit(tiles, True, seed, waits).run() for seed in range(50))
    assert any(PlainExit(tiles, seed, waits).run() for seed in range(50))
