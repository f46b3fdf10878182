"""The grouped product's hand-off protocol, checked on the CPU.

A cluster's roles (in each block: the producer of copies, the warp that tells the tiles, the warps
that zero behind an expert's last rows, the warps that store; in each pair's first block: the warp
that issues the MMAs) hand stages and accumulators to each other through mbarriers whose waits
only test the parity of the phase they want.  Such a wait is sound only when the waiter has seen
the phase before it end.  This module restates, role by role, the waits and arrivals of
hyper_connection_mix_gb300/csrc/hcmix_product.cuh as a model with real parity semantics, runs it
under random interleavings with the MMAs completing in issue order and the copies landing in any
order, and asserts
  * for every wait, that the exact phase it needed had completed, and that no barrier gets more
    arrivals than it expects;
  * for every stage, that it is only written once the MMAs that read it are done, in every block
    that a copy is sent to, and only read whole and with its tail zeroed;
  * for every accumulator, that it is only written once its storing warps have read it;
  * that every run finishes.
It is a model of the kernel's protocol, kept beside the kernel; the GPU tests check the kernel.
"""
import random

import pytest

QUEUE, LEAD, STORERS = 4, 3, 2  # STORERS: two stand for a block's eight or sixteen


class Bar:
    def __init__(self, count, name):
        self.count, self.pending, self.tx, self.phase, self.name = count, count, 0, 0, name

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, expect=0):
        self.pending -= 1
        self.tx += expect
        assert self.pending >= 0, f"{self.name}: more arrivals than expected"
        self._turn()

    def complete(self, n):
        self.tx -= n
        self._turn()


class Cluster:
    def __init__(self, ctas, depths, weight, seed, planted=None):
        """`depths`: of each tile, in stages and, as a half, a last one that is not whole."""
        self.rnd, self.ctas, self.tiles, self.weight, self.planted = random.Random(seed), ctas, depths, weight, planted
        self.depth = 6
        self.copies, self.pipes = [], [[] for _ in range(ctas // 2)]
        self.errors = []
        tailers = 2 if weight else 0
        self.bars = []
        for c in range(ctas):
            lead = c % 2 == 0
            mk = lambda n, count, what: [Bar(count, f"{what}{i} of block {c}") for i in range(n)]  # noqa: E731
            self.bars.append({
                "told": mk(QUEUE, 1, "told"), "taken": mk(QUEUE, STORERS + 1 + lead + tailers, "taken"),
                "full": mk(self.depth, 1, "full"), "empty": mk(self.depth, ctas // 2, "empty"),
                "tail": mk(self.depth, 1, "tail"), "ready": mk(self.depth, 4, "ready"),
                "acc_full": mk(2, 1, "acc_full"), "acc_empty": mk(2, 2 * STORERS, "acc_empty")})
        # per block and slot: what lies there, and the MMAs (a pair's) that still have to read it
        self.stage = [[{"it": None, "parts": 0, "zeroed": False, "readers": 0} for _ in range(self.depth)] for _ in range(ctas)]
        self.acc_unread = [[0, 0] for _ in range(ctas // 2)]

    # ---- roles, as generators that yield (barrier, phase) where they wait

    def wait(self, bar, phase):
        yield bar, phase
        if bar.phase <= phase:
            self.errors.append(f"{bar.name}: phase {phase} taken for done at {bar.phase}")

    def next(self, c, turn):
        b = self.bars[c]
        yield from self.wait(b["told"][turn % QUEUE], turn // QUEUE)
        b["taken"][turn % QUEUE].arrive()

    def scheduler(self, c):
        b = self.bars[c]
        for turn in range(len(self.tiles) + 1):
            if turn >= QUEUE:
                yield from self.wait(b["taken"][turn % QUEUE], turn // QUEUE - 1)
            b["told"][turn % QUEUE].arrive()

    def stages(self, depth):
        """(place in the ring, whether it is a tail), in the order in which they are multiplied;
        they are copied in the order of their places."""
        whole = int(depth)
        if depth == whole or not self.weight:
            return [(i, False) for i in range(whole + (depth > whole))]
        tail = max(0, whole - LEAD)
        return [(i, False) for i in range(whole + 1) if i != tail] + [(tail, True)]

    def producer(self, c):
        it, b = 0, self.bars[c]
        lead = self.bars[c & ~1]
        used = {"full": [0] * self.depth, "tail": [0] * self.depth}
        for turn, depth in enumerate(self.tiles):
            yield from self.next(c, turn)
            for _, tail in sorted(self.stages(depth)):
                s = it % self.depth
                if it >= self.depth:
                    yield from self.wait(b["empty"][s], it // self.depth - 1)
                name = "tail" if tail else "full"
                shares = self.ctas // 2   # A and this block's part of its share of B; the rest is sent here
                if tail:
                    b["tail"][s].arrive(expect=1 + shares)
                elif c % 2 == 0:
                    b["full"][s].arrive(expect=2 * (1 + shares))
                yield None
                self.copies.append((c, s, it, [c], name))
                self.copies.append((c, s, it, [c % 2 + 2 * p for p in range(shares)], name))
                used[name][s] += 1
                it += 1
        yield from self.next(c, len(self.tiles))

    def land(self, copy):
        c, s, it, to, name = copy
        for d in to:
            st = self.stage[d][s]
            if st["it"] != it:
                if st["readers"]:
                    self.errors.append(f"stage {s} of block {d} overwritten before it was read")
                st.update(it=it, parts=0, zeroed=False, readers=1)
            st["parts"] += 1
            self.bars[d if name == "tail" else d & ~1][name][s].complete(1)

    def tailer(self, c, which):
        it, tails, b = 0, 0, self.bars[c]
        uses = [0] * self.depth
        for turn, depth in enumerate(self.tiles):
            yield from self.next(c, turn)
            stages = self.stages(depth)
            it += len(stages)
            if depth == int(depth):
                continue
            mark = it - len(stages) + stages[-1][0]
            s = mark % self.depth
            phase, mine = uses[s], tails % 2 == which
            uses[s] += 1
            tails += 1
            if self.planted == "skip" and not mine:
                self.bars[c & ~1]["ready"][s].arrive()
                continue
            yield from self.wait(b["tail"][s], phase)
            if not mine:
                self.bars[c & ~1]["ready"][s].arrive()
                continue
            st = self.stage[c][s]
            if st["it"] != mark or st["parts"] != 1 + self.ctas // 2:
                self.errors.append(f"zeroed behind stage {s} of block {c} before its copies had landed")
            st["zeroed"] = True
            yield None
            self.bars[c & ~1]["ready"][s].arrive()
        yield from self.next(c, len(self.tiles))

    def mma(self, c):
        it, acc, b, p = 0, 0, self.bars[c], c // 2
        uses = {"full": [0] * self.depth, "ready": [0] * self.depth}
        for turn, depth in enumerate(self.tiles):
            yield from self.next(c, turn)
            stages = self.stages(depth)
            if not stages:
                continue
            buf = acc % 2
            if acc >= 2:
                yield from self.wait(b["acc_empty"][buf], acc // 2 - 1)
            for i, (place, tail) in enumerate(stages):
                s = (it + place) % self.depth
                name = "ready" if tail else "full"
                yield from self.wait(b[name][s], uses[name][s])
                uses[name][s] += 1
                self.pipes[p].append(("read", s, it + place, tail, buf))
                self.pipes[p].append(("empty", s))
                if i == len(stages) - 1:
                    self.pipes[p].append(("acc", buf))
            it += len(stages)
            acc += 1
        yield from self.next(c, len(self.tiles))

    def mma_step(self, p):
        op = self.pipes[p].pop(0)
        if op[0] == "read":
            _, s, it, tail, buf = op
            if self.acc_unread[p][buf]:
                self.errors.append(f"accumulator {buf} of pair {p} written before it was read")
            for c in (2 * p, 2 * p + 1):
                st = self.stage[c][s]
                if st["it"] != it or st["parts"] != 1 + self.ctas // 2:
                    self.errors.append(f"stage {s} of block {c} read before it was whole")
                if tail and not st["zeroed"]:
                    self.errors.append(f"stage {s} of block {c} read before its tail was zeroed")
                st["readers"] = 0
        elif op[0] == "empty":
            for c in range(self.ctas):
                self.bars[c]["empty"][op[1]].arrive()
        else:
            self.acc_unread[p][op[1]] = 2 * STORERS
            for c in (2 * p, 2 * p + 1):
                self.bars[c]["acc_full"][op[1]].arrive()

    def storer(self, c):
        acc, b = 0, self.bars[c]
        for turn, depth in enumerate(self.tiles):
            yield from self.next(c, turn)
            if depth == 0:
                continue
            buf = acc % 2
            yield from self.wait(b["acc_full"][buf], acc // 2)
            yield None
            self.acc_unread[c // 2][buf] -= 1
            self.bars[c & ~1]["acc_empty"][buf].arrive()
            acc += 1
        yield from self.next(c, len(self.tiles))

    def run(self):
        roles = []
        for c in range(self.ctas):
            roles += [self.scheduler(c), self.producer(c)] + [self.storer(c) for _ in range(STORERS)]
            roles += [self.tailer(c, w) for w in range(2)] if self.weight else []
            roles += [self.mma(c)] if c % 2 == 0 else []
        at = [(r, None) for r in roles]
        slow = self.rnd.randrange(len(at))  # a role that lags behind the others
        while (at or self.copies or any(self.pipes)) and not self.errors:
            ready = [i for i, (_, w) in enumerate(at) if w is None or (w[0].phase & 1) != (w[1] & 1)]
            moves = [("role", i) for i in ready] + [("copy", i) for i in range(len(self.copies))]
            moves += [("mma", p) for p, pipe in enumerate(self.pipes) if pipe]
            assert moves, "deadlock: " + ", ".join(f"{w[0].name} phase {w[1]}" for _, w in at)
            kind, i = self.rnd.choice(moves)
            if kind == "copy":
                self.land(self.copies.pop(i))
            elif kind == "mma":
                self.mma_step(i)
            else:
                if i == slow and len(ready) > 1 and self.rnd.random() < 0.9:
                    continue
                role = at[i][0]
                try:
                    at[i] = (role, next(role))
                except StopIteration:
                    at.pop(i)
                    slow = -1 if i == slow else slow - (i < slow)
        return self.errors


def depths(rnd, weight):
    if not weight:
        k = rnd.choice([0.5, 1, 1.5, 3, 7, 12.5])  # the same for every tile
        return [k] * rnd.randint(1, 14)
    return [rnd.choice([0, 0, 0.5, 0.5, 1, 1.5, 2, 4.5, 5.5, 6, 6.5, 12.5]) for _ in range(rnd.randint(1, 14))]


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("ctas", [2, 4])
def test_protocol(ctas, weight):
    for seed in range(150):
        tiles = depths(random.Random(1000 + seed), weight)
        errors = Cluster(ctas, tiles, weight, seed).run()
        assert not errors, (seed, tiles, errors[:3])


def test_a_warp_that_does_not_wait_for_the_others_stages_is_found():
    """It loses count of the phases: the model tells."""
    found = 0
    for seed in range(200):
        tiles = depths(random.Random(1000 + seed), True)
        try:
            found += bool(Cluster(2, tiles, True, seed, planted="skip").run())
        except AssertionError:
            found += 1
    assert found


# ------------------------------------------------------------------------------- plain loads


class Plain(Cluster):
    """One block whose producers copy rows ahead of the stage that they place: up to RAW stages, and
    only of tiles that have been told, while they have one to place."""
    RAW, WARPS = 3, 2

    def __init__(self, depths, seed, planted=None):
        self.rnd, self.tiles, self.weight, self.planted = random.Random(seed), depths, False, planted
        self.errors, self.pipe, self.filled = [], [], [0, 0]
        mk = lambda n, count, what: [Bar(count, f"{what}{i}") for i in range(n)]  # noqa: E731
        self.b = {"told": mk(QUEUE, 1, "told"), "taken": mk(QUEUE, 1 + STORERS + self.WARPS, "taken"),
                  "full": mk(2, self.WARPS, "full"), "empty": mk(2, 1, "empty"),
                  "acc_full": mk(2, 1, "acc_full"), "acc_empty": mk(2, STORERS, "acc_empty")}
        self.bars = [self.b]

    def plain_producer(self):
        copied = placed = left = turn = 0
        more = True
        while True:
            while more and copied - placed < self.RAW:
                while left == 0 and more:
                    told = self.b["told"][turn % QUEUE].phase > turn // QUEUE
                    if not told and copied > placed and self.planted is None:
                        break
                    yield from self.next(0, turn)
                    more = turn < len(self.tiles)
                    left = int(self.tiles[turn]) if more else 0
                    turn += 1
                if left == 0:
                    break
                left, copied = left - 1, copied + 1
            if copied == placed:
                return
            if placed >= 2:
                yield from self.wait(self.b["empty"][placed % 2], placed // 2 - 1)
            yield None
            self.b["full"][placed % 2].arrive()
            placed += 1

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
                self.b["empty"][it % 2].arrive()
                it += 1
            self.b["acc_full"][acc % 2].arrive()
            acc += 1
        yield from self.next(0, len(self.tiles))

    def plain_storer(self):
        acc = 0
        for turn, depth in enumerate(self.tiles):
            yield from self.next(0, turn)
            if depth == 0:
                continue
            yield from self.wait(self.b["acc_full"][acc % 2], acc // 2)
            self.b["acc_empty"][acc % 2].arrive()
            acc += 1
        yield from self.next(0, len(self.tiles))

    def run(self):
        at = [(r, None) for r in [self.scheduler(0), self.plain_mma()] + [self.plain_storer() for _ in range(STORERS)]
              + [self.plain_producer() for _ in range(self.WARPS)]]
        while at and not self.errors:
            ready = [i for i, (_, w) in enumerate(at) if w is None or (w[0].phase & 1) != (w[1] & 1)]
            assert ready, "deadlock: " + ", ".join(f"{w[0].name} phase {w[1]}" for _, w in at)
            i = self.rnd.choice(ready)
            try:
                at[i] = (at[i][0], next(at[i][0]))
            except StopIteration:
                at.pop(i)
        return self.errors


def plain_depths(rnd):
    """Runs of tiles without anything to multiply among others."""
    return [d for _ in range(rnd.randint(1, 8)) for d in [0] * rnd.choice([0, 0, 1, 5, 9]) + [rnd.choice([1, 1, 2, 7])]]


def test_plain_loads():
    for seed in range(200):
        tiles = plain_depths(random.Random(seed))
        errors = Plain(tiles, seed).run()
        assert not errors, (seed, tiles, errors[:3])


def test_plain_loads_that_wait_for_a_tile_with_a_stage_in_hand_are_found():
    found = 0
    for seed in range(50):
        try:
            found += bool(Plain(plain_depths(random.Random(seed)), seed, planted="wait").run())
        except AssertionError:
            found += 1
    assert found
