"""The pair kernel of the 4-bit products as a model on the CPU, in every order in which its parts may go on: the loading warps of both
CTAs, the warp that brings the tile of scales where k ends (of each CTA), the leader, which issues copies of scales,
products and commits that run in that order, and the warps that read the accumulators, three of them here (two of one CTA).
All states that can be reached are visited: nothing is overwritten before it has been read, everything is there when it is
used, every wait is for the phase that it means, and nobody waits for ever.

When a load lands matters to nothing but the wait for its stage, so it counts as landed when it is started, and the
leader waits for both CTAs'. Parities, commits and the order of the waits are a copy of the kernel's by hand; the numbers
of slots and the columns of the accumulators are read from its source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_precision_activation_gb300", "csrc")
with open(os.path.join(CSRC, "rmsq_fp4_pair.cuh")) as f:
    SOURCE = f.read()
SLOTS, LESS = (int(v) for v in re.search(r"SLOTS = (\d+), SCALE_SLOTS = SLOTS - (\d+);", SOURCE).groups())
SECOND = int(re.search(r"SECOND = (\d+);", SOURCE).group(1))
COLUMNS = 256


class Broken(Exception):
    pass


def need(truth, what):
    if not truth:
        raise Broken(what)


def passed(phases, parity):
    """Whether a wait for the phase of that parity passes, on a barrier that has finished so many phases."""
    return phases & 1 != parity


class Model:
    """A state is a tuple: (stages loaded by each CTA, tails brought by each CTA, the leader's place, commands run, each reader's place).
    The leader's place counts its steps, two to a stage (copy, multiply); a reader's two to a tile (the shared columns,
    the rest). Everything else follows from these: barriers from the commits and arrivals so far."""

    def __init__(self, tiles, steps, tail, slots=SLOTS, less=LESS, wait_free=True):
        self.tiles, self.steps, self.tail, self.slots, self.scale_slots = tiles, steps, tail, slots, slots - less
        self.stages, self.wait_free = tiles * steps, wait_free
        # the commands behind the leader's steps, in the order in which they run
        self.commands, self.until = [], [0]
        for g in range(self.stages):
            self.commands += [("copy", g), ("codes", (g - 1) % slots)]
            self.until.append(len(self.commands))
            self.commands.append(("multiply", g))
            if (g + 1) % steps == 0:
                self.commands.append(("tile", g // steps))
            self.until.append(len(self.commands))
        # what has been done after so many commands
        n = len(self.commands) + 1
        self.copied, self.multiplied, self.full_tiles = [0] * n, [0] * n, [0] * n
        self.empty = [[0] * slots for _ in range(n)]
        for i, (kind, at) in enumerate(self.commands):
            self.copied[i + 1] = self.copied[i] + (kind == "copy")
            self.multiplied[i + 1] = self.multiplied[i] + (kind == "multiply")
            self.full_tiles[i + 1] = self.full_tiles[i] + (kind == "tile")
            self.empty[i + 1] = [v + (kind == "codes" and s == at) for s, v in enumerate(self.empty[i])]

    start = ((0, 0), (0, 0), 0, 0, (0, 0, 0))

    def acc_full(self, run, buffer):
        return (self.full_tiles[run] + 1 - buffer) // 2          # phases: tiles 0, 2, ... or 1, 3, ...

    def next(self, state):
        loaded, tails, place, run, readers = state
        # each CTA's loads: stage j
        for c in (0, 1):
            j = loaded[c]
            if j == self.stages:
                continue
            slot, turn = j % self.slots, j // self.slots
            if passed(self.empty[run][slot], turn & 1 if slot == self.slots - 1 else (turn & 1) ^ 1):
                need(j < self.slots or self.multiplied[run] > j - self.slots, "codes still needed")
                need(j < self.scale_slots or self.copied[run] > j - self.scale_slots, "scales still needed")
                yield (loaded[:c] + (j + 1,) + loaded[c + 1:], tails, place, run, readers)
        # each CTA's tails: tile t
        for c in (0, 1):
            t = tails[c]
            if not self.tail or t == self.tiles:
                continue
            if t == 0 or passed(self.acc_full(run, (t - 1) & 1), ((t - 1) >> 1) & 1):
                need(t == 0 or self.copied[run] >= t * self.steps, "the last tile's tail still needed")
                yield (loaded, tails[:c] + (t + 1,) + tails[c + 1:], place, run, readers)
        # the leader's next step
        if place < 2 * self.stages:
            g = place // 2
            tile, first, last = g // self.steps, g % self.steps == 0, (g + 1) % self.steps == 0
            go = True
            if place % 2 == 0:
                go = min(loaded) > g                                       # its stage is there, and the tail
                if go and self.tail and last:
                    go = passed(min(tails), tile & 1)
                    need(not go or min(tails) == tile + 1, "a tail of another tile")
            elif first and tile > 0 and self.wait_free:
                freed = sum(r > 2 * (tile - 1) for r in readers) == len(readers)
                arrived = min((r + 1) // 2 for r in readers)               # phases of acc_free that are over
                go = passed(arrived, (tile - 1) & 1)
                need(not go or freed, "the shared columns still needed")
            if go:
                yield (loaded, tails, place + 1, run, readers)
        # the next command that was issued
        if run < self.until[place]:
            kind, at = self.commands[run]
            if kind == "copy":
                need(min(loaded) > at and max(loaded) <= at + self.scale_slots, "another stage's scales")
                need(not self.tail or (at + 1) % self.steps or min(tails) == max(tails) == at // self.steps + 1, "another tile's tail")
            elif kind == "multiply":
                need(min(loaded) > at and max(loaded) <= at + self.slots, "another stage's codes")
                tile = at // self.steps
                need(tile < 1 or min(readers) >= 2 * tile - 1, "the last accumulator's shared columns are overwritten")
                need(tile < 2 or min(readers) >= 2 * (tile - 1), "an accumulator is overwritten")
            yield (loaded, tails, place, run + 1, readers)
        # each reader's next part
        for i, r in enumerate(readers):
            tile = r // 2
            if tile == self.tiles:
                continue
            if r % 2 or passed(self.acc_full(run, tile & 1), (tile >> 1) & 1):
                need(self.full_tiles[run] > tile, "an accumulator that is not complete")
                yield (loaded, tails, place, run, readers[:i] + (r + 1,) + readers[i + 1:])

    def done(self, state):
        loaded, tails, place, run, readers = state
        return (min(loaded) == self.stages and run == len(self.commands) and min(readers) == 2 * self.tiles
                and (not self.tail or min(tails) == self.tiles))

    def explore(self):
        seen, todo, ended = {self.start}, [self.start], 0
        while todo:
            state = todo.pop()
            after = list(self.next(state))
            if not after:
                need(self.done(state), "everybody waits")
                ended += 1
            for s in after:
                if s not in seen:
                    seen.add(s)
                    todo.append(s)
        assert ended == 1
        return len(seen)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tiles,steps", [(1, 1), (5, 1), (4, 2), (3, 3), (2, 7), (2, 6), (1, 14)])
def test_every_order(tiles, steps, tail):
    Model(tiles, steps, tail).explore()


@pytest.mark.parametrize("change", [dict(less=LESS + 1), dict(wait_free=False)])
def test_less_would_not_do(change):
    # one slot of scales fewer; products that do not wait for the shared columns
    with pytest.raises(Broken):
        Model(3, 3, True, **change).explore()


def test_the_shared_columns_are_read_first():
    # of 8 parts of 32 columns, each of two groups of warps reads two at a time: those of the first step hold the shared ones
    assert re.search(r"c0 = b == 0 \? 6 \+ wg - 2 \* i : wg \+ 2 \* i, c1 = b == 0 \? c0 - 2 : c0 \+ 2;", SOURCE)
    shared = set(range(SECOND, COLUMNS))
    for b in (0, 1):
        steps = []
        for i in (0, 2):
            at = set()
            for wg in (0, 1):
                c0 = 6 + wg - 2 * i if b == 0 else wg + 2 * i
                for c in (c0, c0 - 2 if b == 0 else c0 + 2):
                    at |= set(range(b * SECOND + 32 * c, b * SECOND + 32 * c + 32))
            steps.append(at)
        assert shared <= steps[0] and not shared & steps[1]
        assert steps[0] | steps[1] == set(range(b * SECOND, b * SECOND + COLUMNS)) and not steps[0] & steps[1]
