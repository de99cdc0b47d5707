"""CPU model of the barriers of cross attention's dK/dV kernel.

The roles of a block (load warps of the T0 and T1 slots, tensor-core warp, compute warps) run as coroutines
over mbarriers with phases and parities, in random orders with one role held back at a time, as a block's
warps may be on the GPU.  Copies land and products complete at any later time, products in order.  The model
checks that a compute warp reads the statistics of its own step, and that no wait is for a phase that has gone
round.  Releasing the T1 slot by its product alone, without the barrier of its statistics, fails it."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "streaming_causal_video_gb300", "csrc", "cross_backward.cu")).read()
COMPUTE = 3                    # compute warps of the model


class Wrong(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.bytes = 0
        self.done = 0                          # completed phases

    def arrive(self, expect=0):
        self.left -= 1
        self.bytes += expect
        self.settle()

    def land(self):
        self.bytes -= 1
        self.settle()

    def settle(self):
        if self.left == 0 and self.bytes == 0:
            self.done += 1
            self.left = self.count

    def passed(self, parity):
        """mbarrier.try_wait.parity: the phase with this parity has completed, and the next has not."""
        return (self.done & 1) != parity


class Block:
    """One unit of `steps` streamed tiles; t0, t1: slots of each ring; ordered: the statistics of a T1 slot
    have a barrier of their own."""

    def __init__(self, steps, t0, t1, ordered, rng):
        self.steps, self.t0, self.t1, self.ordered, self.rng = steps, t0, t1, ordered, rng
        one = lambda n: [Barrier(1) for _ in range(n)]
        self.t0full, self.t0empty, self.t1full, self.t1empty, self.dfree = one(t0), one(t0), one(t1), one(t1), one(t1)
        self.sfull, self.dpfull = Barrier(1), Barrier(1)
        self.sread, self.dsfull = Barrier(COMPUTE), Barrier(COMPUTE)
        self.lse, self.delta = [None] * t0, [None] * t1
        self.tensor = []                       # products and commits that have been issued, in order
        self.copies = []                       # (what it does when it lands)

    def copy(self, bar, then=None):
        self.copies.append((bar, then))

    def load(self, first):
        nst = self.t0 if first else self.t1
        full, empty = (self.t0full, self.t0empty) if first else (self.t1full, self.t1empty)
        stats = self.lse if first else self.delta
        for i in range(self.steps):
            slot, phase = i % nst, (i // nst) & 1
            yield empty[slot], phase ^ 1, i // nst
            full[slot].arrive(expect=2)
            self.copy(full[slot])
            if self.ordered and not first:
                yield self.dfree[slot], phase ^ 1, i // nst

            def put(slot=slot, i=i):
                stats[slot] = i
            self.copy(full[slot], put)

    def mma(self):
        def s(i):
            yield self.t0full[i % self.t0], (i // self.t0) & 1, i // self.t0 + 1
            self.tensor.append(self.sfull)

        def dp(i):
            yield self.t1full[i % self.t1], (i // self.t1) & 1, i // self.t1 + 1
            self.tensor.append(self.dpfull)
        yield from s(0)
        yield from dp(0)
        for i in range(self.steps):
            yield self.sread, i & 1, i + 1
            self.tensor.append(self.t1empty[i % self.t1])
            if i + 1 < self.steps:
                yield from s(i + 1)
            yield self.dsfull, i & 1, i + 1
            self.tensor.append(self.t0empty[i % self.t0])
            self.dfree[i % self.t1].arrive()
            if i + 1 < self.steps:
                yield from dp(i + 1)

    def compute(self):
        for i in range(self.steps):
            yield self.t0full[i % self.t0], (i // self.t0) & 1, i // self.t0 + 1
            yield self.sfull, i & 1, i + 1
            if self.lse[i % self.t0] != i:
                raise Wrong("-lse of step %d read as of step %r" % (i, self.lse[i % self.t0]))
            self.sread.arrive()
            yield self.t1full[i % self.t1], (i // self.t1) & 1, i // self.t1 + 1
            yield self.dpfull, i & 1, i + 1
            if self.delta[i % self.t1] != i:
                raise Wrong("-delta of step %d read as of step %r" % (i, self.delta[i % self.t1]))
            self.dsfull.arrive()

    def run(self):
        roles = [self.load(True), self.load(False), self.mma()] + [self.compute() for _ in range(COMPUTE)]
        waits = [None] * len(roles)
        alive = set(range(len(roles)))
        held = None

        def step(r):
            try:
                waits[r] = next(roles[r])
            except StopIteration:
                alive.discard(r)
        for r in list(alive):
            step(r)
        while alive:
            if self.rng.random() < 0.05:
                held = self.rng.randrange(len(roles))
            moves = []
            for r in alive:
                bar, parity, phases = waits[r]
                if bar.done > phases:
                    raise Wrong("a wait for phase %d finds %d complete" % (phases, bar.done))
                if bar.passed(parity):
                    moves.append(r)
            others = [r for r in moves if r != held] + (["tensor"] if self.tensor else []) + (["copy"] if self.copies else [])
            pick = self.rng.choice(others or moves or [None])
            if pick is None:
                raise Wrong("every role waits")
            if pick == "tensor":
                self.tensor.pop(0).arrive()
            elif pick == "copy":
                bar, then = self.copies.pop(self.rng.randrange(len(self.copies)))
                if then:
                    then()
                bar.land()
            else:
                step(pick)


def rings():
    t0 = int(re.search(r"constexpr int T0ST = (\d+);", SOURCE).group(1))
    t1 = int(re.search(r"constexpr int T1ST = DKV \? (\d+) : \d+;", SOURCE).group(1))
    return t0, t1


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7, 13])
def test_statistics_are_read_before_their_slot_is_copied_again(steps):
    t0, t1 = rings()
    for seed in range(300):
        Block(steps, t0, t1, True, random.Random(seed)).run()


def test_the_model_finds_a_slot_that_its_product_alone_releases():
    t0, t1 = rings()
    found = set()
    for seed in range(300):
        try:
            Block(7, t0, t1, False, random.Random(seed)).run()
        except Wrong as e:
            found.add(str(e).split(" ")[0])
    assert found == {"-delta", "a"}            # another step's statistics, and a wait whose phase has gone round


def test_the_kernel_waits_and_arrives_as_the_model_does():
    assert re.search(r"!t0 && !mbar_wait_bounded\(bar\(DFREE \+ slot\), phase \^ 1u, tmo, abort_flag\)\) ok = false;\s*"
                     r"bulk_load\(", SOURCE)
    body = SOURCE[SOURCE.index("if (!wait(DSFULL, count & 1u)) break;"):]
    assert "mbar_arrive_warp(bar(DFREE + a_slot1));" in body[:body.index("ACCFULL")]


@pytest.mark.parametrize("dkv", [True, False])
def test_rows_that_are_zeroed_at_the_start_belong_to_query_tiles(dkv):
    """A block's compute warps zero the rows of query tiles that no load writes.  Nothing orders that with the loads,
    which write the other rows of those tiles, and whole tiles of keys."""
    assert re.search(r"sT0 = sR \+ 2 \* TILE, sT1 = sT0 \+ T0ST \* TILE;", SOURCE)
    t0, t1 = rings()
    held, streamed = {0, 1}, set(range(2, 2 + t0 + (t1 if dkv else 1)))
    queries = streamed if dkv else held
    first, tiles = re.search(r"kFirst = DKV \? (\d+) : (\d+), kTiles = DKV \? T0ST \+ (\d+) : (\d+);", SOURCE).group(
        *((1, 3) if dkv else (2, 4)))
    assert "i < (BM - used_rows) * 16 * kTiles;" in SOURCE and "smem + (kFirst + tile) * TILE +" in SOURCE
    assert set(range(int(first), int(first) + int(tiles) + (t0 if dkv else 0))) == queries
