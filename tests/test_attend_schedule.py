"""The order of attend_rows' products, softmax and reads of its sums
(kv_cache_injection_gather_b200/csrc/attend_rows.cuh), as a model of its
threads and mbarriers run under random delays: tensor-core products and
copies finish whenever they like, products in the order of their issue.

A wait on a barrier names a phase by its parity alone: with phase n open it
returns at once for phase n - 1, and for phase n + 1 just as well, whose parity
is the same.  A wait for phase n is therefore sound only where phase n - 1 is
known to be done.
"""
from __future__ import annotations

import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_injection_gather_b200",
                    "csrc")


class Barrier:
    def __init__(self):
        self.phase = 0

    def arrive(self):
        self.phase += 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Model:
    """One CTA.  `drain`: the products' thread waits for all of them before
    the threads meet; otherwise the softmax waits for the last phase of the
    sums' barrier."""

    def __init__(self, rng, tiles, slots, drain):
        self.rng, self.tiles, self.slots, self.drain = rng, tiles, slots, drain
        self.full = [Barrier() for _ in range(slots)]
        self.empty = [Barrier() for _ in range(slots)]
        self.s, self.p, self.o, self.end = [Barrier(), Barrier()], [Barrier(), Barrier()], Barrier(), Barrier()
        self.queue = []           # tensor cores: products and commits in order
        self.scores, self.sums = 0, 0   # products done
        self.issued = 0           # sums issued
        self.meeting = 0
        self.faults = set()
        slow = rng.choice([1, 1, 30])  # the copies may be what takes long
        self.copy_delay = lambda: rng.randrange(0, 1 + 20 * slow)
        self.product_delay = lambda: rng.randrange(0, rng.choice([2, 60]))

    def gather(self):
        for u in range(2 * self.tiles):
            slot = u % self.slots
            if u >= self.slots:
                yield lambda: self.empty[slot].done((u // self.slots - 1) & 1)
            for _ in range(self.copy_delay()):
                yield None
            self.full[slot].arrive()

    def commit(self, barrier):
        self.queue.append((0, barrier.arrive))

    def products(self):
        def scores(t):
            slot = (2 * t) % self.slots
            yield lambda: self.full[slot].done((2 * t // self.slots) & 1)

            def finish():
                self.scores += 1
            self.queue.append((self.product_delay(), finish))
            self.commit(self.s[t & 1])
            self.commit(self.empty[slot])

        if self.tiles:
            yield from scores(0)
            for t in range(self.tiles):
                if t + 1 < self.tiles:
                    yield from scores(t + 1)
                yield lambda: self.p[t & 1].done((t >> 1) & 1)
                slot = (2 * t + 1) % self.slots
                yield lambda: self.full[slot].done(((2 * t + 1) // self.slots) & 1)

                def finish():
                    self.sums += 1
                self.issued += 1
                self.queue.append((self.product_delay(), finish))
                self.commit(self.empty[slot])
                self.commit(self.o)
            if self.drain:
                self.commit(self.end)
                yield lambda: self.end.done(0)
        self.meeting += 1

    def tensor_cores(self):
        while True:
            if not self.queue:
                yield None
                continue
            delay, finish = self.queue.pop(0)
            for _ in range(delay):
                yield None
            finish()

    def softmax(self):
        for t in range(self.tiles):
            yield lambda: self.s[t & 1].done((t >> 1) & 1)
            if self.scores < t + 1:
                self.faults.add("scores read before they are there")
            for _ in range(self.rng.randrange(0, 20)):
                yield None
            if self.rng.random() < 0.3 and t > 0:  # the reference moves
                yield lambda: self.o.done((t - 1) & 1)
                if self.sums != t or self.issued != t:
                    self.faults.add("sums scaled under way")
            if t >= 2 and self.sums < t - 1:
                self.faults.add("probabilities overwritten")
            self.p[t & 1].arrive()
        if self.tiles and not self.drain:
            yield lambda: self.o.done((self.tiles - 1) & 1)
        self.meeting += 1
        yield lambda: self.meeting == 2
        if self.sums != self.tiles:
            self.faults.add("sums read under way")

    def run(self):
        threads = [iter(x()) for x in (self.gather, self.products, self.tensor_cores, self.softmax)]
        waits = [None] * 4
        alive = {0, 1, 2, 3}
        for _ in range(1_000_000):
            if alive == {2}:
                return self.faults
            i = self.rng.choice(sorted(alive))
            if waits[i] is not None and not waits[i]():
                continue
            try:
                waits[i] = next(threads[i])
            except StopIteration:
                alive.discard(i)
        raise AssertionError("the model hangs")


def faults(drain, seeds):
    found = set()
    for seed in seeds:
        rng = random.Random(seed)
        found |= Model(rng, rng.randint(0, 9), rng.choice([3, 6, 10, 16]), drain).run()
    return found


def test_the_sums_are_read_once_all_products_are_done():
    assert faults(True, range(1500)) == set()


def test_a_wait_for_the_last_phase_alone_returns_early():
    # the scores of the last tile are issued ahead of the sums of the one
    # before, whose phase nothing waits for
    assert faults(False, range(1500)) == {"sums read under way"}


def test_the_kernels_drain_their_products_on_every_path():
    """What the model takes as given: the products' thread commits to a
    barrier of its own and waits for it, failed or not."""
    for name in ("attend_rows.cuh", "attend_tiles.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        branch = text[text.index("// ---------------- products"):text.index("// ---------------- softmax")]
        after = branch[branch.rindex("tc_commit(&bar_"):]
        assert after.startswith("tc_commit(&bar_end"), name
        assert re.search(r"bar_wait\(&bar_end(\[st\])?, 0, nullptr\)", after), name
        loop = branch[branch.rindex("for (int32_t"):]
        depth = 0
        for line in loop[:loop.index("tc_commit(&bar_end")].splitlines():
            depth += line.count("{") - line.count("}")
        assert depth == 0, f"{name}: the last commit is inside the loop or a condition"
