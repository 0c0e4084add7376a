"""The waits of the tcgen05 kernels of 8-bit products (csrc/gemm_fp8.cu), as a model on the host: what they do when one runs out.

Each role of a kernel is a coroutine over barriers that count as the hardware's do (arrivals and bytes of a phase, waits by
parity), copies land and products end some time after they were issued, and a wait gives up after LIMIT steps. Copies that are
later than that, or a grid in front that ends late, make waits run out; whatever the schedule,
  - no barrier is arrived at more often than its phase counts,
  - no copy lands, and no product ends, behind the kernel's end,
  - sums are stored over the ring only where no copy is on its way or still to be issued.
The rules that hold are those of the source. Of those that it had before (who gave up went on giving back stages and
accumulators; only a copying warp that had itself given up waited for its copies) the model finds what goes wrong.
"""
import random

import pytest

LIMIT = 400


class Wrong(AssertionError):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.phase, self.pending, self.bytes = count, 0, count, 0

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, expect=0):
        if self.pending == 0:
            raise Wrong("a phase is arrived at too often")
        self.pending -= 1
        self.bytes += expect
        self._turn()

    def landed(self, n):
        self.bytes -= n
        self._turn()

    def over(self, parity):
        return (self.phase & 1) != parity


class Cluster:
    """`pair`: two CTAs with one ring each, whose halves of the columns have an issuer each; else one CTA, two issuers in turn."""

    def __init__(self, rng, pair, blocks, depth, accumulators, late, old):
        self.rng, self.pair, self.blocks, self.depth, self.nacc, self.late, self.old = rng, pair, blocks, depth, accumulators, late, old
        self.now, self.events, self.flying, self.running, self.ended = 0, [], 0, 0, False
        self.ctas, issuers = (2, 2) if pair else (1, 2)
        self.full = [Barrier(1) for _ in range(depth)]
        self.empty = [[Barrier(2 if pair else 1) for _ in range(depth)] for _ in range(self.ctas)]
        halves = 2 if pair else 1
        self.sfull = [[[Barrier(1) for _ in range(accumulators)] for _ in range(halves)] for _ in range(self.ctas)]
        self.sempty = [[Barrier(self.ctas) for _ in range(accumulators)] for _ in range(halves)]
        self.done = [Barrier(1) for _ in range(issuers)]
        self.wanted = blocks * self.ctas  # copies still to be issued
        self.front = rng.choice((0, 5, rng.randint(LIMIT // 2, 3 * LIMIT)) if late else (0, 5))  # the grid in front ends
        self.roles = [self.copies(c) for c in range(self.ctas)] + [self.products(i) for i in range(issuers)]
        self.roles += [self.adders(c, h) for c in range(self.ctas) for h in range(halves)]

    def after(self, delay, fn):
        self.events.append((self.now + delay, fn))

    def wait(self, bar, parity, ok):
        """Yields until the phase is over; whether it was, or had been given up before."""
        if not ok:
            return False
        for _ in range(LIMIT):
            if bar.over(parity):
                return True
            yield
        return False

    def copies(self, cta):
        # The delays of copies that are late all the same land within a limit's time of their issue; a wait that began before
        # the issue runs out.
        def issue(j):
            if cta == 0:
                self.full[j % self.depth].arrive(expect=self.ctas)
            self.flying += 1
            self.wanted -= 1
            delay = self.rng.randint(LIMIT // 2, LIMIT - 10) if self.late and self.rng.random() < 0.2 else self.rng.randint(3, 12)

            def land():
                if self.ended:
                    raise Wrong("a copy lands behind the end")
                self.flying -= 1
                self.full[j % self.depth].landed(1)
            self.after(delay, land)

        ok, it = True, min(self.depth, self.blocks)
        while self.now < self.front:
            yield
        for j in range(it):
            issue(j)
        while it < self.blocks and ok:
            ok = yield from self.wait(self.empty[cta][it % self.depth], (it // self.depth - 1) & 1, ok)
            if not ok:
                break
            issue(it)
            it += 1
            yield
        if self.old and (ok or cta):
            return
        bars, good = (self.full, True) if cta == 0 else (self.empty[cta], True)
        for j in range(max(0, it - self.depth), it):
            good = yield from self.wait(bars[j % self.depth], (j // self.depth) & 1, True if self.old else good)

    def products(self, i):
        ok, step = True, 1 if self.pair else 2
        half = i if self.pair else 0
        for it in range(0 if self.pair else i, self.blocks, step):
            s, b = it % self.depth, it % self.nacc
            free, ring = (self.sempty[half][b], (it // self.nacc - 1) & 1), (self.full[s], (it // self.depth) & 1)
            for bar, parity in ((ring, free) if self.pair else (free, ring)):
                if bar is free[0] and it < self.nacc:
                    continue
                ok = yield from self.wait(bar, parity, ok)
            if not ok and not self.old:
                break
            if ok:
                self.running += 1
                self.after(6, self.product_ends)

            def commit(s=s, b=b):
                for c in range(self.ctas):
                    self.sfull[c][half][b].arrive()
                    self.empty[c][s].arrive()
            self.after(7, commit)
            yield
        if not self.old:
            self.after(7, self.done[i].arrive)
            yield from self.wait(self.done[i], 0, True)

    def product_ends(self):
        if self.ended:
            raise Wrong("a product ends behind the end")
        self.running -= 1

    def adders(self, cta, half):
        ok = True
        for it in range(self.blocks):
            b = it % self.nacc
            ok = yield from self.wait(self.sfull[cta][half][b], (it // self.nacc) & 1, ok)
            for _ in range(self.rng.randint(1, 4)):
                yield
            if ok or self.old:
                self.sempty[half][b].arrive()
        if ok or self.old:
            if self.flying or self.wanted:
                raise Wrong("sums are stored where copies land")

    def run(self):
        live = list(self.roles)
        while live:
            self.now += 1
            due = [e for e in self.events if e[0] <= self.now]
            self.events = [e for e in self.events if e[0] > self.now]
            for _, fn in due:
                fn()
            for r in self.rng.sample(live, len(live)):
                try:
                    next(r)
                except StopIteration:
                    live.remove(r)
        self.ended = True
        late = self.flying or self.running
        while self.events:
            _, fn = self.events.pop(0)
            fn()
        return late


def runs(pair, late, old, n):
    for seed in range(n):
        rng = random.Random(seed)
        depth = rng.choice((6,) if pair else (4, 5, 6, 8, 10))
        yield Cluster(rng, pair, rng.randint(1, 40), depth, 2 if pair else rng.choice((2, 4)), late, old)


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_whoever_gives_up_the_kernel_ends_in_order(pair, late):
    for c in runs(pair, late, False, 300):
        assert not c.run()
        if not late:  # and nobody did
            assert all(b.phase for b in c.full[:min(c.blocks, c.depth)]) and not c.wanted


@pytest.mark.parametrize("pair", [False, True])
def test_the_rules_before_did_not(pair):
    found = set()
    for c in runs(pair, True, True, 300):
        try:
            if c.run():
                found.add("late")
        except Wrong as e:
            found.add(str(e))
    assert "sums are stored where copies land" in found
    assert found & {"a copy lands behind the end", "a phase is arrived at too often"}
