"""The mbarriers of the two paged attention kernels as a model on the CPU: their roles'
waits and arrivals in random orders with long stalls anywhere.  A wait sees one bit of a
barrier (the parity of the phase under way), so it has to be made when that bit can mean
nothing else: not before the phase ahead of its own is complete (it would pass at once),
nor after the one behind it may be (it would never pass)."""
import random

import pytest

PIECES = [3, 1, 7, 2, 11, 5]  # tiles of a CTA's pieces
# rows a piece: places for tiles, issuers of the scores and of PV
FOUR = {16: dict(ns=5, qk=2, pv=1), 64: dict(ns=4, qk=1, pv=1)}
EIGHT = {16: dict(ns=6, qk=2, pv=1), 64: dict(ns=5, qk=1, pv=2)}
NP, NR = 2, 3                 # 4 bits: places for strips and for the tiles' rope


class Fault(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.here, self.done = count, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.count:
            self.here, self.done = 0, self.done + 1


class Model:
    """Agents are generators that yield what they wait for: a (barrier, phase), or a
    (named barrier's Bar, None) that they have arrived at."""

    def __init__(self, four, rows, rng, planted=()):
        k = (FOUR if four else EIGHT)[rows]
        self.four, self.rows, self.rng, self.planted = four, rows, rng, planted
        self.ns, self.qk, self.pv = k["ns"], k["qk"], k["pv"]
        split = four and rows == 16
        self.split, self.n_live = split, (2 if split else 4)
        bars = lambda n, c: [Bar(c) for _ in range(n)]
        self.full, self.empty = bars(self.ns, 4 if four else 1), bars(self.ns, self.pv)
        self.pack_full, self.pack_empty, self.rope_free = bars(NP, 1), bars(NP, 4), bars(NR, 1)
        self.s_full, self.s_free = bars(2, 1), bars(2, self.n_live)
        self.p_full, self.p_free = bars(2, self.n_live), bars(2, self.pv)
        self.ref, self.q_full, self.o_free = bars(4, 1), bars(2, 4), bars(2, 8)
        self.q_free, self.o_full = Bar(self.qk), Bar(self.pv)
        self.named = bars(2, 4) + [Bar(8)]
        self.moves = [rng.random() < 0.5 for _ in range(sum(PIECES))]
        self.pv_done = [0] * sum(PIECES)
        self.queues = []       # an issuer's MMAs and commits, in order; a copy by itself

    def pieces(self):
        j = 0
        for p, n in enumerate(PIECES):
            yield p, range(j, j + n)
            j += n

    # ---- asynchronous work
    def queue(self):
        self.queues.append([])
        return self.queues[-1]

    # ---- roles
    def load(self):
        for p, tiles in self.pieces():
            for j in tiles:
                if self.four:
                    yield self.pack_empty[j % NP], j // NP - 1
                    self.queue().append([self.pack_full[j % NP].arrive])
                else:
                    yield self.empty[j % self.ns], j // self.ns - 1
                    self.queue().append([self.full[j % self.ns].arrive])

    def expand(self, group):
        for p, tiles in self.pieces():
            for j in tiles:
                if j % 2 != group:
                    continue
                yield self.pack_full[j % NP], j // NP
                self.pack_empty[j % NP].arrive()
                place, rope = (self.empty[j % self.ns], j // self.ns - 1), \
                    (self.rope_free[j % NR], j // NR - 1)
                if self.qk == 1 or "rope beside place" in self.planted:
                    yield rope  # lanes of one warp wait for either, in any order
                    yield place
                else:
                    yield place
                    yield rope
                self.full[j % self.ns].arrive()

    def scores(self, me, q):
        for p, tiles in self.pieces():
            yield self.q_full[p & 1], p >> 1
            for j in tiles:
                if self.qk == 2 and j % 2 != me:
                    continue
                if j >= 2:
                    yield self.s_free[j & 1], (j >> 1) - 1
                yield self.full[j % self.ns], j // self.ns
                q.append([self.s_full[j & 1].arrive] +
                         ([self.rope_free[j % NR].arrive] if self.four else []))
            q.append([self.q_free.arrive])

    def values(self, q):
        def finish(j):
            self.pv_done[j] += 1
        for p, tiles in self.pieces():
            if p > 0:
                yield self.o_free[(p - 1) & 1], (p - 1) >> 1
            for j in tiles:
                yield self.p_full[j & 1], j >> 1
                ahead = j - (1 if "one place for scales" in self.planted else 2)
                if self.four and ahead >= 0 and self.pv_done[ahead] < self.pv:
                    raise Fault("scales are copied under the PV GEMM that reads them")
                q.append([lambda j=j: finish(j), self.empty[j % self.ns].arrive,
                          self.p_free[j & 1].arrive])
            q.append([self.o_full.arrive])

    def q_in(self):
        for k, _ in self.pieces():
            if k > 1:
                yield self.o_free[k & 1], (k >> 1) - 1
            if k > 0:
                yield self.q_free, k - 1
            self.q_full[k & 1].arrive()

    def sync(self, bar):
        bar.arrive()
        return bar, None

    def rescale(self, wg, j):
        if j >= 2 and "rescale behind one phase" not in self.planted:
            yield self.p_free[wg], (j >> 1) - 1
        yield self.p_free[wg ^ 1], (j - 1) >> 1
        if any(n < self.pv for n in self.pv_done[:j]):
            raise Fault("O^T is rescaled under the PV GEMM")

    def softmax(self, wg, q4):
        four, split = self.four, self.split
        live = q4 >> 1 == wg if split else True
        qi = q4 & 1 if split else q4
        for p, tiles in self.pieces():
            yield self.q_full[p & 1], p >> 1
            for j in tiles:
                if j % 2 != wg:
                    continue
                first, move = j == tiles[0], j > tiles[0] and self.moves[j]
                if live or "scores for all warps" in self.planted:
                    yield self.s_full[wg], j >> 1
                if live:
                    self.s_free[wg].arrive()
                if live and not first:
                    yield self.ref[qi], j - 1
                if not four:
                    self.ref[qi].arrive()
                if four or not first:
                    yield self.sync(self.named[wg])
                if split and (first or move):
                    yield self.sync(self.named[wg])
                if move:
                    yield self.sync(self.named[wg])
                    yield from self.rescale(wg, j)
                    yield self.sync(self.named[wg])
                if live:
                    if four:
                        self.ref[qi].arrive()
                    if j >= 2:
                        yield self.p_free[wg], (j >> 1) - 1
                    self.p_full[wg].arrive()
            for _ in range(2):
                yield self.sync(self.named[2])
            yield self.o_full, p
            self.o_free[p & 1].arrive()
            yield self.sync(self.named[2])

    # ---- a run
    def run(self):
        agents = [self.load()] + [self.scores(m, self.queue()) for m in range(self.qk)]
        agents += [self.values(self.queue()) for _ in range(self.pv)]
        agents += [self.softmax(wg, q4) for wg in range(2) for q4 in range(4)]
        agents += [self.q_in() for _ in range(4)]
        if self.four:
            agents += [self.expand(g) for g in range(2) for _ in range(4)]
        waits = {}

        def step(a):
            bar, phase = next(a)
            waits[a] = (bar, bar.done - (bar.here == 0) if phase is None else phase, phase is None)

        for a in agents:
            step(a)
        left, idle = set(agents), 0
        while left:
            stalled = self.rng.random() < 0.1
            slow = self.rng.sample(agents, self.rng.randint(0, 3)) if stalled else []
            lazy = self.rng.random() < 0.5  # nothing asynchronous lands for a while
            for _ in range(60):
                jobs = [q for q in self.queues if q]
                if jobs and not (lazy and self.rng.random() < 0.97) and self.rng.random() < 0.5:
                    for f in self.rng.choice(jobs).pop(0):
                        f()
                    idle = 0
                    continue
                a = self.rng.choice(agents)
                if a not in left or a in slow:
                    continue
                bar, phase, named = waits[a]
                if bar.done > phase + 1 and not named:
                    raise Fault("a wait's phase is over, and the one behind it too")
                if named and bar.done <= phase:
                    idle += 1
                elif not named and (bar.done & 1) == (phase & 1):
                    idle += 1
                else:
                    if bar.done <= phase:
                        raise Fault("a wait passes on a phase two before its own")
                    idle = 0
                    try:
                        step(a)
                    except StopIteration:
                        left.discard(a)
                if idle > 20000:
                    raise Fault("no agent goes on")


def runs(four, rows, n, planted=()):
    for seed in range(n):
        Model(four, rows, random.Random(seed), planted).run()


@pytest.mark.parametrize("rows", [16, 64])
@pytest.mark.parametrize("four", [True, False])
def test_waits_pass_on_their_own_phase(four, rows):
    runs(four, rows, 300)


@pytest.mark.parametrize("four, rows, planted, word", [
    (True, 16, "rescale behind one phase", "two before|under the PV"),
    (True, 64, "rescale behind one phase", "two before|under the PV"),
    (False, 16, "rescale behind one phase", "two before|under the PV"),
    (False, 64, "rescale behind one phase", "two before|under the PV"),
    (True, 16, "scores for all warps", "over|no agent"),
    (True, 16, "rope beside place", "two before"),
    (True, 16, "one place for scales", "scales are copied"),
    (True, 64, "one place for scales", "scales are copied"),
])
def test_the_model_finds(four, rows, planted, word):
    """Orders that the kernels do not have: a rescale that waits for the last tile alone,
    warps that wait for scores which others free, a place for the rope waited for beside
    the one in the ring, one place for the scales of all tiles."""
    with pytest.raises(Fault, match=word):
        runs(four, rows, 400, (planted,))
