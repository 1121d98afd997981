"""A random-schedule model of the positional attention kernel's synchronisation
(``qsa_causal.cu``): its barriers with their parities, the ring of K/V units, the
two S / P buffers, the two issuing threads, the softmax halves and the copy
engine, each taking steps in any order.  A wait by parity that returns before
its own use of the barrier has completed (the parity of two uses earlier looks the
same), a unit read before it landed or refilled before it was read, a
product over scores not yet consumed, a sum rescaled under a running product, and
a schedule in which nothing can move are errors.  Variants with one wait moved or
left out have to be caught: the model would see the mistake in the kernel too.
"""

import random

import pytest

UNITS = 5


class Bad(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.left, self.tx, self.phase = count, count, 0, 0

    def _turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase += 1
            self.left = self.count

    def arrive(self, tx=0):
        if self.left == 0:
            raise Bad("an arrival too many")
        self.left -= 1
        self.tx += tx
        self._turn()

    def land(self):
        self.tx -= 1
        if self.tx < 0:
            raise Bad("bytes that nobody expected")
        self._turn()

    def over(self, use):
        """What a test of use's parity says; it must not be two uses off."""
        says = (self.phase & 1) != (use & 1)
        if says and self.phase <= use:
            raise Bad("a wait that took another use of its barrier for its own")
        if self.phase > use + 1:
            raise Bad("a wait that came a use late")
        return says


class Model:
    """``pieces``: key tiles of each item part that the CTA walks."""

    def __init__(self, pieces, rng, variant=""):
        self.pieces, self.rng, self.variant = pieces, rng, variant
        self.full = [Bar(1) for _ in range(UNITS)]
        self.empty = [Bar(1) for _ in range(UNITS)]
        self.q_full, self.q_empty = Bar(1), Bar(1)
        self.s, self.p, self.pv = ([Bar(c) for _ in range(2)] for c in (1, 2, 1))
        self.slot = [None] * UNITS           # what has landed in a unit and is still wanted
        self.flying = []                     # copies on their way: (slot, what)
        self.pipe = {"S": [], "O": []}       # per issuing thread, in order
        self.q = None                        # the piece whose Q rows are in place
        self.scores = [None, None]           # tile whose S is in the buffer
        self.probs = [0, 0]                  # halves of P written
        self.clean = set()                   # V units put right in edge tiles
        self.sums = None                     # (piece, tiles added)
        tiles, t = [], 0
        for k, n in enumerate(pieces):
            tiles.append(list(range(t, t + n)))
            t += n
        self.tiles = tiles
        self.edge = {t: rng.random() < 0.5 for ts in tiles for t in ts}
        self.jump = {t: rng.random() < 0.4 for ts in tiles for t in ts}
        self.read = set()                    # halves that have read an item's sums
        self.meet = [0, 0]                   # rendezvous of the two halves

    # ---- the order of units in the ring, as the producer walks it
    def order(self):
        for ts in self.tiles:
            for y, t in enumerate(ts):
                yield from (("K", t, 0), ("K", t, 1))
                if y > 0:
                    yield from (("V", ts[y - 1], 0), ("V", ts[y - 1], 1))
            yield from (("V", ts[-1], 0), ("V", ts[-1], 1))

    def producer(self):
        for i, what in enumerate(self.order()):
            slot, use = i % UNITS, i // UNITS
            while use > 0 and not self.empty[slot].over(use - 1):
                yield
            if self.slot[slot] is not None:
                raise Bad("a unit refilled before it was read")
            self.full[slot].arrive(tx=2)
            self.flying += [(slot, what), (slot, what)]  # two boxes, landing in any order
            yield

    def copies(self):
        seen = {}
        while True:
            if self.flying:
                slot, what = self.flying.pop(self.rng.randrange(len(self.flying)))
                seen[what] = seen.get(what, 0) + 1
                if seen[what] == 2:
                    self.slot[slot] = what
                self.full[slot].land()
            yield

    def tensor_core(self):
        while True:
            ready = [n for n, q in self.pipe.items() if q]
            if ready:
                self.pipe[self.rng.choice(ready)].pop(0)()
            yield

    def loader(self):
        for k in range(len(self.pieces)):
            while k > 0 and not self.q_empty.over(k - 1):
                yield
            self.q = None
            yield
            self.q = k
            self.q_full.arrive()
            yield

    # ---- issuing threads
    def index(self):
        if not hasattr(self, "_at"):
            self._at = {w: i for i, w in enumerate(self.order())}
        return self._at

    def unit(self, what):
        i = self.index()[what]
        return i % UNITS, i // UNITS

    def scores_of(self, t, k, u):
        def run():
            slot, _ = self.unit(("K", t, u))
            if self.slot[slot] != ("K", t, u):
                raise Bad("a product over a unit of K that is not there")
            if self.q != k:
                raise Bad("a product over another item's Q")
            if u == 0 and self.scores[t & 1] is not None:
                raise Bad("scores written over P that has not been read")
            if u == 1:
                self.scores[t & 1], self.probs[t & 1] = t, 0
        return run

    def free(self, what):
        def run():
            slot, _ = self.unit(what)
            self.slot[slot] = None
            self.empty[slot].arrive()
        return run

    def issue_s(self):
        for k, ts in enumerate(self.tiles):
            while not self.q_full.over(k):
                yield
            for y, t in enumerate(ts):
                first = y >= 2 if self.variant != "K always first" else True
                units = [self.unit(("K", t, u)) for u in range(2)]
                if first:
                    for slot, use in units:
                        while not self.full[slot].over(use):
                            yield
                while t >= 2 and self.variant != "S over P" and not self.pv[t & 1].over((t - 2) >> 1):
                    yield
                if not first:
                    for slot, use in units:
                        while not self.full[slot].over(use):
                            yield
                for u in range(2):
                    self.pipe["S"] += [self.scores_of(t, k, u), self.free(("K", t, u))]
                    yield
                self.pipe["S"].append(self.s[t & 1].arrive)
                yield
            self.pipe["S"].append(self.q_empty.arrive)
            yield

    def sums_of(self, t, k, y, u):
        def run():
            slot, _ = self.unit(("V", t, u))
            if self.slot[slot] != ("V", t, u):
                raise Bad("a product over a unit of V that is not there")
            if self.edge[t] and {(t, u, h) for h in range(2)} - self.clean:
                raise Bad("a product over V that has not been put right")
            if self.scores[t & 1] != t or self.probs[t & 1] != 2:
                raise Bad("a product over P that is not there")
            if y == 0 and u == 0 and self.sums not in (None, "read"):
                raise Bad("sums started over before they were read")
            if u == 1:
                self.sums = (k, t)
                self.scores[t & 1] = None
            else:
                self.sums = (k, t, "running")
        return run

    def issue_o(self):
        for k, ts in enumerate(self.tiles):
            for y, t in enumerate(ts):
                units = [self.unit(("V", t, u)) for u in range(2)]
                while self.variant != "V before S" and not self.s[t & 1].over(t >> 1):
                    yield
                for slot, use in units:
                    while not self.full[slot].over(use):
                        yield
                while not self.p[t & 1].over(t >> 1):
                    yield
                for u in range(2):
                    self.pipe["O"] += [self.sums_of(t, k, y, u), self.free(("V", t, u))]
                    yield
                self.pipe["O"].append(self.pv[t & 1].arrive)
                yield

    # ---- softmax
    def both(self, half):
        self.meet[half] += 1
        while self.meet[half ^ 1] < self.meet[half]:
            yield

    def softmax(self, half):
        for k, ts in enumerate(self.tiles):
            for y, t in enumerate(ts):
                while not self.s[t & 1].over(t >> 1):
                    yield
                if self.scores[t & 1] != t:
                    raise Bad("scores read that are not there")
                yield from self.both(half)
                if self.jump[t] and y > 0:
                    while self.variant != "rescale at once" and not self.pv[(t - 1) & 1].over((t - 1) >> 1):
                        yield
                    for _ in range(2):
                        if self.sums != (k, t - 1):
                            raise Bad("sums rescaled under a product")
                        yield
                self.probs[t & 1] += 1
                yield
                if self.edge[t]:
                    if y > 0 and self.variant != "V by parity alone":
                        while not self.pv[(t - 1) & 1].over((t - 1) >> 1):
                            yield
                    for u in range(2):  # (the model's half puts both units right; a kernel thread has one of them)
                        slot, use = self.unit(("V", t, u))
                        while not self.full[slot].over(use):
                            yield
                        if self.slot[slot] != ("V", t, u):
                            raise Bad("V put right before it landed")
                        self.clean.add((t, u, half))
                        yield
                self.p[t & 1].arrive()
                yield
            yield from self.both(half)
            last = ts[-1]
            while self.variant != "sums read early" and not self.pv[last & 1].over(last >> 1):
                yield
            for _ in range(2):
                if self.sums not in ((k, last), "read"):
                    raise Bad("sums read that are not there")
                yield
            self.read.add((k, half))  # (the next item's sums start over P, which both halves write after this)
            if self.read >= {(k, 0), (k, 1)}:
                self.sums = "read"

    def run(self):
        agents = {"producer": self.producer(), "loader": self.loader(), "S": self.issue_s(), "O": self.issue_o(),
                  "half0": self.softmax(0), "half1": self.softmax(1)}
        engines = [self.copies(), self.tensor_core()]
        weight = {n: self.rng.choice([1, 1, 3, 10]) for n in [*agents, "copies", "tensor"]}
        idle = 0
        while agents:
            names = [*agents, "copies", "tensor"]
            n = self.rng.choices(names, [weight[x] for x in names])[0]
            before = self.state()
            if n == "copies":
                next(engines[0])
            elif n == "tensor":
                next(engines[1])
            else:
                try:
                    next(agents[n])
                    if agents[n].gi_frame is not None and before == self.state():
                        idle += 1
                        if idle > 5000:
                            raise Bad("nothing moves")
                        continue
                except StopIteration:
                    del agents[n]
            idle = 0 if before != self.state() else idle + 1
            if idle > 5000:
                raise Bad("nothing moves")
        if any(self.slot) or self.flying or any(self.pipe.values()):
            # what is still in the pipe at the end is the last commits
            for q in self.pipe.values():
                for f in q:
                    f()
        if any(self.slot) or self.flying:
            raise Bad("units left over")

    def state(self):
        bars = [*self.full, *self.empty, self.q_full, self.q_empty, *self.s, *self.p, *self.pv]
        return ([(b.phase, b.left, b.tx) for b in bars], len(self.flying), [len(q) for q in self.pipe.values()],
                list(self.meet), self.q, list(self.probs), len(self.clean), self.sums)


def _walks(rng):
    return [rng.choice([1, 1, 2, 2, 3, 4, 7]) for _ in range(rng.randint(1, 5))]


@pytest.mark.parametrize("seed", range(60))
def test_any_schedule_is_right(seed):
    rng = random.Random(seed)
    Model(_walks(rng), rng).run()


@pytest.mark.parametrize("variant", ["K always first", "S over P", "V before S", "rescale at once",
                                     "V by parity alone", "sums read early"])
def test_a_wait_moved_or_left_out_is_caught(variant):
    for seed in range(400):
        rng = random.Random(1000 + seed)
        try:
            Model(_walks(rng), rng, variant).run()
        except Bad:
            return
    raise AssertionError(f"no schedule showed the mistake: {variant}")
