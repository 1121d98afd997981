"""A second random-schedule model of the positional attention kernel
(``qsa_causal.cu``), role by role: the eight softmax warps apart (those of a short
tile without a row of their own skip the exchange and the sums, and each waits for
the unit of V that its rows lie in), the hardware barriers they meet at, the flags of
values taken out, the loader's wait for a whole item, and the way out when any role
gives up a wait.  Like the other model it restates the kernel; the last test holds
the restatement to the source, wait by wait and arrival by arrival.
"""

import os
import random
import re

import pytest
from test_causal_protocol import UNITS, Bad, Bar

from token_indexed_sparse_b200 import build

WARPS = [(half, wq) for half in range(2) for wq in range(4)]
BUDGET = 6  # tiles that may go by while one wait polls without starting over


class Meet:
    """A hardware barrier of n warps."""

    def __init__(self, n):
        self.n, self.here, self.turn = n, 0, 0

    def __call__(self):
        mine = self.turn
        self.here += 1
        if self.here == self.n:
            self.here, self.turn = 0, self.turn + 1
        while self.turn == mine:
            yield


class Model:
    """``pieces``: (key tiles, row groups of 32 with a row) of each item part that the CTA walks;
    ``quits``: the role that gives up one of its waits."""

    def __init__(self, pieces, rng, variant="", quits=None):
        self.rng, self.variant, self.quits = rng, variant, quits
        self.tiles, self.live, t = [], [], 0
        for n, live in pieces:
            self.tiles.append(list(range(t, t + n)))
            self.live.append(live)
            t += n
        self.n_tiles = t
        self.quit_at = rng.randint(1, 3 * t) if quits else 0
        self.abort = False
        self.full = [Bar(1) for _ in range(UNITS)]
        self.empty = [Bar(1) for _ in range(UNITS)]
        self.q_full, self.q_empty = Bar(1), Bar(1)
        self.s, self.p, self.pv = ([Bar(c) for _ in range(2)] for c in (1, 8, 1))
        self.drain = {"S": Bar(1), "O": Bar(1)}
        self.pair = [Meet(2) for _ in range(4)]
        self.all8 = Meet(8)
        self.slot, self.flying, self.copied = [None] * UNITS, [], {}
        self.pipe = {"S": [], "O": []}
        self.q, self.scores, self.probs = None, [None, None], [set(), set()]
        self.clean, self.sums, self.read = set(), None, set()
        self.poison, self.truth = [False] * 3, [False] * len(pieces)
        self.tile = 0                          # tiles whose scores have been issued
        self.edge = [rng.random() < 0.5 for _ in range(t)]
        self.jump = {(t, wq): rng.random() < 0.3 for t in range(t) for wq in range(4)}
        self.at = {w: i for i, w in enumerate(self.order())}

    def bad(self, what):
        if not self.abort:  # (behind a wait that gave up the outputs are marked wrong)
            raise Bad(what)

    def wait(self, role, bar, use):
        """True once the wait is over, False when it gives up; polls at least once."""
        while True:
            if self.abort:
                return (bar.phase & 1) != (use & 1)
            if bar.over(use):
                return True
            if role == self.quits:
                self.quit_at -= 1
                if self.quit_at <= 0:
                    self.abort = True
                    return False
            yield

    def wait_item(self, bar, use):
        seen = self.tile
        while True:
            if self.abort:
                return (bar.phase & 1) != (use & 1)
            if bar.over(use):
                return True
            if self.quits == "loader":
                self.quit_at -= 1
                if self.quit_at <= 0:
                    self.abort = True
                    return False
            if self.tile - seen >= BUDGET:     # the polls of one budget
                if self.variant == "one budget for an item":
                    raise Bad("a legal item took longer than a wait's polls")
                seen = self.tile
            yield

    def order(self):
        for ts in self.tiles:
            for y, t in enumerate(ts):
                yield from (("K", t, 0), ("K", t, 1))
                if y > 0:
                    yield from (("V", ts[y - 1], 0), ("V", ts[y - 1], 1))
            yield from (("V", ts[-1], 0), ("V", ts[-1], 1))

    def unit(self, what):
        i = self.at[what]
        return i % UNITS, i // UNITS

    # ---- copies
    def producer(self):
        issued, ok = 0, True
        for i, what in enumerate(self.order()):
            slot, use = i % UNITS, i // UNITS
            if use > 0:
                ok = yield from self.wait("producer", self.empty[slot], use - 1)
            if not ok:
                break
            if self.slot[slot] is not None:
                self.bad("a unit refilled before it was read")
            self.full[slot].arrive(tx=2)
            self.flying += [(slot, what), (slot, what)]
            issued += 1
            yield
        if self.variant == "copies left in flight" or (ok and self.variant == "only a producer that gave up drains"):
            return
        for j in range(min(issued, UNITS)):
            slot, use = (issued - 1 - j) % UNITS, (issued - 1 - j) // UNITS
            while self.full[slot].phase <= use:
                yield

    def copies(self):
        while True:
            if self.flying:
                slot, what = self.flying.pop(self.rng.randrange(len(self.flying)))
                self.copied[what] = self.copied.get(what, 0) + 1
                if self.copied[what] == 2:
                    self.slot[slot] = what
                self.full[slot].land()
            yield

    def tensor_core(self):
        while True:
            ready = [n for n, q in self.pipe.items() if q]
            if ready:
                self.pipe[self.rng.choice(ready)].pop(0)[1]()
            yield

    def loader(self):
        for k in range(len(self.tiles)):
            if k > 0 and not (yield from self.wait_item(self.q_empty, k - 1)):
                break
            self.q = None
            yield
            self.q = k
            self.q_full.arrive()
            yield

    # ---- issuing threads
    def scores_of(self, t, k, u):
        def run():
            slot, _ = self.unit(("K", t, u))
            if self.slot[slot] != ("K", t, u):
                self.bad("a product over a unit of K that is not there")
            if self.q != k:
                self.bad("a product over another item's Q")
            if u == 0 and self.scores[t & 1] is not None:
                self.bad("scores written over P that has not been read")
            if u == 1:
                self.scores[t & 1], self.probs[t & 1] = t, set()
        return "product", run

    def free(self, what):
        def run():
            slot, _ = self.unit(what)
            self.slot[slot] = None
            self.empty[slot].arrive()
        return "arrival", run

    def finish(self, name):
        """The issuing thread's products end before tensor memory is freed."""
        self.pipe[name].append(("arrival", self.drain[name].arrive))
        while not self.drain[name].phase:
            yield

    def issue_s(self):
        ok = True
        for k, ts in enumerate(self.tiles):
            ok = yield from self.wait("S", self.q_full, k)
            for y, t in enumerate(ts):
                if not ok:
                    break
                waits = [(self.full[s], u) for s, u in (self.unit(("K", t, h)) for h in range(2))]
                before = [(self.pv[t & 1], (t - 2) >> 1)] if t >= 2 else []
                for bar, use in (waits + before if y >= 2 else before + waits):
                    ok = ok and (yield from self.wait("S", bar, use))
                if not ok:
                    break
                self.tile = t + 1
                for u in range(2):
                    self.pipe["S"] += [self.scores_of(t, k, u), self.free(("K", t, u))]
                    yield
                self.pipe["S"].append(("arrival", self.s[t & 1].arrive))
                yield
            if not ok:
                break
            self.pipe["S"].append(("arrival", self.q_empty.arrive))
            yield
        if not ok or self.variant != "only who gave up drains":
            yield from self.finish("S")

    def sums_of(self, t, k, y, u):
        def run():
            slot, _ = self.unit(("V", t, u))
            if self.slot[slot] != ("V", t, u):
                self.bad("a product over a unit of V that is not there")
            if self.edge[t] and {(t, u, h, wq) for h in range(2) for wq in (2 * u, 2 * u + 1)} - self.clean:
                self.bad("a product over V that has not been put right")
            want = {(h, wq) for h, wq in WARPS if wq < self.live[k]}
            if self.scores[t & 1] != t or self.probs[t & 1] != want:
                self.bad("a product over P that is not there")
            if y == 0 and u == 0 and k > 0 and self.sums != "read":
                self.bad("sums started over before they were read")
            self.sums = (k, t) if u == 1 else (k, t, "running")
            if u == 1:
                self.scores[t & 1] = None
        return "product", run

    def issue_o(self):
        ok = True
        for k, ts in enumerate(self.tiles):
            for y, t in enumerate(ts):
                waits = [(self.s[t & 1], t >> 1)]
                waits += [(self.full[s], u) for s, u in (self.unit(("V", t, h)) for h in range(2))]
                waits += [(self.p[t & 1], t >> 1)]
                for bar, use in waits:
                    ok = ok and (yield from self.wait("O", bar, use))
                if not ok:
                    break
                for u in range(2):
                    self.pipe["O"] += [self.sums_of(t, k, y, u), self.free(("V", t, u))]
                    yield
                self.pipe["O"].append(("arrival", self.pv[t & 1].arrive))
                yield
            if not ok:
                break
        if not ok or self.variant != "only who gave up drains":
            yield from self.finish("O")

    # ---- softmax
    def softmax(self, half, wq):
        gone = [False]

        def wait(bar, use):
            if not gone[0]:
                gone[0] = not (yield from self.wait("softmax", bar, use))

        for k, ts in enumerate(self.tiles):
            live = wq < self.live[k]
            for y, t in enumerate(ts):
                last = self.pv[(t - 1) & 1], (t - 1) >> 1
                yield from wait(self.s[t & 1], t >> 1)
                if live:
                    if self.scores[t & 1] != t:
                        self.bad("scores read that are not there")
                    yield from self.pair[wq]()
                    if y > 0 and self.jump[t, wq]:
                        yield from wait(*last)
                        for _ in range(2):
                            if self.sums != (k, t - 1):
                                self.bad("sums rescaled under a product")
                            yield
                    self.probs[t & 1].add((half, wq))
                    yield
                if self.edge[t]:
                    if y > 0 and self.variant != "V by parity alone":
                        yield from wait(*last)
                    unit = ("V", t, wq >> 1 if self.variant != "the other unit" else 1 - (wq >> 1))
                    slot, use = self.unit(unit)
                    yield from wait(self.full[slot], use)
                    if self.slot[self.unit(("V", t, wq >> 1))[0]] != ("V", t, wq >> 1):
                        self.bad("V put right before it landed")
                    self.clean.add((t, wq >> 1, half, wq))
                    if self.rng.random() < 0.2:
                        self.poison[k % 3] = self.truth[k] = True
                    yield
                self.p[t & 1].arrive()
                yield
            if (half, wq) == (0, 0):
                self.poison[(k + 1) % 3] = False
                yield
            if self.variant != "no meeting at an item's end":
                yield from self.all8()
            if self.poison[k % 3] != self.truth[k]:
                self.bad("another item's flag")
            yield from self.pair[wq]()
            yield from wait(self.pv[ts[-1] & 1], ts[-1] >> 1)
            if live:
                for _ in range(2):
                    if self.sums not in ((k, ts[-1]), "read"):
                        self.bad("sums read that are not there")
                    yield
                self.read.add((k, half, wq))
                if len([r for r in self.read if r[0] == k]) == 2 * self.live[k]:
                    self.sums = "read"

    def run(self):
        roles = {"producer": self.producer(), "loader": self.loader(), "S": self.issue_s(), "O": self.issue_o()}
        roles |= {f"warp{h}{w}": self.softmax(h, w) for h, w in WARPS}
        engines = {"copies": self.copies(), "tensor": self.tensor_core()}
        weight = {n: self.rng.choice([1, 1, 3, 10]) for n in roles}
        weight |= {n: self.rng.choice([0.1, 1, 3, 10]) for n in engines}
        for _ in range(4000 + 20000 * self.n_tiles):
            if not roles:
                break
            names = [*roles, *engines]
            n = self.rng.choices(names, [weight[x] for x in names])[0]
            try:
                next(engines[n] if n in engines else roles[n])
            except StopIteration:
                del roles[n]
        if roles:
            raise Bad(f"never ends: {sorted(roles)}")
        # the block ends here: nothing may still write its shared or tensor memory
        if self.flying:
            raise Bad("copies in flight at the end")
        if any(kind == "product" for q in self.pipe.values() for kind, _ in q):
            raise Bad("products in flight at the end")
        for q in self.pipe.values():
            for _, f in q:
                f()
        if not self.abort and any(self.slot):
            raise Bad("units left over")
        return self


def _pieces(rng):
    return [(rng.choice([1, 1, 2, 2, 3, 4, 7]), rng.choice([1, 1, 2, 4, 4])) for _ in range(rng.randint(1, 5))]


@pytest.mark.parametrize("seed", range(60))
def test_any_schedule_is_right(seed):
    rng = random.Random(seed)
    assert not Model(_pieces(rng), rng).run().abort


def test_a_long_item_is_not_given_up():
    for seed in range(10):
        rng = random.Random(seed)
        assert not Model([(60, 4), (2, 1), (30, 2)], rng).run().abort


def _way_out(seed, variant="", quits=None):
    """A walk, often a short one whose roles are near their ends, in which one role gives up a wait."""
    rng = random.Random(5000 + seed)
    pieces = _pieces(rng) if rng.random() < 0.3 else [(rng.choice([1, 1, 2]), rng.choice([1, 4]))] * rng.randint(1, 2)
    return Model(pieces, rng, variant, quits=quits or rng.choice(["producer", "loader", "S", "O", "softmax"])).run()


@pytest.mark.parametrize("quits", ["producer", "loader", "S", "O", "softmax"])
def test_every_role_ends_when_one_gives_up(quits):
    given_up = [_way_out(seed, quits=quits).abort for seed in range(150)]
    assert sum(given_up) > 50


@pytest.mark.parametrize("variant", ["one budget for an item", "V by parity alone", "the other unit",
                                     "no meeting at an item's end"])
def test_a_wait_changed_is_caught(variant):
    for seed in range(400):
        rng = random.Random(1000 + seed)
        try:
            Model(_pieces(rng) + [(12, 4), (1, 1)], rng, variant).run()
        except Bad:
            return
    raise AssertionError(f"no schedule showed the mistake: {variant}")


@pytest.mark.parametrize("variant", ["copies left in flight", "only a producer that gave up drains",
                                     "only who gave up drains"])
def test_a_way_out_that_leaves_work_behind_is_caught(variant):
    for seed in range(400):
        try:
            _way_out(seed, variant)
        except Bad:
            return
    raise AssertionError(f"no schedule showed the mistake: {variant}")


# What the kernel waits for and signals, in the order of its source, role by role.  A change here is a
# change of the protocol: both models have to follow it.
SITES = {
    "K / V units": [("warp_wait", "kBEmpty"), ("mbar_arrive_tx", "kBFull"), ("tma", "kBFull"), ("tma", "kBFull"),
                    ("mbar_wait", "kBFull")],
    "tensor core": [("wait", "kBQFull"), ("wait", "kBFull"), ("wait", "kBFull"), ("wait", "kBPv"),
                    ("commit", "kBEmpty"), ("commit", "kBS"), ("commit", "kBQEmpty"),
                    ("wait", "kBS"), ("wait", "kBFull"), ("wait", "kBFull"), ("wait", "kBP"),
                    ("commit", "kBEmpty"), ("commit", "kBPv"), ("commit", "kBDrain"), ("mbar_wait", "kBDrain")],
    "Q rows": [("warp_wait_item", "kBQEmpty"), ("mbar_arrive", "kBQFull")],
    "softmax": [("wait", "kBS"), ("wait", "kBPv"), ("wait", "kBPv"), ("wait", "kBFull"), ("mbar_arrive", "kBP"),
                ("wait", "kBPv")],
}


def test_the_models_restate_the_source():
    text = open(os.path.join(build.CSRC, "qsa_causal.cu")).read()
    kernel = text[text.index("\ncausal_kernel("):text.index("causal_join_kernel(")]
    parts = re.split(r"// -{20,} (K / V units|tensor core|Q rows|softmax)\n", kernel)
    assert parts[1::2] == list(SITES)
    for role, body in zip(parts[1::2], parts[2::2]):
        body = re.sub(r"//[^\n]*", "", body)
        # the drain's barrier is named in a variable first
        body = re.sub(r"const int i = kBDrain[^;]*;", "", body).replace("bar(i))", "bar(kBDrain))").replace(
            "bar(i), 0", "bar(kBDrain), 0")
        found = []
        for m in re.finditer(r"\bkB[A-Z]\w*", body):
            head = body[:m.start()]
            call = [c for c in re.findall(r"\b(wait|warp_wait|warp_wait_item|mbar_wait|mbar_arrive|mbar_arrive_tx|"
                                          r"commit|tma_load)\(", head)][-1]
            found.append(("tma" if call == "tma_load" else call, m.group()))
        assert found == SITES[role], role
    order = [kernel.index(x) for x in ("*tile = static_cast<int>(tau + 1)", "commit(bar(kBS")]
    assert order == sorted(order)
