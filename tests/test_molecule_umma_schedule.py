"""Host-side model of the barriers of the tcgen05 attention within molecules
(`mol_fwd_umma_kernel`, csrc/molecule_umma.cu), with waits that give up.

A CTA has a copying thread (stages of keys into three buffers), a thread that
issues products (scores of stage i into buffer i % 2, then the weights' product
into the accumulator) and eight softmax warps, two to a row.  Copies land in any
order; products end in issue order, and a commit arrives on its barrier some time
after the products before it.  The model runs them under random schedules and
checks, while no wait gives up:

* every wait names the phase that carries its stage;
* products read a stage only when it has landed, and no copy lands in one that is
  still read, by products or for its positions;
* scores never replace weights that a product still reads, and the accumulator is
  rescaled only while no product adds to it;

and always, with waits that give up at random places (what they wait for is late,
not lost): the roles all end, and when shared and tensor memory are released no
copy, product or commit is in flight.  No GPU is involved.
"""
import random

import pytest

STAGES, WARPS = 3, 8


class Violation(AssertionError):
    pass


def need(ok, what):
    if not ok:
        raise Violation(what)


class Bar:
    def __init__(self, count=1):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def ready(self, parity):
        return self.done & 1 != parity


class Cta:
    def __init__(self, stages, seed, give_up, late_flag=True, spare_freed=True):
        """late_flag: the flag is read after the barrier that every role reaches; spare_freed: no commit on
        `freed` for a buffer that takes no further stage."""
        self.n, self.rng, self.give_up = stages, random.Random(seed), give_up
        self.late_flag, self.spare_freed = late_flag, spare_freed
        self.full, self.freed = [Bar() for _ in range(STAGES)], [Bar() for _ in range(STAGES)]
        self.qfull, self.drained = Bar(), Bar()
        self.sfull, self.pvdone = [Bar(), Bar()], [Bar(), Bar()]
        self.pready = [Bar(WARPS), Bar(WARPS)]
        self.abort = self.released = False
        self.copies, self.queue = [], []      # in flight: (buffer, stage or "q"); ("s" | "pv", stage) or ("commit", barrier)
        self.held = [None] * STAGES           # stage that a buffer holds
        self.scores = [None, None]            # ("s" | "p", stage)
        self.reading = {}                     # warp -> stage whose positions it reads
        self.rescaling = set()

    # ---- engines
    def engine(self):
        """One asynchronous step; False when nothing is in flight."""
        if not self.copies and not self.queue:
            return False
        if self.copies and (not self.queue or self.rng.random() < 0.5):
            b, i = self.copies.pop(self.rng.randrange(len(self.copies)))
            need(not self.released, "a copy lands in released shared memory")
            if i == "q":
                self.qfull.arrive()
                return True
            if not self.abort:
                need(self.held[b] is None, "a copy lands in a stage that is still read")
            self.held[b] = i
            self.full[b].arrive()
            return True
        kind, x = self.queue.pop(0)
        need(not self.released, f"{kind} in flight when the memory is released")
        if kind == "commit":
            x.arrive()
        elif not self.abort:
            need(self.held[x % STAGES] == x, "a product reads a stage that is not there")
            if kind == "s":
                need(self.scores[x & 1] is None, "scores replace weights that a product reads")
                self.scores[x & 1] = ("s", x)
            else:
                need(self.scores[x & 1] == ("p", x), "a product reads weights that are not there")
                need(not self.rescaling, "a product adds to an accumulator that is rescaled")
                need(x not in self.reading.values(), "a stage is freed while its positions are read")
                self.scores[x & 1] = None
                self.held[x % STAGES] = None
        return True

    # ---- waits: generators that yield while they poll
    def wait(self, bar, phase):
        while not bar.ready(phase & 1):
            if self.abort:
                return False
            if (yield "poll") == "give up":
                self.abort = True
                return False
        if not self.abort:
            need(bar.done == phase + 1, f"phase {phase} of a barrier at {bar.done}")
        return True

    def drain(self, bar, phase):
        while not bar.ready(phase & 1):
            yield "drain"

    def copier(self):
        self.issued = 0
        if self.n:
            self.copies.append((None, "q"))
            for i in range(self.n):
                b = i % STAGES
                if i >= STAGES and not (yield from self.wait(self.freed[b], i // STAGES - 1)):
                    break
                self.copies.append((b, i))
                self.issued = i + 1
        flag = self.abort
        if not self.late_flag:      # the flag as it is when this role ends
            if flag:
                yield from self.land()
            yield "barrier"
            return
        yield "barrier"
        if self.abort:
            yield from self.land()
            yield "barrier"

    def land(self):
        if self.issued:
            yield from self.drain(self.qfull, 0)
        for i in range(max(0, self.issued - STAGES), self.issued):
            yield from self.drain(self.full[i % STAGES], i // STAGES)

    def products(self):
        yield from self.issue()
        flag = self.abort
        if not self.late_flag:
            if flag:
                self.queue.append(("commit", self.drained))
                yield from self.drain(self.drained, 0)
            yield "barrier"
            return
        yield "barrier"
        if self.abort:
            self.queue.append(("commit", self.drained))
            yield from self.drain(self.drained, 0)
            yield "barrier"

    def issue(self):
        if not self.n or not (yield from self.wait(self.qfull, 0)) or not (yield from self.wait(self.full[0], 0)):
            return

        def score(i):
            self.queue.extend([("s", i), ("commit", self.sfull[i & 1])])
        score(0)
        for i in range(self.n):
            if i + 1 < self.n and not (yield from self.wait(self.full[(i + 1) % STAGES], (i + 1) // STAGES)):
                return
            if i > 0 and not (yield from self.wait(self.pvdone[(i - 1) & 1], (i - 1) >> 1)):
                return
            if i + 1 < self.n:
                score(i + 1)
            if not (yield from self.wait(self.pready[i & 1], i >> 1)):
                return
            self.queue.extend([("pv", i), ("commit", self.pvdone[i & 1])])
            if not self.spare_freed or i + STAGES < self.n:
                self.queue.append(("commit", self.freed[i % STAGES]))

    def softmax(self, w):
        ok = True
        for i in range(self.n):
            ok = (yield from self.wait(self.sfull[i & 1], i >> 1)) and ok
            ok = (yield from self.wait(self.full[i % STAGES], i // STAGES)) and ok
            self.reading[w] = i
            if not self.abort:
                need(self.held[i % STAGES] == i and self.scores[i & 1] == ("s", i), "a warp reads another stage's scores")
            yield "pair"
            del self.reading[w]
            if i > 0 and self.rng.random() < 0.5:
                ok = (yield from self.wait(self.pvdone[(i - 1) & 1], (i - 1) >> 1)) and ok
                self.rescaling.add(w)
                yield "run"
                self.rescaling.discard(w)
            yield "run"
            self.pready[i & 1].arrive()
            if not self.abort and self.pready[i & 1].left == WARPS:
                self.scores[i & 1] = ("p", i)
        if ok and self.n:
            yield from self.wait(self.pvdone[(self.n - 1) & 1], (self.n - 1) >> 1)
        yield "barrier"
        if self.late_flag and self.abort:
            yield "barrier"

    # ---- the schedule
    def run(self):
        roles = {"copier": self.copier(), "products": self.products(), **{w: self.softmax(w) for w in range(WARPS)}}
        state = {r: "run" for r in roles}
        speed, idle = self.rng.choice([0.5, 0.1, 0.01]), 0   # of the engines beside the roles
        while roles:
            movable = []
            for r in list(roles):
                s = state[r]
                if s == "barrier" and any(state[x] != "barrier" for x in roles):
                    continue
                if s == "pair" and state.get(r ^ 1) != "pair":
                    continue
                movable.append(r)
            # a barrier opens for all of its roles at once
            if movable and all(state[r] == "barrier" for r in roles):
                group = list(roles)
            else:
                r = self.rng.choice(movable) if movable else None
                group = [] if r is None else [r, r ^ 1] if state[r] == "pair" else [r]
            before = (len(self.copies), len(self.queue), dict(state))
            for r in group:
                polling = state[r] == "poll"
                try:
                    # late, not lost: a wait may run out whatever is in flight
                    msg = "give up" if polling and not self.abort and self.rng.random() < self.give_up else None
                    state[r] = roles[r].send(msg)
                except StopIteration:
                    del roles[r], state[r]
            if self.rng.random() < speed:
                self.engine()
            after = (len(self.copies), len(self.queue), dict(state))
            idle = idle + 1 if before == after else 0
            if idle > 400:
                idle = 0
                need(self.engine() or self.give_up, "nothing in flight and nothing moves")
        self.released = True
        while self.engine():
            pass


@pytest.mark.parametrize("stages", [0, 1, 2, 3, 4, 5, 7, 12])
def test_schedules_without_a_give_up(stages):
    for seed in range(60):
        Cta(stages, seed, 0.0).run()


@pytest.mark.parametrize("stages", [1, 2, 3, 4, 5, 9])
@pytest.mark.parametrize("rate", [0.3, 0.05, 0.005])
def test_nothing_in_flight_after_a_give_up(stages, rate):
    for seed in range(80):
        Cta(stages, seed, rate).run()


def _seen(rates, **rules):
    found = set()
    for rate in rates:
        for stages in (1, 2, 4):
            for seed in range(200):
                try:
                    Cta(stages, seed, rate, **rules).run()
                except Violation as e:
                    found.add(str(e))
    return found


def test_a_flag_read_before_the_barrier_is_seen():
    """A role that looks at the flag when it ends does not see a wait that gives up after it."""
    found = _seen((0.05, 0.005), late_flag=False)
    assert "a copy lands in released shared memory" in found and any("in flight when the memory is released" in f for f in found)


def test_a_commit_that_nothing_waits_for_is_seen():
    assert "commit in flight when the memory is released" in _seen((0.0,), spare_freed=False)
