"""A host-side model of the pipeline of a CTA pair and of its end (rlk_pair.cuh).

Two CTAs of a cluster work one tile: each has a producer (copies into a ring
of S stages, counted on the even CTA's `full` barriers) and an epilogue; the
even CTA's issuer runs the MMAs and signals `empty` and `tfull` in both CTAs;
the epilogues hand accumulators back on the even CTA's `tempty`.  Everything
that one agent sends to a barrier or to shared memory arrives after a random
delay.  Any wait may expire at any moment in which it is not satisfied.

What has to hold when the pair exits: nothing is still on its way to either
CTA's shared memory or barriers (the memory may be another block's by then),
and no wait of the end was for something that never comes.

`rule` "even" is an end in which the even producer arms each stage for both
CTAs and, alone, waits for the stages that it issued itself; "both" is
rlk_pair.cuh's.
"""
import random

from ring_protocol_model import Bar


class Leak(AssertionError):
    pass


class Pair:
    def __init__(self, seed, stages=3, tiles=3, kblocks=4, rule="both", expire=0.0):
        self.rng = random.Random(seed)
        self.S, self.tiles, self.K, self.rule, self.expire = stages, tiles, kblocks, rule, expire
        self.full = [Bar(2 if rule == "both" else 1) for _ in range(stages)]  # the even CTA's
        self.empty = [[Bar(1) for _ in range(stages)] for _ in range(2)]
        self.tfull = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.tempty = [Bar(2) for _ in range(2)]                              # the even CTA's: one arrival a CTA
        self.drain = [Bar(1) for _ in range(2)]
        self.abort = [False, False]
        self.issued = [0, 0]
        self.drained = False
        self.flights = []  # (delivery time, what is sent, by a thread's own instruction?)
        self.now = 0
        self.stuck = 0     # waits of the end that nothing satisfies
        self.slow = False  # whether the pair took the way of an expired wait

    def send(self, action, most=30, own=False):
        self.flights.append((self.now + self.rng.randint(0, most), action, own))

    def step(self):
        self.now += 1
        due = [f for f in self.flights if f[0] <= self.now]
        self.flights = [f for f in self.flights if f[0] > self.now]
        for f in due:
            f[1]()

    # An agent is a generator: it yields while it waits.
    def wait(self, cta, bar, parity):
        while not bar.try_wait(parity):
            if self.abort[cta]:
                return False
            if self.rng.random() < self.expire:
                self.abort[cta] = True
                return False
            yield
        return True

    def until(self, bar, parity, limit=500):
        """A wait of the end: bounded, for what has to come."""
        for _ in range(limit):
            if bar.try_wait(parity):
                return
            yield
        self.stuck += 1

    @staticmethod
    def landed(bar, nbytes):
        bar.tx -= nbytes
        bar.check()

    @staticmethod
    def arm(bar, nbytes):
        bar.tx += nbytes
        bar.arrive()

    def producer(self, cta):
        ok, j, n = True, 0, self.tiles * self.K
        while ok and j < n:
            s = j % self.S
            ok = yield from self.wait(cta, self.empty[cta][s], (j // self.S) & 1 ^ 1)
            if not ok:
                break
            bar = self.full[s]
            if self.rule == "both":
                self.send(lambda bar=bar: self.arm(bar, 10), most=30 if cta else 0, own=True)
            elif cta == 0:
                self.arm(bar, 20)
            self.send(lambda bar=bar: self.landed(bar, 10))
            j += 1
            if self.rng.random() < 0.5:
                yield
        self.issued[cta] = j
        if self.rule == "even":
            if cta == 0:
                for k in range(max(0, j - self.S), j):
                    yield from self.until(self.full[k % self.S], (k // self.S) & 1)
            return
        for k in range(j, j + self.S):  # its stages are free again: their copies and their signals have landed
            ok = ok and (yield from self.wait(cta, self.empty[cta][k % self.S], (k // self.S) & 1 ^ 1))

    def issuer(self):
        ok, j, t = True, 0, 0
        while ok and t < self.tiles:
            ok = yield from self.wait(0, self.tempty[t % 2], (t // 2) & 1 ^ 1)
            for _ in range(self.K):
                ok = ok and (yield from self.wait(0, self.full[j % self.S], (j // self.S) & 1))
                if not ok:
                    break
                yield
                for cta in range(2):
                    self.send(self.empty[cta][j % self.S].arrive)
                j += 1
            if ok:
                for cta in range(2):
                    self.send(self.tfull[cta][t % 2].arrive)
                t += 1
        if self.rule == "both":
            for k in range(t, t + 2):  # the accumulators are handed back
                ok = ok and (yield from self.wait(0, self.tempty[k % 2], (k // 2) & 1 ^ 1))
        if self.rule == "even" or not ok:
            last = max([f[0] for f in self.flights], default=self.now)
            for cta in range(2):  # behind everything that the issuer has signalled so far
                self.flights.append((last + self.rng.randint(0, 10), self.drain[cta].arrive, False))
            self.drained = True
            yield from self.until(self.drain[0], 0)

    def epilogue(self, cta):
        for t in range(self.tiles):
            if not (yield from self.wait(cta, self.tfull[cta][t % 2], (t // 2) & 1)):
                return
            for _ in range(self.rng.randint(0, 6)):
                yield
            self.send(self.tempty[t % 2].arrive, most=30 if cta else 0, own=True)

    def end(self, cta):
        """The ends of the two CTAs after they met, when a wait has expired in either."""
        if cta == 0:
            lo, hi = min(self.issued), max(self.issued)
            for k in range(lo, hi):  # stages that only one CTA issued: the other's arrival, without bytes
                self.full[k % self.S].arrive()
            for k in range(max(0, hi - self.S), hi):
                yield from self.until(self.full[k % self.S], (k // self.S) & 1)
        elif self.drained:
            yield from self.until(self.drain[1], 0)

    def run_all(self, agents):
        agents = list(agents)
        for _ in range(100000):
            if not agents:
                return
            self.rng.shuffle(agents)
            for a in list(agents):
                if self.rng.random() < 0.7:
                    try:
                        next(a)
                    except StopIteration:
                        agents.remove(a)
            self.step()
        raise Leak("the pair does not end")

    def run(self):
        self.run_all([self.producer(0), self.producer(1), self.issuer(), self.epilogue(0), self.epilogue(1)])
        self.slow = any(self.abort)
        if self.rule == "both" and self.slow:
            # the two CTAs have met and both know: a barrier that releases and acquires, the end, another
            self.flush()
            self.run_all([self.end(0), self.end(1)])
            self.flush()
        if self.flights:
            raise Leak(f"{len(self.flights)} signals or copies on their way to a CTA that has left")
        if self.stuck:
            raise Leak(f"{self.stuck} waits of the end for what never comes")

    def flush(self):
        """A barrier that releases performs its threads' own arrivals, not their asynchronous copies and commits."""
        for f in [f for f in self.flights if f[2]]:
            self.flights.remove(f)
            f[1]()
