"""The pair's pipeline as the FP8 products run it (rlk_fp8_gemm.cuh), on pair_protocol_model's barriers and end.

A tile has a number of K groups of its own: none for a group without rows and for the rows behind the groups.  Each K
group is a stage of the ring and an accumulator, of which two or (half tiles) four are in flight.  A CTA without a row
of the tile copies its half of B only, so that the two producers arm a stage for different bytes.  Scales come by runs
of several K groups through two slots of each CTA's own, whose producer's copies arrive by themselves and are waited
for at its end.
"""
from pair_protocol_model import Leak, Pair
from ring_protocol_model import Bar

OF_A, OF_B = 7, 10  # bytes of a stage's copies
RUN, SLOTS = 3, 2   # K groups of a run of scales


class Tiles(Pair):
    def __init__(self, seed, stages, accs, tiles, expire=0.0, hand_back=None):
        """tiles: (K groups, whether the even and the odd CTA have a row) of each.  hand_back: accumulators that the
        issuer waits for at its end (all of them where None)."""
        super().__init__(seed, stages, len(tiles), 0, "both", expire)
        self.accs, self.work = accs, tiles
        self.hand_back = accs if hand_back is None else hand_back
        self.tfull = [[Bar(1) for _ in range(accs)] for _ in range(2)]
        self.tempty = [Bar(2) for _ in range(accs)]
        self.sfull = [[Bar(1) for _ in range(SLOTS)] for _ in range(2)]
        self.sempty = [[Bar(1) for _ in range(SLOTS)] for _ in range(2)]
        self.read = [[], []]  # (tile, K group) that each CTA's epilogue has summed
        self.held = [[None] * accs for _ in range(2)]  # what an accumulator holds, of each CTA

    def producer(self, cta):
        ok, j = True, 0
        for groups, rows in self.work:
            for _ in range(groups):
                s = j % self.S
                ok = yield from self.wait(cta, self.empty[cta][s], (j // self.S) & 1 ^ 1)
                if not ok:
                    break
                bar, mine = self.full[s], rows[cta]
                self.send(lambda bar=bar, n=OF_B + (OF_A if mine else 0): self.arm(bar, n), most=30 if cta else 0, own=True)
                if mine:
                    self.send(lambda bar=bar: self.landed(bar, OF_A))
                self.send(lambda bar=bar: self.landed(bar, OF_B))
                j += 1
                if self.rng.random() < 0.5:
                    yield
            if not ok:
                break
        self.issued[cta] = j
        for k in range(j, j + self.S):
            ok = ok and (yield from self.wait(cta, self.empty[cta][k % self.S], (k // self.S) & 1 ^ 1))

    def issuer(self):
        ok, j, A = True, 0, self.accs
        for tile, (groups, _) in enumerate(self.work):
            for g in range(groups):
                ok = yield from self.wait(0, self.full[j % self.S], (j // self.S) & 1)
                ok = ok and (yield from self.wait(0, self.tempty[j % A], (j // A) & 1 ^ 1))
                if not ok:
                    break
                yield
                for cta in range(2):
                    def done(cta=cta, a=j % A, what=(tile, g)):
                        self.held[cta][a] = what
                        self.tfull[cta][a].arrive()
                    self.send(done)
                    self.send(self.empty[cta][j % self.S].arrive)
                j += 1
            if not ok:
                break
        for k in range(j, j + self.hand_back):
            ok = ok and (yield from self.wait(0, self.tempty[k % A], (k // A) & 1 ^ 1))
        if not ok:
            last = max([f[0] for f in self.flights], default=self.now)
            for cta in range(2):
                self.flights.append((last + self.rng.randint(0, 10), self.drain[cta].arrive, False))
            self.drained = True
            yield from self.until(self.drain[0], 0)

    def scales(self, cta):
        ok, n, landed = True, 0, []
        for groups, _ in self.work:
            for _ in range(0, groups, RUN):
                ok = yield from self.wait(cta, self.sempty[cta][n % SLOTS], (n // SLOTS) & 1 ^ 1)
                if not ok:
                    break

                def land(bar=self.sfull[cta][n % SLOTS]):
                    landed.append(1)
                    bar.arrive()
                self.send(land)
                n += 1
            if not ok:
                break
        while len(landed) < n:
            yield

    def epilogue(self, cta):
        j, n, A = 0, 0, self.accs
        for tile, (groups, _) in enumerate(self.work):
            for g in range(groups):
                if g % RUN == 0 and not (yield from self.wait(cta, self.sfull[cta][n % SLOTS], (n // SLOTS) & 1)):
                    return
                if not (yield from self.wait(cta, self.tfull[cta][j % A], (j // A) & 1)):
                    return
                for _ in range(self.rng.randint(0, 4)):
                    yield
                if self.held[cta][j % A] != (tile, g):
                    raise Leak(f"accumulator {j % A} holds {self.held[cta][j % A]}, not {(tile, g)}")
                self.read[cta].append((tile, g))
                self.send(self.tempty[j % A].arrive, most=30 if cta else 0, own=True)
                j += 1
                if g % RUN == RUN - 1 or g == groups - 1:
                    self.sempty[cta][n % SLOTS].arrive()
                    n += 1
            for _ in range(self.rng.randint(0, 9)):  # the tile's results go to memory
                yield

    def run(self):
        self.run_all([self.producer(0), self.producer(1), self.issuer(), *(f(c) for f in (self.epilogue, self.scales)
                                                                           for c in range(2))])
        self.slow = any(self.abort)
        if self.slow:
            self.flush()
            self.run_all([self.end(0), self.end(1)])
            self.flush()
        if self.flights:
            raise Leak(f"{len(self.flights)} signals or copies on their way to a CTA that has left")
        if self.stuck:
            raise Leak(f"{self.stuck} waits of the end for what never comes")
