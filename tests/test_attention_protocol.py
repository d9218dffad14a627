"""A model of paged_attention.cuh's barrier protocol: the producer, the thread
that counts landed copies, the MMA issuer and the two softmax groups as
processes over parity barriers, with random delays and copies that land out of
order.  No schedule may deadlock, arrive too often at a barrier, or let a role
read a stage, Q, S, P or O that is not the one it wants."""
import heapq
import random

import pytest


class Bar:
    """An mbarrier: `count` arrivals (and the announced copies) end a phase."""

    def __init__(self, count):
        self.count, self.left, self.copies, self.phase = count, count, 0, 0

    def _step(self):
        if self.left == 0 and self.copies == 0:
            self.phase, self.left = self.phase + 1, self.count

    def arrive(self, copies=0):
        assert self.left > 0, "one arrival too many"
        self.copies += copies
        self.left -= 1
        self._step()

    def landed(self):
        self.copies -= 1
        self._step()

    def done(self, parity):
        """What try_wait.parity says: the running phase has the other parity."""
        return self.phase & 1 != parity


class Model:
    def __init__(self, seed, stages, in_order=True, early=False):
        self.r, self.S, self.in_order, self.early = random.Random(seed), stages, in_order, early
        r = self.r
        # (halves take turns, tiles) of the CTA's items
        self.items = [(r.random() < 0.6, r.choice([1, 1, 2, 3, 4, 5, 9, 20])) for _ in range(r.randint(3, 14))]
        self.slow = r.choice([1, 10, 60])
        self.full = [Bar(1) for _ in range(stages)]
        self.empty = [Bar(1) for _ in range(stages)]
        self.holds = [None] * stages
        self.qfull, self.qempty, self.qholds = [Bar(1), Bar(1)], [Bar(1), Bar(1)], [None, None]
        self.sfull, self.pvdone = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
        self.ready, self.landed, self.total = [0, 0], 0, -1
        self.oempty, self.altbar = Bar(8), Bar(8)
        self.itfull, self.itempty = [Bar(1) for _ in range(4)], [Bar(9) for _ in range(4)]
        self.S_holds, self.O_holds = [None, None], [[], []]
        self.now, self.events, self.serial, self.tensor = 0, [], 0, 0

    def at(self, when, what, *args):
        self.serial += 1
        heapq.heappush(self.events, (when, self.serial, what, args))

    # ---- places of an item's tiles in the ring
    @staticmethod
    def ahead(alt):
        return 2 if alt else 1

    def k_place(self, base, alt, t):
        a = self.ahead(alt)
        return base + (t if t < a else 2 * t - a + 1)

    def v_place(self, base, alt, n, t):
        return base + t + min(n, t + self.ahead(alt))

    # ---- roles: generators that yield a condition to wait for, or a delay
    def producer(self):
        place = q = 0
        for i, (alt, n) in enumerate(self.items):
            yield lambda: self.itempty[i % 4].done(i // 4 & 1 ^ 1)
            self.itfull[i % 4].arrive()
            for h in (0,) if alt else (0, 1):
                yield lambda: self.qempty[q & 1].done(q >> 1 & 1 ^ 1)
                self.qfull[q & 1].arrive(1)
                self.at(self.now + self.r.randint(5, 20 * self.slow), self.q_lands, q & 1, (i, h))
                q += 1
            a = self.ahead(alt)
            order = [("K", t) for t in range(min(a, n))]
            for t in range(n):
                order.append(("V", t))
                if t + a < n:
                    order.append(("K", t + a))
            for kind, t in order:
                where = self.k_place(self._base(i), alt, t) if kind == "K" else self.v_place(self._base(i), alt, n, t)
                assert where == place
                s = place % self.S
                yield lambda: self.empty[s].done(place // self.S & 1 ^ 1)
                self.full[s].arrive(1)
                self.at(self.now + self.r.randint(5, 20 * self.slow), self.stage_lands, s, (i, kind, t))
                place += 1
                yield self.r.randint(1, 5)
        i = len(self.items)
        yield lambda: self.itempty[i % 4].done(i // 4 & 1 ^ 1)
        self.itfull[i % 4].arrive()
        self.total = place
        for p in range(max(0, place - self.S), place):
            yield lambda: self.full[p % self.S].done(p // self.S & 1)

    def _base(self, item):
        return sum(2 * n for _, n in self.items[:item])

    def q_lands(self, s, what):
        self.qholds[s] = what
        self.qfull[s].landed()

    def stage_lands(self, s, what):
        self.holds[s] = what
        self.full[s].landed()

    def lander(self):
        place = 0
        if not self.in_order:
            self.landed = 10 ** 9
            return
        while True:
            yield lambda: self.full[place % self.S].done(place // self.S & 1) or self.total == place
            if self.total == place:
                return
            place += 1
            self.landed = place

    def issue(self, what, *args):
        self.tensor = max(self.tensor, self.now) + 8
        self.at(self.tensor - 0.5, what, *args)

    def commit(self, bar):
        self.at(max(self.tensor, self.now + 1), bar.arrive)

    def does_s(self, h, i, t, s, q):
        want = (i, 0 if self.items[i][0] else h)
        assert self.holds[s] == (i, "K", t) and self.qholds[q & 1] == want, (self.holds[s], i, t)
        self.S_holds[h] = ("S", i, t)

    def does_pv(self, h, i, t, s, first):
        assert self.holds[s] == (i, "V", t) and self.S_holds[h] == ("P", i, t), (self.holds[s], self.S_holds[h], i, t)
        self.O_holds[h] = ([] if first else self.O_holds[h]) + [(i, t)]

    def issuer(self):
        place, count, q = 0, [0, 0], 0
        for i, (alt, n) in enumerate(self.items + [(False, 0)]):
            yield lambda: self.itfull[i % 4].done(i // 4 & 1)
            self.itempty[i % 4].arrive()
            if i == len(self.items):
                return
            k = place % self.S
            place += 1
            for u in (q,) if alt else (q, q + 1):
                yield lambda: self.qfull[u & 1].done(u >> 1 & 1)
            yield lambda: self.landed >= place
            self.issue(self.does_s, 0, i, 0, k, q)
            self.commit(self.sfull[0])
            if not alt:
                self.issue(self.does_s, 1, i, 0, k, q + 1)
                self.commit(self.sfull[1])
            elif n > 1:
                k = place % self.S
                place += 1
                yield lambda: self.landed >= place
                self.issue(self.does_s, 1, i, 1, k, q)
                self.commit(self.sfull[1])
            yield lambda: self.oempty.done(i & 1 ^ 1)
            a = self.ahead(alt)
            for t in range(n):
                v = place % self.S
                place += 1
                if t + a < n:
                    k = place % self.S
                    place += 1
                for h in ([t & 1] if alt else [0, 1]):
                    count[h] += 1
                    yield lambda: self.landed >= place and self.ready[h] == 4 * count[h]
                    self.issue(self.does_pv, h, i, t, v, t < a)
                    if t + a < n:
                        self.issue(self.does_s, h, i, t + a, k, q if alt else q + h)
                        self.commit(self.sfull[h])
                    else:
                        self.commit(self.pvdone[h])
                    yield self.r.randint(1, 10)
            q += a ^ 3

    def softmax(self, h):
        scount = done = turns = q = 0
        for i, (alt, n) in enumerate(self.items + [(False, 0)]):
            yield lambda: self.itfull[i % 4].done(i // 4 & 1)
            if i == len(self.items):
                return
            base = self._base(i)
            tiles = [t for t in range(n) if not alt or t % 2 == h]
            v = 0
            for j, t in enumerate(tiles):
                yield lambda: self.sfull[h].done(scount & 1)
                scount += 1
                assert self.S_holds[h] == ("S", i, t)
                if alt or h == 1:
                    self.empty[self.k_place(base, alt, t) % self.S].arrive()
                    if self.early:
                        self.empty[self.v_place(base, alt, n, t) % self.S].arrive()
                    elif j > 0:
                        self.empty[v % self.S].arrive()
                    if t == n - 1:
                        for u in (q,) if alt else (q, q + 1):
                            self.qempty[u & 1].arrive()
                v = self.v_place(base, alt, n, t)
                yield self.r.randint(1, 30)
                if t == n - 1 or self.r.random() < 0.3:      # a tile with hidden keys
                    yield lambda: self.full[v % self.S].done(v // self.S & 1)
                    assert self.holds[v % self.S] == (i, "V", t)
                self.S_holds[h] = ("P", i, t)
                for _ in range(4):
                    self.ready[h] += 1
            if tiles:
                yield lambda: self.pvdone[h].done(done)
                done ^= 1
                if (alt or h == 1) and not self.early:
                    self.empty[v % self.S].arrive()
            if alt:
                for _ in range(4):
                    self.altbar.arrive()
                yield lambda: self.altbar.done(turns)
                turns ^= 1
            q += 1 if alt else 2
            yield self.r.randint(1, 40)
            for g in (0, 1) if alt else (h,):
                want = [(i, t) for t in range(n) if not alt or t % 2 == g]
                assert not want or self.O_holds[g] == want
            for _ in range(4):
                self.oempty.arrive()
                self.itempty[i % 4].arrive()

    def run(self):
        roles = [self.producer(), self.lander(), self.issuer(), self.softmax(0), self.softmax(1)]
        waits, wake = [None] * 5, [0] * 5
        while any(r is not None for r in roles):
            moved = False
            while self.events and self.events[0][0] <= self.now:
                _, _, what, args = heapq.heappop(self.events)
                what(*args)
                moved = True
            for k in self.r.sample(range(5), 5):
                if roles[k] is None or (callable(waits[k]) and not waits[k]()) or wake[k] > self.now:
                    continue
                moved = True
                try:
                    waits[k] = next(roles[k])
                except StopIteration:
                    roles[k] = None
                    continue
                if not callable(waits[k]):
                    wake[k] = self.now + waits[k]
            if not moved:
                later = [w for k, w in enumerate(wake) if roles[k] is not None and w > self.now]
                later += [self.events[0][0]] if self.events else []
                assert later, f"deadlock: {self.items}"
                self.now = min(later)


@pytest.mark.parametrize("stages", [5, 11])
def test_every_schedule_ends_and_reads_what_it_wants(stages):
    for seed in range(250):
        Model(seed, stages).run()


@pytest.mark.parametrize("mistake", [dict(in_order=False), dict(early=True)])
def test_the_model_sees_mistakes(mistake):
    """An issuer that does not wait for copies, or a stage released with its
    tile's scores instead of its product, is caught."""
    caught = 0
    for seed in range(50):
        try:
            Model(seed, 5, **mistake).run()
        except AssertionError:
            caught += 1
    assert caught > 25
