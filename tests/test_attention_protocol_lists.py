"""The model of paged_attention.cuh's barriers for listed positions: two warps
copy half of each tile's rows with cp.async and say so themselves when a copy
is complete, the oldest first, at the latest when three newer ones are under
way, and before that wherever one of them has to wait for a stage."""
import heapq

import pytest

from tests.test_attention_protocol import Bar
from tests.test_attention_protocol_results import Results


class Lists(Results):
    """`under_way`: copies that may be under way at once; `stubborn`: none is
    handed over while a warp waits for a stage; `blind`: copies are handed over
    before they are complete."""

    by_hand_share = 0.0                      # what is not listed comes as zeros

    def __init__(self, seed, stages, under_way=3, stubborn=False, blind=False):
        super().__init__(seed, stages)
        self.under_way, self.stubborn, self.blind = under_way, stubborn, blind
        self.items = [(True, n) for _, n in self.items]
        self.full = [Bar(2) for _ in range(stages)]
        self.parts = [[None, None] for _ in range(stages)]
        self.complete = [set(), set()]

    def does_s(self, h, i, t, s, q):
        assert self.parts[s] == [(i, "K", t)] * 2, (self.parts[s], i, t)
        assert self.qholds[q & 1] == (i, 0)
        self.S_holds[h] = ("S", i, t)

    def does_pv(self, h, i, t, s, first):
        assert self.parts[s] == [(i, "V", t)] * 2, (self.parts[s], i, t)
        assert self.S_holds[h] == ("P", i, t)
        self.O_holds[h] = ([] if first else self.O_holds[h]) + [(i, t)]

    def part_lands(self, half, place, what):
        self.parts[place % self.S][half] = what
        self.complete[half].add(place)

    def copier(self, half):
        S, lead = self.S, half == 0
        pos = handed = q = 0

        def hand_over():
            nonlocal handed
            assert pos - handed - 1 <= self.under_way     # newer ones
            if not self.blind:
                yield lambda: all(p in self.complete[half] for p in range(handed + 1))
            self.full[handed % S].arrive()
            handed += 1

        for i, (_, n) in enumerate(self.items):
            if lead:
                yield lambda: self.itempty[i % 4].done(i // 4 & 1 ^ 1)
                self.itfull[i % 4].arrive()
                yield lambda: self.qempty[q & 1].done(q >> 1 & 1 ^ 1)
                self.qfull[q & 1].arrive(1)
                self.at(self.now + self.r.randint(5, 20 * self.slow), self.q_lands, q & 1, (i, 0))
                q += 1
            nk = nv = 0
            while nv < n:
                is_k = nk < n and nk - nv < 2
                what = (i, "K", nk) if is_k else (i, "V", nv)
                assert pos == (self.k_place(self._base(i), True, nk) if is_k else
                               self.v_place(self._base(i), True, n, nv))
                while not self.empty[pos % S].done(pos // S & 1 ^ 1):
                    if handed < pos and not self.stubborn:
                        yield from hand_over()
                    else:
                        yield lambda: self.empty[pos % S].done(pos // S & 1 ^ 1)
                self.at(self.now + self.r.randint(5, 20 * self.slow), self.part_lands, half, pos, what)
                pos += 1
                if pos - handed > self.under_way:
                    yield from hand_over()
                nk, nv = (nk + 1, nv) if is_k else (nk, nv + 1)
                yield self.r.randint(1, 5)
        while handed < pos:
            yield from hand_over()
        if lead:
            i = len(self.items)
            yield lambda: self.itempty[i % 4].done(i // 4 & 1 ^ 1)
            self.itfull[i % 4].arrive()
            self.total = pos
            for p in range(max(0, pos - S), pos):
                yield lambda: self.full[p % S].done(p // S & 1)

    def run(self):
        roles = [self.copier(0), self.copier(1), self.lander(), self.issuer(), self.softmax(0), self.softmax(1)]
        waits, wake = [None] * len(roles), [0] * len(roles)
        while any(r is not None for r in roles):
            moved = False
            while self.events and self.events[0][0] <= self.now:
                _, _, what, args = heapq.heappop(self.events)
                what(*args)
                moved = True
            for k in self.r.sample(range(len(roles)), len(roles)):
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
        Lists(seed, stages).run()


@pytest.mark.parametrize("mistake", [dict(under_way=5, stubborn=True), dict(blind=True)])
def test_the_model_sees_mistakes(mistake):
    """As many copies kept back as there are stages, or a stage announced
    before its rows are there."""
    caught = 0
    for seed in range(50):
        try:
            Lists(seed, 5, **mistake).run()
        except AssertionError:
            caught += 1
    assert caught > 25
