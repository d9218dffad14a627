"""The model of paged_attention.cuh's barriers with what the softmax groups
hand each other at an item's end: the maxima and sums of the two halves that
saw the same rows.  A group must find what the other one left for this item.
And with tiles whose product with V a group adds to O itself: O must be its
own by then."""
import pytest

from tests.test_attention_protocol import Model


class Results(Model):
    """`always`: a half without a tile writes its (empty) statistics, too;
    `hasty`: a product is added by hand without a wait for O."""

    by_hand_share = 0.3

    def __init__(self, seed, stages, always=False, hasty=False):
        super().__init__(seed, stages)
        self.always, self.hasty = always, hasty
        self.by_hand = set()
        self.stats, self.turns = [None, None], [0, 0]

    def does_pv(self, h, i, t, s, first):
        if (h, i, t) not in self.by_hand:
            super().does_pv(h, i, t, s, first)

    def joins(self, h, i, n, tiles):
        """The item's end where both halves hold its rows; a generator."""
        if tiles or self.always:
            self.stats[h] = (i, bool(tiles))
        for _ in range(4):
            self.altbar.arrive()
        yield lambda: self.altbar.done(self.turns[h])
        self.turns[h] ^= 1
        yield self.r.choice([1, 10, 150])        # a warp may be late to read
        assert self.stats[0] == (i, True)
        if n > 1:
            assert self.stats[1] == (i, True)

    def softmax(self, h):
        scount = done = q = 0
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
                    if j > 0:
                        self.empty[v % self.S].arrive()
                    if t == n - 1:
                        for u in (q,) if alt else (q, q + 1):
                            self.qempty[u & 1].arrive()
                v = self.v_place(base, alt, n, t)
                yield self.r.randint(1, 30)
                self.S_holds[h] = ("P", i, t)
                if self.r.random() < self.by_hand_share:     # hidden rows of V hold an infinity
                    yield lambda: self.full[v % self.S].done(v // self.S & 1)
                    assert self.holds[v % self.S] == (i, "V", t)
                    if j == 0 and not self.hasty:
                        yield lambda: self.oempty.done(i & 1 ^ 1)
                    self.by_hand.add((h, i, t))
                    before = self.O_holds[h]
                    assert j == 0 or before == [(i, u) for u in tiles[:j]]
                    self.O_holds[h] = ([] if j == 0 else before) + [(i, t)]
                    yield self.r.randint(1, 30)
                    assert self.holds[v % self.S] == (i, "V", t)
                for _ in range(4):
                    self.ready[h] += 1
            if tiles:
                yield lambda: self.pvdone[h].done(done)
                done ^= 1
                if alt or h == 1:
                    self.empty[v % self.S].arrive()
            if alt:
                yield from self.joins(h, i, n, tiles)
            q += 1 if alt else 2
            yield self.r.choice([1, 20, 40, 150])    # a warp may be late to read O, too
            for g in (0, 1) if alt else (h,):
                want = [(i, t) for t in range(n) if not alt or t % 2 == g]
                assert not want or self.O_holds[g] == want
            for _ in range(4):
                self.oempty.arrive()
                self.itempty[i % 4].arrive()


def caught(seeds, **mistake):
    n = 0
    for seed in range(seeds):
        try:
            Results(seed, 5, **mistake).run()
        except AssertionError:
            n += 1
    return n


@pytest.mark.parametrize("stages", [5, 11])
def test_groups_find_each_other_s_statistics(stages):
    for seed in range(250):
        Results(seed, stages).run()


def test_a_group_without_a_tile_must_not_write():
    """Half 1 sees none of an item of one tile: its group comes to the end at
    once and may overtake the other group's look at the item before."""
    assert caught(100, always=True) > 5


def test_a_product_added_by_hand_must_wait_for_o():
    """Where both halves hold an item's rows, each group reads both halves' O
    at its end, and either may be in its next item's first tile by then."""
    assert caught(100, hasty=True) > 5
