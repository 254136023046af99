"""The page ring of the cache attention kernel with loads that take their time, as a model on the CPU: a warp's loads of a page
are done some time after it has issued them.  Released before, the slot's next page may land under them."""
import random

import pytest

import test_attend_ring as ring_model


class Load:
    """Data of a slot, as a load sees it when it is done."""

    def __init__(self, data):
        self.data, self.done = data, False

    def __setitem__(self, slot, page):
        if self.data[slot] != page:
            raise ring_model.Broken(f"page {self.data[slot]} read for {page}")

    def landed(self):
        self.done = True


class Ring(ring_model.Ring):
    def __init__(self, *a, fence=True, **kw):
        super().__init__(*a, **kw)
        self.fence = fence

    def load(self, data, st, mine):
        x = Load(data)
        self.flying.append((x, x, st, mine))  # done at any time
        while self.fence and not x.done:
            yield False

    def consume(self, warp):
        before, bars = 0, 0
        for side, pages in self.ranges:
            grp, ng = warp // side, ring_model.WARPS // side
            for mine in range(before + grp, before + len(pages), ng):
                st, ph = mine % self.ring, mine // self.ring & 1
                yield from self._wait(self.has_k, self.full_k, st, mine, ph)
                yield True
                there = pages[mine - before]
                if there:
                    yield from self.load(self.k, st, mine)
                self.empty_k[st].arrive(self.wt // side)
                yield True
                yield from self._wait(self.has_v, self.full_v, st, mine, ph)
                if there:
                    yield from self.load(self.v, st, mine)
                self.empty_v[st].arrive(self.wt // side)
                yield True
            before += len(pages)
            bars += 1
            self.at_barrier[warp] = bars
            yield True
            while min(self.at_barrier) < bars:
                yield False


@pytest.mark.parametrize("warps", [4, 8])
@pytest.mark.parametrize("length", [3, 5, 10, 23])
def test_slots_are_released_when_their_loads_are_done(monkeypatch, warps, length):
    monkeypatch.setattr(ring_model, "WARPS", warps)
    broken = 0
    for seed in range(10):
        for fence in (True, False):
            rng = random.Random(seed * 100 + length)
            ranges = ring_model.ranges_of("loaded", 1, rng) + [(1, [True] * 60)]
            try:
                assert Ring(length, 1, ranges, 0, True, rng, fence=fence).run()
            except ring_model.Broken:
                assert not fence
                broken += 1
    assert broken
