"""The page ring of the cache attention kernel (``csrc/attend.cu``) as a model on the CPU: one producer, eight consumer
warps, four barriers a slot, copies that land at any time, under random interleavings.

A page is *absent* where a tile's rows see none of it, or where its number is out of range: it takes its turn in the ring
and is not loaded.  The model counts arrivals as the hardware does (an arrival at a phase that has none left is an error),
checks that what a warp reads is its own page, and finds interleavings in which nobody can go on.
"""
import random

import pytest

WARPS = 8
SMEM = 227 * 1024


class Broken(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.tx = self.phase = 0

    def _turn(self):
        if self.left == 0 and self.tx == 0:
            self.left, self.phase = self.count, self.phase + 1

    def arrive(self, n=1, tx=0):
        if n > self.left:
            raise Broken("an arrival at a phase that has none left")
        self.left -= n
        self.tx += tx
        self._turn()

    def landed(self):
        self.tx -= 1
        self._turn()

    def done(self, parity):
        """Has the phase of this parity completed? (as far as a parity can say)"""
        return self.phase & 1 != parity


class Ring:
    """pages: for each range the CTA walks, (warps side by side, [is the page loaded?])."""

    def __init__(self, ring, full_side, ranges, softmax, wait_for_v, rng, give_up=None, land=True):
        """give_up: the step at which a warp's time runs out; land: the producer waits for its last
        copies always, not only where it has given up itself."""
        self.give_up, self.land, self.steps, self.fills = give_up, land, 0, {}
        self.ring, self.wt, self.ranges, self.softmax, self.wait_for_v, self.rng = ring, full_side, ranges, softmax, wait_for_v, rng
        self.full_k = [Barrier(2) for _ in range(ring)]
        self.full_v = [Barrier(1) for _ in range(ring)]
        self.empty_k = [Barrier(full_side) for _ in range(ring)]
        self.empty_v = [Barrier(full_side) for _ in range(ring)]
        self.has_k, self.has_v = [-1] * ring, [-1] * ring
        self.k, self.v = [None] * ring, [None] * ring
        self.flying = []  # (barrier, array, slot, page)
        self.at_barrier = [0] * WARPS

    def fly(self, bar, where, slot, page):
        self.flying.append((bar, where, slot, page))
        self.fills[id(bar)] = bar, page // self.ring + 1

    # every step yields whether it got on
    def produce(self):
        k_todo, v_todo = set(), set()
        pages = [x for _, r in self.ranges for x in r]
        for base in range(0, len(pages), self.ring):
            lanes = range(min(self.ring, len(pages) - base))
            turn = base // self.ring
            k_todo, v_todo = set(lanes), set(lanes)
            ph = (turn & 1) ^ 1
            while k_todo or v_todo:
                some = False
                for i in lanes:
                    n, there = base + i, pages[base + i]
                    k = i in k_todo and (turn == 0 or self.empty_k[i].done(ph))
                    if k and there:
                        self.full_k[i].arrive(1, 1)
                        self.fly(self.full_k[i], self.k, i, n)
                    v = i in v_todo and (turn == 0 or self.empty_v[i].done(ph))
                    if v:
                        self.has_v[i] = n
                        yield True
                        if there:
                            self.full_v[i].arrive(1, 1)
                            self.fly(self.full_v[i], self.v, i, n)
                    if k:
                        self.has_k[i] = n
                        yield True
                        self.full_k[i].arrive()
                        if not there:
                            self.full_k[i].arrive()
                    if v and not there:
                        self.full_v[i].arrive()
                    if k:
                        k_todo.discard(i)
                    if v:
                        v_todo.discard(i)
                    some |= k or v
                if not some and self.gone():
                    break
                yield some
            if k_todo or v_todo:
                break
        while (self.land or k_todo or v_todo) and any(bar.phase < n for bar, n in self.fills.values()):
            yield False

    def gone(self):
        return self.give_up is not None and self.steps > self.give_up

    def _wait(self, has, full, st, n, ph):
        while has[st] != n and not self.gone():
            yield False
        while not full[st].done(ph) and not self.gone():
            yield False

    def consume(self, warp):
        before, bars = 0, 0
        for side, pages in self.ranges:
            grp, ng = warp // side, WARPS // side
            for mine in range(before + grp, before + len(pages), ng):
                st, ph = mine % self.ring, mine // self.ring & 1
                if not self.gone():
                    yield from self._wait(self.has_k, self.full_k, st, mine, ph)
                if self.gone():
                    continue
                there = pages[mine - before]
                yield True
                if there and self.k[st] != mine:
                    raise Broken(f"K of page {self.k[st]} read for {mine}")
                self.empty_k[st].arrive(self.wt // side)
                yield True
                if there or self.wait_for_v:
                    for _ in range(self.softmax if there else 0):
                        yield True
                    yield from self._wait(self.has_v, self.full_v, st, mine, ph)
                    if self.gone():
                        continue
                    if there and self.v[st] != mine:
                        raise Broken(f"V of page {self.v[st]} read for {mine}")
                yield True
                self.empty_v[st].arrive(self.wt // side)
                yield True
            before += len(pages)
            bars += 1
            self.at_barrier[warp] = bars
            yield True
            while min(self.at_barrier) < bars:
                yield False

    def run(self):
        """True if everybody came to the end; False if nobody can go on."""
        actors = [self.produce()] + [self.consume(w) for w in range(WARPS)]
        idle = set()  # actors that last found nothing to do
        while actors:
            self.steps += 1
            if self.steps - 1 == self.give_up:
                idle.clear()
            i = self.rng.randrange(len(actors) + (len(self.flying) > 0))
            if i == len(actors):
                bar, where, slot, page = self.flying.pop(self.rng.randrange(len(self.flying)))
                where[slot] = page
                bar.landed()
                idle.clear()
                continue
            try:
                if next(actors[i]):
                    idle.clear()
                else:
                    idle.add(actors[i])
            except StopIteration:
                actors.pop(i)
                idle.clear()
            if actors and not self.flying and len(idle) == len(actors):
                return False
        if self.flying:
            raise Broken("the block ended with copies in flight")
        return True


def ring_of(D, P, rt, batch):
    """Slots of the ring, as the launch sizes it."""
    nt = 1 if rt == 8 else 2
    fixed = WARPS * 8 * nt * (D + 4) * 4 + WARPS * 8 * nt * 2 * 4 + 32 * 48 + 16 + batch * 16 + (batch + 1) * 8 + 128
    return min(32, (SMEM - fixed) // (2 * P * D))


def ranges_of(kind, side, rng):
    """What a CTA may have to walk: ranges of pages of which some are absent."""
    if kind == "loaded":
        return [(side, [True] * rng.randrange(20, 60)) for _ in range(2)]
    if kind == "prompt":  # tiles of one prompt: each sees a few more pages than the one before
        n = rng.randrange(16, 40)
        return [(side, [j <= i * n // 3 for j in range(n)]) for i in range(4)]
    if kind == "window":  # pages before and behind a tile's window
        n = rng.randrange(30, 60)
        return [(side, [a <= j <= a + 2 for j in range(n)]) for a in (0, n // 2, n - 2)]
    return [(side, [rng.random() < 0.9 for _ in range(rng.randrange(30, 60))]) for _ in range(2)]  # bad numbers here and there


@pytest.mark.parametrize("kind", ["loaded", "prompt", "window", "bad"])
@pytest.mark.parametrize("D, P", [(64, 32), (64, 64), (128, 32), (128, 64)])
def test_ring_comes_to_the_end_with_the_right_pages(D, P, kind):
    rng = random.Random(D + P + len(kind))
    for rt in (8, 16, 32, 64):
        full = rt // (8 * (1 if rt == 8 else 2))
        for batch in (1, 1024):
            for side in (1, 2, 4):
                if side > full:
                    continue
                for softmax in (0, 2, 12):
                    ring = ring_of(D, P, rt, batch)
                    assert ring >= WARPS
                    for _ in range(2):
                        assert Ring(ring, full, ranges_of(kind, side, rng), softmax, True, rng).run(), (rt, batch, side)


@pytest.mark.parametrize("ring", [1, 2, 3, 5, 8, 9, 11])
def test_ring_of_any_length(ring):
    """Rings shorter than the warps, and lengths that no number of groups divides."""
    rng = random.Random(ring)
    for full, side in ((1, 1), (2, 1), (2, 2), (4, 1), (4, 2), (4, 4)):
        for kind in ("loaded", "prompt", "window", "bad"):
            for softmax in (0, 6):
                assert Ring(ring, full, ranges_of(kind, side, rng), softmax, True, rng).run(), (full, side, kind)


@pytest.mark.parametrize("ring, side", [(9, 4), (12, 1), (32, 2)])
def test_a_warp_that_gives_up_leaves_no_copy_behind(ring, side):
    """Wherever time runs out, all come to the end and every copy has landed before the block does."""
    for seed in range(120):
        for kind in ("loaded", "prompt", "bad"):
            rng = random.Random(seed)
            a = ring, side, ranges_of(kind, side, rng), 3, True, rng
            whole = Ring(*a)
            assert whole.run()
            assert Ring(*a, give_up=rng.randrange(whole.steps)).run()
    left = 0  # a producer that is done before a warp gives up has to wait too
    for seed in range(20):
        a = ring, side, [(side, [True] * ring)], 3, True
        assert Ring(*a, random.Random(seed), give_up=30).run()
        try:
            Ring(*a, random.Random(seed), give_up=30, land=False).run()
        except Broken:
            left += 1
    assert left > 10


def test_model_finds_a_slot_released_too_early():
    """Warps that release an absent page's V without waiting for its turn: the model has to find it."""
    def broken(kind, softmax):
        bad = 0
        for seed in range(40):
            rng = random.Random(seed)
            try:
                bad += not Ring(9, 4, ranges_of(kind, 4, rng), softmax, False, rng).run()
            except Broken:
                bad += 1
        return bad
    assert broken("loaded", 6) == 0
    assert broken("prompt", 6) > 20 and broken("window", 6) > 0 and broken("bad", 12) > 0
