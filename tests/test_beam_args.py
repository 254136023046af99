"""Attention over shared prefixes, sinks, beam selection and reordering on the CPU: what the calls refuse before any launch,
which stream they use, the plain implementations that the GPU tests compare with, and a model of the tiles' pipeline."""
import ctypes as C
import itertools
import math
import random

import pytest
import torch

import beam_ref
import test_attend_ring as ring_model
from persistent_megakernel_decode_gb300 import runtime as rt
from test_serve_args import A, attend, desc
from test_serve_streams import BF16, I32, Stream, cache, machine  # noqa: F401  (machine is a fixture)


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()


REFUSED = (rt.MK_ERR_INVALID, rt.MK_ERR_UNSUPPORTED)


# ---- the C ABI ----
def test_sinks_refusals():
    lib = rt.load()
    for bad in (dict(sinks=-1), dict(window=5, sinks=-7)):
        assert lib.mk_cache_attend(C.byref(desc()), 0, C.byref(attend(**bad)), A, 1 << 30, None) == rt.MK_ERR_INVALID


@pytest.mark.parametrize("groups, kw", [
    (dict(groups=-1), {}), (dict(groups=4), {}), (dict(first=0), {}), (dict(shared=0), {}), (dict(first=A + 2), {}),
    ({}, dict(window=8)), ({}, dict(window=8, sinks=2)), ({}, dict(sinks=1)), ({}, dict(q=0)), ({}, dict(q_heads=6)),
    ({}, dict(batch=1024, tokens=1024)), (dict(groups=513), dict(batch=513, tokens=513)), ({}, dict(scale=-1.0))])
def test_shared_refusals(groups, kw):
    lib, s = rt.load(), rt.SharedDesc(A, A, 2)
    for k, v in groups.items():
        setattr(s, k, v)
    assert lib.mk_cache_attend_shared(C.byref(desc()), 0, C.byref(attend(**kw)), C.byref(s), A, 1 << 40, None) in REFUSED


def test_shared_refuses_layers_and_workspaces():
    lib, a, s, need, plain = rt.load(), attend(), rt.SharedDesc(A, A, 2), C.c_uint64(), C.c_uint64()
    assert lib.mk_cache_attend_shared_workspace(C.byref(desc()), C.byref(a), C.byref(s), C.byref(need)) == rt.MK_OK
    assert lib.mk_cache_attend_workspace(C.byref(desc()), C.byref(a), C.byref(plain)) == rt.MK_OK and need.value > plain.value
    for layer, ws, n in ((-1, A, need.value), (2, A, need.value), (0, None, need.value), (0, A + 4, need.value), (0, A, need.value - 1)):
        assert lib.mk_cache_attend_shared(C.byref(desc()), layer, C.byref(a), C.byref(s), ws, n, None) == rt.MK_ERR_INVALID
    assert lib.mk_cache_attend_shared(C.byref(desc()), 0, C.byref(a), None, A, need.value, None) == rt.MK_ERR_INVALID
    for kw in (dict(batch=0, tokens=0), dict(tokens=0, max_tokens=0)):  # nothing to do
        s0 = rt.SharedDesc(A, A, 0)
        assert lib.mk_cache_attend_shared(C.byref(desc()), 0, C.byref(attend(**kw)), C.byref(s0), A, 1 << 30, None) == rt.MK_OK


def beam(**kw):
    d = rt.BeamDesc()
    d.logits = d.scores = d.out_scores = d.parents = d.tokens = A
    d.row_stride, d.batch, d.beams, d.vocab, d.num, d.end = 1000, 2, 4, 1000, 8, 0
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("bad", [dict(logits=0), dict(scores=0), dict(out_scores=0), dict(parents=0), dict(tokens=0), dict(batch=-1),
                                 dict(beams=0), dict(beams=65), dict(num=0), dict(num=129), dict(vocab=0), dict(row_stride=999),
                                 dict(vocab=622593, row_stride=622593), dict(logits=A + 2), dict(tokens=A + 1),
                                 dict(finished=A, end=-1), dict(finished=A, end=1000), dict(batch=1 << 30)])
def test_select_refusals(bad):
    lib = rt.load()
    assert lib.mk_beam_select(C.byref(beam(**bad)), A, 1 << 40, None) in REFUSED


def test_select_workspaces_and_nothing_to_do():
    lib, need = rt.load(), C.c_uint64()
    assert lib.mk_beam_select_workspace(C.byref(beam()), C.byref(need)) == rt.MK_OK and need.value > 0
    for ws, n in ((None, need.value), (A + 8, need.value), (A, need.value - 1)):
        assert lib.mk_beam_select(C.byref(beam()), ws, n, None) == rt.MK_ERR_INVALID
    assert lib.mk_beam_select(C.byref(beam(batch=0)), None, 0, None) == rt.MK_OK
    assert lib.mk_beam_select(None, A, 1 << 30, None) == rt.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(beams=0), dict(beams=65), dict(width=0), dict(table=None), dict(lens=None),
                                 dict(parents=None), dict(out=None), dict(out=A + 32), dict(out=A), dict(batch=1 << 30)])
def test_reorder_refusals(bad):
    a = dict(table=A, lens=A, parents=A, out=A + (1 << 20), batch=3, beams=4, width=8)
    a.update(bad)
    call = lambda: rt.load().mk_cache_reorder(C.byref(desc()), *[a[k] for k in ("table", "lens", "parents", "out", "batch", "beams", "width")],  # noqa: E731
                                              None)
    assert call() in REFUSED
    a.update(batch=0, beams=4, width=8)
    assert call() == rt.MK_OK  # nothing to do
    d = desc(page_tokens=16)
    assert rt.load().mk_cache_reorder(C.byref(d), A, A, A, A + 999, 1, 2, 3, None) == rt.MK_ERR_UNSUPPORTED


# ---- the binding ----
def test_select_checks_its_tensors(machine):
    z, s = torch.zeros(6, 100), torch.zeros(2, 3)
    for args in ((z[0], s), (z.double(), s), (z, s[0]), (z, torch.zeros(2, 2)), (z, s.double()), (z.T, torch.zeros(20, 5))):
        with pytest.raises(ValueError):
            rt.beam_select(*args)
    for fin in (torch.zeros(2, 3), torch.zeros(3, 2, dtype=torch.bool)):
        with pytest.raises(ValueError, match="finished"):
            rt.beam_select(z, s, finished=fin)
    assert not machine.launches
    out = rt.beam_select(z, s, num=5)
    assert [tuple(x.shape) for x in out] == [(2, 5)] * 3 and out[1].dtype == out[2].dtype == I32
    (_, call, args), = machine.launches
    assert call is rt.load().mk_beam_select and args[0]._obj.num == 5 and args[2] >= 6 * 5 * 8


def test_select_works_on_its_own_stream(machine):
    z, sc, s = torch.zeros(4, 100), torch.zeros(2, 4)[:, ::2], Stream(9)
    fin = torch.zeros(2, 4, dtype=torch.bool)[:, ::2]
    out = rt.beam_select(z, sc, finished=fin, stream=s)
    (handle, _, _), = machine.launches
    assert handle == 9 and {h for _, h in machine.made} == {9}
    for t in (z, sc, fin):
        assert (t.data_ptr(), 9) in machine.recorded
    for t in out:
        assert (t.data_ptr(), 0) in machine.recorded


def test_shared_and_reorder_check_and_use_their_stream(machine, monkeypatch):
    c = cache(monkeypatch)
    monkeypatch.setattr(c, "_workspace", lambda a, share=None: 4096 * a.batch + (share.groups if share else 0))
    q, tab, lens = torch.zeros((4, 1, 2, 64), dtype=BF16), torch.zeros((4, 3), dtype=I32), torch.ones(4, dtype=I32)
    first, shared = torch.tensor([0, 2, 4], dtype=I32), torch.zeros(2, dtype=I32)
    for bad in ((first.long(), shared), (first, shared[:1]), (first[:0], shared), (first, shared.float()), (first[::2], shared[:1])):
        with pytest.raises(ValueError):
            c.attend_shared(q, tab, lens, *bad)
    s = Stream(9)
    c.attend_shared(q, tab, lens, first, shared, stream=s)
    handle, call, args = machine.launches[-1]
    assert handle == 9 and call is c._lib.mk_cache_attend_shared and args[3]._obj.groups == 2 and args[5] == 4096 * 4 + 2
    for t in (q, tab, lens, first, shared, c.k, c.status):
        assert (t.data_ptr(), 9) in machine.recorded
    par = torch.zeros((2, 2), dtype=I32)
    for bad in ((tab, lens, par[0]), (tab[:3], lens, par), (tab, lens[:2], par), (tab, lens, par.long()), (tab.T, lens, par)):
        with pytest.raises(ValueError):
            c.reorder(*bad)
    with pytest.raises(ValueError, match="out"):
        c.reorder(tab, lens, par, out=torch.zeros((4, 2), dtype=I32))
    out = c.reorder(tab, lens, par, stream=s)
    assert machine.launches[-1][0] == 9 and tuple(out.shape) == (4, 3) and (out.data_ptr(), 0) in machine.recorded
    c.attend(q, tab, lens, window=5, sinks=2 ** 40)
    assert machine.launches[-1][2][2]._obj.sinks == 2 ** 31 - 1


# ---- the plain implementations ----
def test_reference_selection_by_hand():
    z = torch.log(torch.tensor([[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]))
    got = beam_ref.select(z, torch.tensor([[math.log(0.5), math.log(0.4)]]), 4)[0]
    assert [x[1:] for x in got] == [(1, 1), (0, 0), (0, 1), (0, 2)]
    assert [round(math.exp(x[0]), 5) for x in got] == [0.32, 0.25, 0.125, 0.125]
    fin = torch.tensor([[False, True]])
    got = beam_ref.select(z, torch.tensor([[math.log(0.5), math.log(0.4)]]), 9, fin, end=2)[0]
    assert [x[1:] for x in got] == [(1, 2), (0, 0), (0, 1), (0, 2)]
    assert beam_ref.select(z, torch.full((1, 2), -math.inf), 3) == [[]]


def test_reference_reordering_by_hand():
    table = [[0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11]]
    # 40 tokens of pages of 32: page 0 is full, page 1 being filled, page 2 for later
    new, copies = beam_ref.reorder(table, [40] * 4, [[2, 2, 2, 0]], 32)
    # row 2 keeps its page, row 3 goes on with row 0's; the pages of rows 1 and 3 are free for rows 0 and 1
    assert new == [[6, 4, 2], [6, 10, 5], [6, 7, 8], [0, 1, 11]]
    assert copies == [(7, 4, 8), (7, 10, 8)]
    new, copies = beam_ref.reorder(table, [64] * 4, [[3, 3, -1, 0]], 32)
    assert new == [[9, 10, 2], [9, 10, 5], [6, 7, 8], [0, 1, 11]] and copies == []


# ---- the ring with four warps ----
@pytest.mark.parametrize("length", [3, 4, 5, 7, 10, 22, 32])
def test_ring_of_four_warps(monkeypatch, length):
    """The launch of sequences behind a shared prefix: CTAs of four consumer warps, shorter rings."""
    monkeypatch.setattr(ring_model, "WARPS", 4)
    rng = random.Random(length)
    for full, side in ((1, 1), (2, 1), (2, 2), (4, 1), (4, 2), (4, 4)):
        for kind in ("loaded", "prompt", "window", "bad"):
            for softmax in (0, 6):
                assert ring_model.Ring(length, full, ring_model.ranges_of(kind, side, rng), softmax, True, rng).run(), (full, side, kind)


# ---- the pipeline of the tiles of 128 rows (csrc/prefix.cu) ----
class Pipeline:
    """Its roles as they wait for one another: producer, warps that expand K and V, the thread that issues products, two streams
    of softmax warps (four each, which arrive one by one).  Products complete in their order, at any time."""

    def __init__(self, ring, segments, rng):
        B = ring_model.Barrier
        self.ring, self.segments, self.rng = ring, segments, rng
        self.full, self.empty = [B(1) for _ in range(ring)], [B(8) for _ in range(ring)]
        two = lambda n: [B(n), B(n)]  # noqa: E731
        self.s_ready, self.s_done, self.o_ready, self.o_done = two(8), two(1), two(8), two(1)
        self.q_full, self.q_empty = B(4), B(1)
        self.raw, self.k, self.v, self.s, self.p = [None] * ring, [None] * 2, [None] * 2, [None] * 2, [None] * 2
        self.o = [[], []]        # pages in a stream's accumulator
        self.queue = []          # products issued: functions, done in order
        self.q = None
        self.at_bar = [0] * 8

    def wait(self, bar, parity):
        while not bar.done(parity):
            yield False

    def produce(self):
        for n in range(sum(self.segments)):
            slot, turn = n % self.ring, n // self.ring
            if turn:
                yield from self.wait(self.empty[slot], (turn & 1) ^ 1)
            self.raw[slot] = n
            self.full[slot].arrive()
            yield True

    def expand(self, values):
        ready, done, tile = (self.o_ready, self.o_done, self.v) if values else (self.s_ready, self.s_done, self.k)
        for n in range(sum(self.segments)):
            x, slot = n & 1, n % self.ring
            yield from self.wait(self.full[slot], n // self.ring & 1)
            assert self.raw[slot] == n
            yield True
            if n > 1:
                yield from self.wait(done[x], (n >> 1 & 1) ^ 1)
            tile[x] = n
            yield True
            for _ in range(4):
                ready[x].arrive()
                self.empty[slot].arrive()
                yield True

    def products(self):
        n = 0
        for seg, count in enumerate(self.segments):
            yield from self.wait(self.q_full, seg & 1)
            for i in range(count + 2):
                if i < count:
                    k, x = n + i, n + i & 1
                    yield from self.wait(self.s_ready[x], k >> 1 & 1)

                    def scores(k=k, x=x, seg=seg):
                        assert self.k[x] == k and self.q == seg
                        self.s[x] = k
                        self.s_done[x].arrive()
                    self.queue.append(scores)
                    yield True
                if i + 1 == count:
                    self.queue.append(self.q_empty.arrive)
                    yield True
                if i > 1:
                    k, x = n + i - 2, n + i & 1
                    yield from self.wait(self.o_ready[x], k >> 1 & 1)

                    def outputs(k=k, x=x, first=i < 4):
                        assert self.v[x] == k and self.p[x] == k
                        self.o[x] = [k] if first else self.o[x] + [k]
                        self.o_done[x].arrive()
                    self.queue.append(outputs)
                    yield True
            n += count

    def softmax(self, x, warp):
        n = 0
        self.s_ready[x].arrive()
        yield True
        for seg, count in enumerate(self.segments):
            if x == 0:
                if seg:
                    yield from self.wait(self.q_empty, (seg - 1) & 1)
                self.q = seg
                yield True
                self.q_full.arrive()
                yield True
            yield from self.wait(self.q_full, seg & 1)
            last, mine = -1, []
            for k in range(n + ((n ^ x) & 1), n + count, 2):
                yield from self.wait(self.s_done[x], k >> 1 & 1)
                assert self.s[x] == k
                yield True
                assert self.s[x] == k
                self.s_ready[x].arrive()
                yield True
                if last >= 0:
                    yield from self.wait(self.o_done[x], last >> 1 & 1)
                self.p[x] = k
                yield True
                self.o_ready[x].arrive()
                yield True
                last = k
                mine.append(k)
            if last >= 0:
                yield from self.wait(self.o_done[x], last >> 1 & 1)
                assert self.o[x] == mine
            me = x * 4 + warp
            self.at_bar[me] += 1
            yield True
            while min(self.at_bar) < self.at_bar[me]:  # the streams join their parts
                yield False
            n += count

    def run(self):
        actors = [self.produce(), self.expand(False), self.expand(True), self.products()]
        actors += [self.softmax(x, w) for x in (0, 1) for w in range(4)]
        idle = set()
        while actors:
            i = self.rng.randrange(len(actors) + (len(self.queue) > 0))
            if i == len(actors):
                self.queue.pop(0)()
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
            if actors and not self.queue and len(idle) == len(actors):
                return False
        return True


@pytest.mark.parametrize("ring", [2, 3, 7, 32])
def test_pipeline_comes_to_the_end_with_the_right_pages(ring):
    for seed in range(30):
        rng = random.Random(seed * 40 + ring)
        segments = [rng.choice((1, 1, 2, 3, 4, 5, 9, 16)) for _ in range(rng.randrange(1, 6))]
        assert Pipeline(ring, segments, rng).run(), segments
    for segments in itertools.product((1, 2, 3), repeat=3):
        assert Pipeline(ring, list(segments), random.Random(1)).run(), segments
