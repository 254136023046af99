"""Beam selection, reordering of beams' states, attention with sinks and over shared prefixes, on the GPU against plain
64-bit implementations (``serve_ref``, ``beam_ref``).

Tolerances, from the arithmetic:
* beams and tokens: none where totals are further apart than their error; scores: fp32's half step 2^-24 |total|, and 2^-27
  for the sum of exponentials;
* reorder: none;
* attention: as for the cache's attention without them (``test_gpu_serve``).  A shared prefix adds a merge of two parts, whose
  fp32 rounding (2^-22 relative) lies within delta.  Where a group's rows go through tiles of 128, a weight 2^(s + log2 scale)
  is f16 relative to 2^-7 of a reference that is 2^8 below the row's largest at most: 2^-11 of itself or 2^-32 of the largest
  such product with a code of up to 448, and a page's scale is at most 2^-7 of its largest value: 2^-30 max|v| a token in the
  place of 2^-39.
"""
import math
import random

import pytest
import torch

import beam_ref
import serve_ref as ref
from persistent_megakernel_decode_gb300 import kvcache
from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_serve import DEV, both, check_attend, codes, deal, fill, gen, i32, table_of

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


# ---- selection ----
def check_select(logits, scores, num, finished=None, end=0, got=None):
    """Against the definition; totals nearer than 2^-26 of each other may change places (none of the inputs has such)."""
    got = got or rt.beam_select(logits.to(DEV), scores.to(DEV), num, None if finished is None else finished.to(DEV), end)
    s, p, t = (x.cpu() for x in got)
    for b, want in enumerate(beam_ref.select(logits, scores, num, finished, end)):
        k = len(want)
        assert p[b].tolist() == [x[1] for x in want] + [-1] * (num - k), b
        assert t[b].tolist() == [x[2] for x in want] + [-1] * (num - k), b
        w = torch.tensor([x[0] for x in want], dtype=torch.float64)
        assert ((s[b, :k].double() - w).abs() <= 2.0 ** -24 * w.abs() + 2.0 ** -27).all(), (s[b, :k], w)
        assert (s[b, k:] == -math.inf).all()


def logits_of(rows, v, seed, spread=3.0, dtype=torch.float32):
    return (torch.randn(rows, v, generator=torch.Generator().manual_seed(seed)) * spread).to(dtype)


def scores_of(b, w, seed):
    g = torch.Generator().manual_seed(seed)
    return -30 * torch.rand(b, 1, generator=g) - torch.rand(b, w, generator=g).cumsum(1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b, w, v, num", [(1, 1, 1, 1), (1, 2, 1, 4), (2, 3, 5, 8), (3, 4, 63, 4), (1, 64, 700, 128),
                                          (2, 5, 1023, 10), (1, 4, 1025, 8), (5, 3, 4099, 6), (3, 8, 32003, 16),
                                          (9, 8, 9001, 8), (2, 16, 65536, 32), (1, 2, 262147, 4), (1, 1, 622592, 3)])
def test_select_against_definition(b, w, v, num, dtype):
    z = logits_of(b * w, v, seed=v + w, dtype=dtype)
    check_select(z, scores_of(b, w, seed=num), num)


def test_select_rows_apart_and_unaligned():
    """Row strides, rows that begin off a 16-byte boundary, scores and flags with strides."""
    for dtype in (torch.float32, torch.bfloat16):
        for off in range(9):
            store = logits_of(6, 1300, seed=off, dtype=dtype)
            z = store[:, off: off + 1201 + off]
            sc = scores_of(2, 6, seed=off)[:, ::2]
            fin = torch.zeros(2, 6, dtype=torch.bool)
            fin[1, 2] = True
            fin = fin[:, ::2]
            got = rt.beam_select(store.to(DEV)[:, off: off + 1201 + off], torch.zeros(2, 6, device=DEV).copy_(
                scores_of(2, 6, seed=off))[:, ::2], 5, fin.to(DEV), 7)
            check_select(z, sc, 5, fin, 7, got)


@pytest.mark.parametrize("v", [40, 2000, 33000])
def test_select_ties_go_to_the_lowest_index(v):
    """Rows of one value, of few values, zeros of both signs, equal rows of equal scores."""
    sc = torch.tensor([[-1.0, -1.0, -1.5]])
    z = torch.zeros(3, v)
    check_select(z, sc, 7)
    z[:, ::2] = -0.0
    check_select(z, sc, 7)
    z = torch.randint(0, 3, (3, v), generator=torch.Generator().manual_seed(v)).float()
    z[1] = z[0]
    check_select(z, sc, 20)
    z[0, v // 2] = 9.0  # one above many ties
    z[1] = z[0]
    check_select(z, sc, 30)
    z = logits_of(3, v, seed=1)
    z[1] = z[0]
    z[2] = z[0]
    check_select(z, sc, 12)
    z[:, 5::7] = z.max()  # most threads hold the largest
    check_select(z, sc, 64)


def test_select_all_large_values_in_one_threads_places():
    """Logits far above the rest where one thread or one CTA has them all."""
    v = 40000
    for place in (slice(0, 4), slice(100, 104), slice(2048, 2300), slice(v - 9, v), slice(0, v, 2048)):
        z = logits_of(2, v, seed=3)
        z[:, place] += 40 + torch.rand(z[:, place].shape, generator=torch.Generator().manual_seed(4))
        check_select(z, scores_of(1, 2, seed=8), 64)


@pytest.mark.parametrize("num", [4, 128])
def test_select_rising_logits_and_few_places(num):
    """Each piece of a row above the one before; all large logits in a few threads' places, piece after piece."""
    v = 70001
    z = logits_of(4, v, seed=21, spread=0.3)
    z[0] += torch.arange(v) * 1e-3
    z[1] -= torch.arange(v) * 1e-3
    z[2] += torch.floor(torch.arange(v) / 4096) * 3
    z[3] += 30 * ((torch.arange(v) // 4 % 256) < 9)
    check_select(z, scores_of(1, 4, seed=1), num)
    check_select(z.to(torch.bfloat16), scores_of(2, 2, seed=2), num)


def test_select_values_that_are_not_finite():
    z = logits_of(8, 1111, seed=9)
    z[0, ::3] = math.nan
    z[1] = -math.inf
    z[2] = math.nan
    z[3, 5:] = -math.inf
    z[4, [7, 900]] = math.inf
    z[5] = math.inf
    z[6, :] = -3e38
    z[7, 3] = 3e38
    sc = scores_of(2, 4, seed=2)
    check_select(z, sc, 9)
    check_select(z, sc, 128)  # more than there are finite candidates in some rows
    for bad in (-math.inf, math.inf, math.nan):
        sc[0, 1] = sc[1, 3] = bad
        check_select(z, sc, 9)
    check_select(z, torch.full((2, 4), -math.inf), 5)  # nothing at all
    check_select(z[:4], torch.tensor([[-0.5, -math.inf, -math.inf, -math.inf]]), 4)  # a first step


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 300.0, 1e6, 1e30])
def test_select_logits_of_all_magnitudes(scale):
    check_select(logits_of(6, 3001, seed=11) * scale, scores_of(2, 3, seed=5), 6)


@pytest.mark.parametrize("offset", [1e4, -9e4, 99999.0, -3e5])
def test_select_logits_far_from_zero(offset):
    check_select(logits_of(4, 5003, seed=12) + offset, scores_of(1, 4, seed=6), 8)


def test_select_finished_beams():
    z, sc = logits_of(8, 500, seed=13), torch.tensor([[-1.0, -1.0, -2.0, -50.0], [-3.0, -9.0, -1.0, -2.0]])
    fin = torch.tensor([[False, True, True, True], [True, True, True, True]])
    for end in (0, 2, 499):
        check_select(z, sc, 4, fin, end)
    z[1] = math.nan  # a finished beam's logits are not looked at
    check_select(z, sc, 8, fin, 3)


def test_select_sum_of_exponentials_is_good_to_a_few_2_28():
    """Two beams whose totals differ by less than fp32 shows: their order follows the 64-bit sums."""
    wrong = 0
    for seed in range(40):
        z = logits_of(2, 30011, seed=100 + seed, spread=0.5 + seed % 5)
        lse = [float(torch.logsumexp(z[i].double(), 0)) for i in range(2)]
        first = [float(z[i].double().max()) - lse[i] for i in range(2)]
        # the second beam's score such that its best total is nearly the first's: fp32 scores near 0 are fine enough
        gap = torch.tensor([[0.0, first[0] - first[1]]]).float()
        total = [first[0], float(gap[0, 1].double()) + first[1]]
        if abs(total[0] - total[1]) < 2.0 ** -28:
            continue
        p = rt.beam_select(z.to(DEV), gap.to(DEV), 1)[1].item()
        wrong += p != (1 if total[1] > total[0] else 0)
    assert wrong == 0


@pytest.mark.parametrize("w, v, num", [(8, 40000, 128), (64, 300, 128), (8, 151936, 16), (2, 9000, 100)])
@pytest.mark.parametrize("step", [0.0, 2.0 ** -21])
def test_select_beams_that_are_almost_equal(w, v, num, step):
    """The same logits after every beam, scores equal or an fp32 step at 4 to 8 apart: totals that fp32 would not tell apart."""
    z = logits_of(1, v, seed=v).expand(w, v).contiguous()
    check_select(z, -5 - step * torch.arange(w, dtype=torch.float32)[None], num)


def test_select_totals_beyond_fp32():
    """Differences of logits that overflow fp32: in order, and -inf only as their rounded score."""
    z = torch.tensor([[3e38, -3e38, 0.0, -2e38], [1.0, 1.0, -3e38, 2.0]])
    s, p, t = (x.cpu() for x in rt.beam_select(z.to(DEV), torch.tensor([[-1.0, -2.0]], device=DEV), 8))
    assert p.tolist() == [[0, 1, 1, 1, 0, 1, 0, 0]] and t.tolist() == [[0, 3, 0, 1, 2, 2, 3, 1]]
    assert s[0, 0] == -1 and s[0, 4] == s[0, 5] == torch.tensor(-3e38) and s[0, 6] == s[0, 7] == -math.inf


def test_select_nothing_to_do():
    out = rt.beam_select(torch.zeros(0, 10, device=DEV), torch.zeros(0, 4, device=DEV), 4)
    assert [tuple(x.shape) for x in out] == [(0, 4)] * 3


# ---- reorder ----
def state(L, N, H, P, D, seed):
    """A cache of random codes (NaN codes among them) and scales."""
    g = torch.Generator().manual_seed(seed)
    c = kvcache.Kv8Cache.empty(L, N, H, D, P, DEV)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(2.0 ** torch.randint(-9, 3, t.shape, generator=g))
    return c


def check_reorder(c, table, lens, parents, P, **kw):
    before = [t.view(torch.uint8).cpu().clone() for t in (c.k, c.v)]
    scales = [t.cpu().clone() for t in (c.k_scale, c.v_scale)]
    got = c.reorder(i32(table), i32(lens), i32(parents), **kw)
    want, copies = beam_ref.reorder(table, lens, parents, P)
    assert got.cpu().tolist() == want
    for src, dst, n in copies:
        before[0][:, dst, :, :n] = before[0][:, src, :, :n]
        before[1][:, dst, :, :, :n] = before[1][:, src, :, :, :n]
        for s in scales:
            s[:, dst] = s[:, src]
    for t, w in zip((c.k, c.v), before):
        assert torch.equal(t.view(torch.uint8).cpu(), w)
    for t, w in zip((c.k_scale, c.v_scale), scales):
        assert torch.equal(t.cpu(), w)
    c.check()
    return want


@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("L, H, w", [(1, 1, 1), (2, 3, 4), (3, 2, 7), (1, 2, 64)])
def test_reorder_against_definition(P, D, L, H, w):
    rng = random.Random(P + D + w)
    for n in (0, 1, 15, 16, 17, P - 1, P, P + 1, 2 * P + 31):
        B = 3
        lens = [x for x in (n, max(0, n - 1), 2 * P) for _ in range(w)]
        width = -(-max(lens) // P) + 1
        N = B * w * width + 2
        ids = rng.sample(range(N), B * w * width)
        table = [ids[i * width: (i + 1) * width] for i in range(B * w)]
        parents = [[rng.randrange(w) for _ in range(w)], [rng.choice((0, w - 1, -1)) for _ in range(w)], list(range(w))[::-1]]
        c = state(L, N, H, P, D, seed=n)
        check_reorder(c, table, lens, parents, P)


def test_reorder_again_and_again():
    """Several steps: full pages become common, the beams' pages being filled stay their own."""
    rng, P, w = random.Random(4), 32, 6
    width = 4
    c = state(2, 60, 2, P, 64, seed=1)
    table = [list(range(i * width, (i + 1) * width)) for i in range(w)]
    for n in range(1, 3 * P + 2, 5):
        table = check_reorder(c, table, [n] * w, [[rng.randrange(w) for _ in range(w)]], P)
        rows = [r[n // P:] for r in table]
        assert len({x for r in rows for x in r}) == sum(map(len, rows))  # no page from there on is in two rows


def test_reorder_checks():
    P, w = 32, 3
    table = [[0, 1], [2, 3], [4, 5], [6, 7], [8, 9], [10, 11]]
    good = [[0, 0, 0], [2, 1, 2]]
    for lens, parents in (([40, 40, 41, 40, 40, 40], good), ([-1] * 3 + [40] * 3, good), ([65] * 3 + [40] * 3, good),
                          ([40] * 6, [[0, 3, 0], good[1]]), ([40] * 6, [[0, -2, 0], good[1]])):
        c = state(1, 12, 2, P, 64, seed=2)
        before = c.k.view(torch.uint8).cpu().clone()
        got = c.reorder(i32(table), i32(lens), i32(parents)).cpu().tolist()
        assert got[:3] == table[:3]  # that prompt stays as it is
        want, copies = beam_ref.reorder(table, [40] * 6, [[0, 1, 2], good[1]], P)
        assert got[3:] == want[3:]
        for src, dst, n in copies:
            before[:, dst, :, :n] = before[:, src, :, :n]
        assert torch.equal(c.k.view(torch.uint8).cpu(), before)
        with pytest.raises(rt.MkError):
            c.check()
    # pages out of range: named, but not copied
    c = state(1, 12, 2, P, 64, seed=3)
    before = c.k.view(torch.uint8).cpu().clone()
    bad = [[0, 1], [2, 99], [4, 5]]
    got = c.reorder(i32(bad), i32([40] * 3), i32([[0, 0, 0]])).cpu().tolist()
    assert got == beam_ref.reorder(bad, [40] * 3, [[0, 0, 0]], P)[0]
    before[:, 5, :, :8] = before[:, 1, :, :8]
    assert torch.equal(c.k.view(torch.uint8).cpu(), before)
    with pytest.raises(rt.MkError, match="page 99"):
        c.check()
    out = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    assert c.reorder(i32(table[:3]), i32([32] * 3), i32([[1, 1, -1]]), out=out) is out
    assert out.cpu().tolist() == [[2, 1], [2, 3], [4, 5]]
    c.check()


# ---- attention with sinks ----
@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("hq, hkv, T", [(4, 2, 1), (6, 2, 3), (8, 1, 11), (3, 3, 1)])
@pytest.mark.parametrize("window, sinks", [(1, 1), (7, 4), (40, 33), (64, 64), (5, 200), (300, 1), (33, 0)])
def test_sinks_against_definition(P, D, hq, hkv, T, window, sinks):
    lens = [T, 5 * P + 3, 2 * P, P - 1 + T, 9 * P + 17]
    c, r = both(2, 40, hkv, P, D, poison=True)
    pages = deal(lens, P, 40, random.Random(window + sinks))
    fill(c, r, pages, lens, seed=T, layers=2)
    q = [gen(T, hq, D, seed=50 + b, scale=2.0) for b in range(len(lens))]
    got = c.attend(torch.stack(q).to(DEV), table_of(pages), i32(lens), layer=1, window=window, sinks=sinks)
    c.check()
    check_sinks(r, got, q, pages, lens, 1, window, sinks)


def check_sinks(r, got, q, pages, lens, layer, window, sinks):
    """The first, the middle and the last query: the tokens that one sees as a sequence of their own, without a window."""
    for b, x in enumerate(q):
        T, P = x.shape[0], r.P
        for i in sorted({0, T // 2, T - 1}):
            pos = lens[b] - T + i
            seen = [j for j in range(pos + 1) if j > pos - window or j < sinks] if pos >= 0 else []
            sub = ref.RefCache(1, max(1, -(-len(seen) // P)), r.code["k"].shape[2], P, x.shape[-1])
            for n in "kv":
                sub.scale[n].fill_(1.0)
                for y, j in enumerate(seen):
                    sub.code[n][0, y // P, :, y % P] = r.token(n, layer, pages[b], j)
            check_attend(sub, ([got[0][b, i: i + 1]], [got[1][b, i: i + 1]]), [x[i: i + 1]], [list(range(-(-len(seen) // P)))],
                         [len(seen)], 0, 0)


def test_sinks_packed_rows_and_empty_sequences():
    P, D = 32, 64
    counts, lens = [0, 3, 1, 5, 0, 2], [0, 3, 150, 201, 90, 0]
    start = [sum(counts[:i]) for i in range(len(counts) + 1)]
    c, r = both(1, 40, 2, P, D)
    pages = deal(lens, P, 40, random.Random(3))
    fill(c, r, pages, lens, seed=1, layers=1)
    q = gen(start[-1], 4, D, seed=2)
    out, lse = c.attend(q.to(DEV), table_of(pages), i32(lens), q_start=i32(start), max_tokens=5, window=20, sinks=35)
    c.check()
    for b, n in enumerate(counts):
        if n:
            part = slice(start[b], start[b + 1])
            check_sinks(r, (out[None, part], lse[None, part]), [q[part]], [pages[b]], [lens[b]], 0, 20, 35)


def test_sinks_see_nan_only_where_they_are_seen():
    """NaN codes between the sinks and the window, and in the sinks' page behind them, reach no query."""
    P, D, T = 32, 64, 2
    n, window, sinks = 6 * P + 5, 40, 5
    c, r = both(1, 12, 1, P, D)
    pages = deal([n], P, 12, random.Random(1))
    fill(c, r, pages, [n], seed=1, layers=1)
    q = gen(1, T, 3, D, seed=4)
    want = c.attend(q.to(DEV), table_of(pages), i32([n]), window=window, sinks=sinks)
    k, v = c.k.view(torch.uint8), c.v.view(torch.uint8)
    for j in range(sinks, n - T - window + 1):
        k[0, pages[0][j // P], 0, j % P] = 0x7F
        v[0, pages[0][j // P], 0, :, j % P] = 0xFF
    got = c.attend(q.to(DEV), table_of(pages), i32([n]), window=window, sinks=sinks)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    v[0, pages[0][0], 0, 3, 2] = 0x7F  # a sink's value
    got = c.attend(q.to(DEV), table_of(pages), i32([n]), window=window, sinks=sinks)[0]
    assert torch.isnan(got[..., 3]).all() and not torch.isnan(got[..., :3]).any()


def test_sinks_without_a_window_or_hole_change_nothing():
    P, D = 64, 128
    lens = [500, 130, 64]
    c, r = both(1, 20, 2, P, D)
    pages = deal(lens, P, 20, random.Random(2))
    fill(c, r, pages, lens, seed=1, layers=1)
    q = gen(3, 1, 8, D, seed=4).to(DEV)
    ask = lambda **kw: c.attend(q, table_of(pages), i32(lens), **kw)  # noqa: E731
    for a, b in ((ask(), ask(sinks=3)), (ask(), ask(window=100, sinks=500)), (ask(), ask(window=500, sinks=2 ** 31 - 1)),
                 (ask(window=90), ask(window=90, sinks=0))):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---- attention over shared prefixes ----
def shared_table(rng, N, P, prefix, lens, first):
    """Pages of sequences that share prefix[g] tokens' full pages, from a shuffled pool."""
    ids, pages = rng.sample(range(N), N), []
    groups = [range(a, b) for a, b in zip(first, first[1:])]
    head = {}
    for g, seqs in enumerate(groups):
        full = prefix[g] // P
        mine = [ids.pop() for _ in range(full)]
        for b in seqs:
            head[b] = mine
    for b, n in enumerate(lens):
        have = head.get(b, [])[: -(-n // P)]
        pages.append(have + [ids.pop() for _ in range(-(-n // P) - len(have))])
    return pages


def shared_case(P, D, hq, hkv, first, prefix, lens, seed, N=400, poison=True):
    rng = random.Random(seed)
    c, r = both(1, N, hkv, P, D, poison=poison)
    pages = shared_table(rng, N, P, prefix, lens, first)
    # every page is stored once: sequence by sequence, the shared ones by their first
    done = set()
    for b, n in enumerate(lens):
        lo = 0
        while (lo // P) < len(pages[b]) and pages[b][lo // P] in done:
            lo += P
        if lo >= n:
            continue
        kv = {x: gen(1, 1, n - lo, hkv, D, seed=seed + 10 * b + i, scale=1.0 + i) for i, x in enumerate("kv")}
        c.store(kv["k"].to(DEV), kv["v"].to(DEV), table_of([pages[b]]), i32([lo]), i32([n - lo]))
        for x in "kv":
            r.store(x, kv[x][:, 0], pages[b], lo)
        done.update(pages[b])
    return c, r, pages


# How a call is done goes by its size: each sequence by itself; groups of few rows; groups in tiles of 128 rows.  Planned for
# few SMs, small calls are large ones; q heads make rows.
FORMS = {"alone": (0, 1), "groups": (3, 1), "tiles": (5, 12)}


def formed(c, form):
    c.num_sms = FORMS[form][0]
    return FORMS[form][1]


@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("hq, hkv, T", [(4, 2, 1), (6, 2, 3), (8, 1, 1)])
@pytest.mark.parametrize("form", FORMS)
def test_shared_against_definition(P, D, hq, hkv, T, form):
    first, prefix = [0, 3, 4, 9], [3 * P + 5, 2 * P, 5 * P]
    lens = [3 * P + 5 + T, 3 * P + 9 + T, 5 * P + 1, 2 * P + T, *[5 * P + x + T for x in (0, 1, P, 3, 2 * P)], 40]
    c, r, pages = shared_case(P, D, hq, hkv, first, prefix, lens, seed=P + T)
    hq *= formed(c, form)
    q = [gen(T, hq, D, seed=70 + b, scale=2.0) for b in range(len(lens))]
    got = c.attend_shared(torch.stack(q).to(DEV), table_of(pages), i32(lens), i32(first), i32(prefix))
    c.check()
    check_attend(r, got, q, pages, lens, 0, 0)


@pytest.mark.parametrize("members, T, hq", [(2, 1, 8), (20, 1, 8), (40, 2, 6), (70, 1, 16), (33, 5, 4)])
def test_shared_groups_of_many_rows(members, T, hq):
    """One group of up to more than 256 rows a kv head, over more pages than CTAs hold at once."""
    P, D, hkv = 64, 128, 2
    prefix = [41 * P]
    lens = [41 * P + T + (7 * b) % 90 for b in range(members)]
    c, r, pages = shared_case(P, D, hq, hkv, [0, members], prefix, lens, seed=members)
    q = [gen(T, hq, D, seed=b, scale=2.0) for b in range(members)]
    got = c.attend_shared(torch.stack(q).to(DEV), table_of(pages), i32(lens), i32([0, members]), i32(prefix))
    c.check()
    some = sorted({0, 1, members // 2, members - 1})
    check_attend(r, ([got[0][b] for b in some], [got[1][b] for b in some]), [q[b] for b in some], [pages[b] for b in some],
                 [lens[b] for b in some], 0, 0)
    plain = c.attend(torch.stack(q).to(DEV), table_of(pages), i32(lens))
    assert ((got[0].double() - plain[0].double()).norm() <= 2.0 ** -8 * plain[0].double().norm())
    assert (got[1] - plain[1]).abs().max() <= 2.0 ** -12


@pytest.mark.parametrize("form", FORMS)
def test_shared_what_counts_of_a_prefix(form):
    """Bounds larger than what every query sees, shorter sequences, members without queries or tokens, groups of one, none."""
    P, D, hq, hkv = 32, 64, 4, 2
    counts = [1, 2, 0, 1, 3, 1, 1, 2, 0]
    lens = [4 * P + 1, 4 * P + 2, 0, 2 * P + 1, 3 * P, 4 * P, 70, 3 * P + 7, 0]
    start = [sum(counts[:i]) for i in range(len(counts) + 1)]
    first = [1, 1, 4, 6, 7, 7]
    c, r, pages = shared_case(P, D, hq, hkv, [1, 4, 6], [2 * P, 3 * P], lens, seed=5)
    hq *= formed(c, form)
    q = gen(start[-1], hq, D, seed=6)
    for shared in ([0, 2 * P, 3 * P, 9999, 5], [7, 2 * P + 1, 3 * P - 1, 0, 0], [0] * 5):
        out, lse = c.attend_shared(q.to(DEV), table_of(pages), i32(lens), i32(first), i32(shared), q_start=i32(start),
                                   max_tokens=3)
        c.check()
        part = [slice(a, b) for a, b in zip(start, start[1:])]
        check_attend(r, ([out[x] for x in part], [lse[x] for x in part]), [q[x] for x in part], pages, lens, 0, 0)
    # whole sequences in common: the last query of one sees no token beyond the prefix, that of another sees fewer
    same = [pages[0], pages[0], pages[0]]
    n = [4 * P + 1, 4 * P, 2 * P + 3]
    x = [gen(2, hq, D, seed=b) for b in range(3)]
    got = c.attend_shared(torch.stack(x).to(DEV), table_of(same), i32(n), i32([0, 3]), i32([4 * P + 1]))
    c.check()
    check_attend(r, got, x, same, n, 0, 0)


@pytest.mark.parametrize("form", FORMS)
def test_shared_checks(form):
    P, D = 32, 64
    lens = [3 * P, 3 * P + 1, 2 * P + 5]
    c, r, pages = shared_case(P, D, 4, 2, [0, 3], [2 * P], lens, seed=7)
    q = [gen(1, 4 * formed(c, form), D, seed=b) for b in range(3)]
    ask = lambda first, shared, n=lens, tab=pages: c.attend_shared(  # noqa: E731
        torch.stack(q).to(DEV), table_of(tab), i32(n), i32(first), i32(shared))
    for first, shared in (([0, 2, 1], [64, 64]), ([-1, 3], [64]), ([0, 4], [64]), ([0, 3], [-1]), ([3, 0], [64])):
        got = ask(first, shared)  # nothing is shared: each sequence by itself
        check_attend(r, got, q, pages, lens, 0, 0)
        with pytest.raises(rt.MkError):
            c.check()
    # a sequence longer than its table row gets nothing, and keeps the others from sharing with it
    got = ask([0, 3], [2 * P], n=[3 * P, 99 * P, 2 * P + 5])
    assert (got[0][1] == 0).all() and (got[1][1] == -math.inf).all()
    check_attend(r, ([got[0][b] for b in (0, 2)], [got[1][b] for b in (0, 2)]), [q[0], q[2]], [pages[0], pages[2]],
                 [lens[0], lens[2]], 0, 0)
    with pytest.raises(rt.MkError):
        c.check()
    # a shared page out of range is masked for all rows of the group
    bad = [[999] + p[1:] for p in pages]
    got = ask([0, 3], [2 * P], tab=bad)
    with pytest.raises(rt.MkError, match="page 999"):
        c.check()
    check_attend(r, got, q, [p[1:] for p in pages], [n - P for n in lens], 0, 0)


@pytest.mark.parametrize("form", FORMS)
def test_shared_results_do_not_depend_on_where_they_are_computed(form):
    """The same bits again, on another stream, with a workspace of one's own full of NaN, and replayed from a graph."""
    P, D = 64, 64
    first, prefix = [0, 5, 11], [9 * P, 20 * P]
    lens = [9 * P + 3 + b for b in range(5)] + [20 * P + 9 * b + 1 for b in range(6)]
    c, r, pages = shared_case(P, D, 8, 2, first, prefix, lens, seed=9)
    hq = 8 * formed(c, form)
    q = torch.stack([gen(1, hq, D, seed=b) for b in range(11)]).to(DEV)
    args = q, table_of(pages), i32(lens), i32(first), i32(prefix)
    want = c.attend_shared(*args)
    again = c.attend_shared(*args)
    ws = torch.full((c.attend_shared_workspace(11, hq, 2),), 0xFF, dtype=torch.uint8, device=DEV)
    own = c.attend_shared(*args, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = c.attend_shared(*args, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = c.attend_shared(*args)
    for _ in range(3):
        kept[0].fill_(7)
        graph.replay()
    torch.cuda.synchronize()
    for got in (again, own, other, kept):
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    c.check()


def by_hand(L, N, H, P, D, seed):
    """A cache of random codes without NaN and its 64-bit counterpart, scales 2^-7."""
    c, r = both(L, N, H, P, D)
    g = torch.Generator().manual_seed(seed)
    for n in "kv":
        t = getattr(c, n).view(torch.uint8)
        x = torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8)
        t.copy_(torch.where((x & 127) == 127, x & 128, x))
        getattr(c, n + "_scale").fill_(2.0 ** -7)
    return c, r


def copied(c, r):
    """The counterpart, brought up to what the cache holds."""
    for n in "kv":
        r.code[n] = codes(c, n)
        r.scale[n] = getattr(c, n + "_scale").double().cpu()


@pytest.mark.parametrize("P, D", [(32, 64), (64, 128)])
@pytest.mark.parametrize("form", FORMS)
def test_shared_pages_of_very_different_scales_and_scores(P, D, form):
    """Scores that rise by hundreds from page to page, V scales from 2^-100 to 2^60, pages of zeros (scale 0)."""
    T, members, n = 1, 5, 7
    c, r = by_hand(1, 40, 1, P, D, seed=3)
    hq = 4 * formed(c, form)
    head = list(range(3, 3 + n))
    pages = [head + [20 + b] for b in range(members)]
    lens = [n * P + 5 + b for b in range(members)]
    q = [gen(T, hq, D, seed=b, scale=0.2) for b in range(members)]

    def check(extra=0.0):
        copied(c, r)
        got = c.attend_shared(torch.stack(q).to(DEV), table_of(pages), i32(lens), i32([0, members]), i32([n * P]))
        c.check()
        for b in range(members):
            want, lse = r.attend(q[b], 0, pages[b], lens[b])
            k = torch.stack([r.token("k", 0, pages[b], j) for j in range(lens[b])])
            v = torch.stack([r.token("v", 0, pages[b], j) for j in range(lens[b])])
            # the largest product of a weight and a value of each row bounds what the f16 weights round away
            p = torch.exp(torch.einsum("thd,jhd->thj", q[b].double(), k.expand(-1, hq, -1)) * D ** -0.5 - lse[..., None])
            most = (p * v.abs().amax((1, 2))).amax(-1)
            S = D ** 0.5 * q[b].abs().max().item() * k.abs().max().item()
            delta = 2.0 ** -21 * S + 2.0 ** -20
            mag = torch.einsum("thj,jd->thd", p, v[:, 0].abs())
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + delta) * mag + (lens[b] * 2.0 ** -30 * most)[..., None] + 1e-37
            out, far = got[0][b].double().cpu(), got[1][b].double().cpu()
            assert ((out - want).abs() <= tol).all(), (b, ((out - want).abs() / tol).max())
            assert ((far - lse).abs() <= delta + 2.0 ** -21 * lse.abs()).all()

    check()
    for i, e in enumerate((-9, -7, -4, -2, 0, 1, -12)):  # K scales: the largest score moves from page to page, up and down
        c.k_scale[0, head[i]] = 2.0 ** e
    check()
    for order in ((-7, -100, 0, 60, -30, 20, -120), (60, -7, -7, -100, -7, 0, 3)):
        for i, e in enumerate(order):
            c.v_scale[0, head[i]] = 2.0 ** e
        check()
    c.k_scale[0, head] = 2.0 ** -9
    for i, e in enumerate((-110, -3, -110, 0, -5, -60, -110)):
        c.v_scale[0, head[i]] = 2.0 ** e
    check()
    for i in (0, 3):
        c.v.view(torch.uint8)[0, head[i]] = 0
        c.v_scale[0, head[i]] = 0
    check()
    c.k_scale[0, head[2]] = 0  # scores of zero
    check()


@pytest.mark.parametrize("form", FORMS)
def test_shared_nan_reaches_whom_it_should(form):
    """NaN codes and scales in shared pages reach every row of the group and no other; a query with NaN itself alone; rows
    behind the last sequence stay."""
    P, D, members = 32, 64, 4
    first, prefix = [0, members, 2 * members], [4 * P, 3 * P]
    lens = [4 * P + 3 + b for b in range(members)] + [3 * P + 1 + b for b in range(members)]
    c, r, pages = shared_case(P, D, 4, 2, first, prefix, lens, seed=4)
    hq = 4 * formed(c, form)
    q = torch.cat([gen(len(lens), hq, D, seed=1), gen(3, hq, D, seed=2)]).to(DEV)
    start = list(range(len(lens) + 1))

    def ask(x=q):
        out = torch.full((len(lens) + 3, hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((len(lens) + 3, hq), 7.0, device=DEV)
        c.attend_shared(x, table_of(pages), i32(lens), i32(first), i32(prefix), q_start=i32(start), max_tokens=1, out=out, lse=lse)
        c.check()
        assert (out[len(lens):] == 7).all() and (lse[len(lens):] == 7).all()
        return out[:len(lens)], lse[:len(lens)]

    clean = ask()
    half = hq // 2  # q heads of a kv head
    k, v = c.k.view(torch.uint8), c.v.view(torch.uint8)
    page = pages[0][2]
    old = int(v[0, page, 1, 9, 5])
    v[0, page, 1, 9, 5] = 0x7F
    out, lse = ask()
    assert torch.isnan(out[:members, half:, 9]).all() and torch.isnan(out).sum() == members * half
    assert torch.equal(lse, clean[1]) and torch.equal(out[members:], clean[0][members:]) and torch.equal(out[:, :half], clean[0][:, :half])
    v[0, page, 1, 9, 5] = old
    old = int(k[0, page, 0, 3, 7])
    k[0, page, 0, 3, 7] = 0xFF
    out, lse = ask()
    assert torch.isnan(out[:members, :half]).all() and torch.isnan(lse[:members, :half]).all()
    assert torch.equal(out[:, half:], clean[0][:, half:]) and torch.equal(out[members:], clean[0][members:])
    k[0, page, 0, 3, 7] = old
    for name in ("k_scale", "v_scale"):
        t = getattr(c, name)
        keep = float(t[0, page, 1])
        t[0, page, 1] = math.nan
        out, lse = ask()
        assert torch.isnan(out[:members, half:]).all() and not torch.isnan(out[members:]).any()
        if name == "k_scale":
            assert torch.isnan(lse[:members, half:]).all()
        else:  # the sum of such a page may be formed in another way
            assert ((lse - clean[1]).abs() <= 2.0 ** -19 * (1 + clean[1].abs())).all()
        t[0, page, 1] = keep
    for bad in (math.nan, math.inf):
        x = q.clone()
        x[1, 0, 3] = bad
        out, lse = ask(x)
        assert torch.isnan(out[1, 0]).all() and torch.isnan(lse[1, 0])
        assert torch.isnan(out).sum() == D and torch.isnan(lse).sum() == 1


def test_shared_prefix_beyond_32_bit_offsets():
    """Pages whose codes lie more than 2^32 bytes into the cache, through both groups' forms."""
    P, D, hkv = 64, 128, 8
    N = (1 << 32) // (P * D * hkv) + 40
    c = kvcache.Kv8Cache.empty(1, N, hkv, D, P, DEV)
    small, r, pages = shared_case(P, D, 8, hkv, [0, 4], [2 * P], [2 * P + 3, 2 * P + 9, 2 * P + 1, 3 * P], seed=8, N=20)
    used = sorted({x for p in pages for x in p})
    at = {x: N - 1 - i for i, x in enumerate(used)}
    for name in ("k", "v", "k_scale", "v_scale"):
        a, b = getattr(small, name), getattr(c, name)
        a, b = (a.view(torch.uint8), b.view(torch.uint8)) if name in "kv" else (a, b)
        for x in used:
            b[:, at[x]] = a[:, x]
    far = [[at[x] for x in p] for p in pages]
    lens = [2 * P + 3, 2 * P + 9, 2 * P + 1, 3 * P]
    for form in ("groups", "tiles"):
        hq = 8 * formed(c, form)
        q = [gen(1, hq, D, seed=b) for b in range(4)]
        got = c.attend_shared(torch.stack(q).to(DEV), table_of(far), i32(lens), i32([0, 4]), i32([2 * P]))
        c.check()
        check_attend(r, got, q, pages, lens, 0, 0)


def test_shared_batches_as_large_as_they_may_be():
    """512 sequences in 512 groups and in one; 1024 of both is the limit."""
    P, D, B = 32, 64, 512
    c, r = both(1, 40, 1, P, D)
    pages = [[3, 4, 5 + b % 30] for b in range(B)]
    kv = {x: gen(1, 1, 35 * P, 1, D, seed=i) for i, x in enumerate("kv")}
    c.store(kv["k"].to(DEV), kv["v"].to(DEV), table_of([list(range(35))]), i32([0]), i32([35 * P]))
    for x in "kv":
        r.store(x, kv[x][:, 0], list(range(35)), 0)
    lens = [2 * P + 1 + b % P for b in range(B)]
    q = gen(B, 1, 2, D, seed=5)
    want = c.attend(q.to(DEV), table_of(pages), i32(lens))
    for first in (list(range(B + 1)), [0] + [B] * B, [0, B], [0, 100, 100, 300, B]):
        got = c.attend_shared(q.to(DEV), table_of(pages), i32(lens), i32(first), i32([2 * P] * (len(first) - 1)))
        c.check()
        assert ((got[0].double() - want[0].double()).norm() <= 2.0 ** -8 * want[0].double().norm())
        assert (got[1] - want[1]).abs().max() <= 2.0 ** -14
        check_attend(r, ([got[0][7]], [got[1][7]]), [q[7]], [pages[7]], [lens[7]], 0, 0)
    with pytest.raises(rt.MkError):
        c.attend_shared(q.to(DEV), table_of(pages), i32(lens), i32(list(range(B + 2))), i32([0] * (B + 1)))


def test_calls_on_two_streams_and_two_graphs_at_once():
    """Shared attention, selection and reordering, each captured into a graph of its own and replayed beside the other."""
    P, D, W = 64, 64, 8
    first, prefix = [0, W, 2 * W], [10 * P, 12 * P]
    lens = [10 * P + 7] * W + [12 * P + 7] * W
    c, r, pages = shared_case(P, D, 32, 2, first, prefix, lens, seed=2)
    c.num_sms = 20
    table, n = table_of([p + [0] * (14 - len(p)) for p in pages]), i32(lens)
    z, sc = logits_of(2 * W, 9001, seed=4).to(DEV), scores_of(2, W, seed=3).to(DEV)
    par = i32([list(range(W))[::-1], list(range(W))])  # one child each: nothing is copied under the attention
    graphs, outs, want = [], [], []
    for seed in (1, 2):
        q = gen(2 * W, 1, 32, D, seed=seed).to(DEV)
        zz = z + seed
        def work(q=q, zz=zz):
            a = c.attend_shared(q, table, n, i_first, i_prefix)
            return [*a, *rt.beam_select(zz, sc, 2 * W), c.reorder(table, n, par)]
        i_first, i_prefix = i32(first), i32(prefix)
        torch.cuda.synchronize()
        want.append([x.clone() for x in work()])
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(work())
        graphs.append((g, i_first, i_prefix, q, zz))  # (its inputs live as long as the graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        torch.cuda.synchronize()
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(a[:5], b[:5])) and torch.equal(a[5], b[5])
    c.check()


# ---- all together ----
def test_a_beam_search_over_a_shared_prompt():
    """Beams of two prompts over several steps, the model a fixed map from tokens to queries, keys, values and logits: the
    loop on the cache (store, attention over the shared prompt, selection, reordering) against one that keeps every beam's
    tokens and recomputes everything from them."""
    torch.manual_seed(0)
    P, D, hq, hkv, V, W, B, steps = 32, 64, 4, 2, 301, 4, 2, 40
    prompts = [torch.randint(0, V, (n,)).tolist() for n in (70, 45)]
    emb = {n: gen(V, h, D, seed=i, scale=1.5) for i, (n, h) in enumerate((("q", hq), ("k", hkv), ("v", hkv)))}
    head = (torch.randn(hq * D, V, generator=torch.Generator().manual_seed(9)) * 0.2).to(DEV)
    logits_from = lambda out: out.float().reshape(-1, hq * D).to(DEV) @ head  # noqa: E731

    N = 200
    pool, c = kvcache.PagePool(N), kvcache.Kv8Cache.empty(1, N, hkv, D, P, DEV)
    rows, lens = [], []
    for tokens in prompts:
        full, n = len(tokens) // P, len(tokens)
        common = pool.alloc(full)
        for w in range(W):
            if w:
                pool.share(common)
            rows.append(common + pool.alloc(-(-(n + steps) // P) - full))
            lens.append(n)
    table = table_of(rows)
    for b, tokens in enumerate(prompts):  # the prompt's full pages once, its rest for every beam
        n, full = len(tokens), len(tokens) // P * P
        kv = {x: emb[x][tokens].to(DEV)[None, None] for x in "kv"}
        c.store(kv["k"], kv["v"], table[b * W: b * W + 1], i32([0]), i32([n]))
        for w in range(1, W):
            c.store(*(kv[x][:, :, full:].contiguous() for x in "kv"), table[b * W + w: b * W + w + 1], i32([full]), i32([n - full]))
    first, shared = i32([0, W, 2 * W]), i32([len(t) for t in prompts])
    score = torch.full((B, W), -math.inf, device=DEV)
    score[:, 0] = 0
    done = torch.zeros((B, W), dtype=torch.bool, device=DEV)
    lens = i32(lens)
    last = torch.tensor([t[-1] for t in prompts for _ in range(W)])
    histories = [[list(t) for _ in range(W)] for t in prompts]
    alive = [[0.0] + [-math.inf] * (W - 1) for _ in prompts]
    for step in range(steps):
        q = emb["q"][last][:, None].to(DEV)
        out, _ = c.attend_shared(q, table, lens, first, shared)
        z = logits_from(out)
        new, parent, token = rt.beam_select(z, score, finished=done, end=1)
        # the same step from the kept tokens: every beam's attention in 64 bits over its own history
        want = c.attend(q, table, lens)[0]
        assert ((out.double() - want.double()).norm() <= 2.0 ** -7 * want.double().norm())
        for b in range(B):
            for w in range(W):
                if alive[b][w] == -math.inf:
                    continue
                t = histories[b][w]
                stored = [c.k[0, table[b * W + w, j // P], :, j % P].float() * c.k_scale[0, table[b * W + w, j // P]][:, None]
                          for j in (0, len(t) // 2, len(t) - 1)]
                for j, x in zip((0, len(t) // 2, len(t) - 1), stored):
                    y = emb["k"][t[j]].float()
                    assert ((x.cpu() - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -5).all(), (step, b, w, j)
        p, k, s = parent.cpu().tolist(), token.cpu().tolist(), new.cpu().tolist()
        histories = [[histories[b][p[b][w]] + [k[b][w]] for w in range(W)] for b in range(B)]
        alive = s
        done = done.gather(1, parent.long()) | (token == 1)
        score = new
        table = c.reorder(table, lens, parent)
        last = token.cpu().flatten()
        kv = {x: emb[x][last].to(DEV)[None, :, None] for x in "kv"}
        c.store(kv["k"], kv["v"], table, lens, torch.ones_like(lens))
        lens = lens + 1
    c.check()
    assert sorted({x for r in table.cpu().tolist() for x in r if x >= 0} - {x for r in rows for x in r}) == []
