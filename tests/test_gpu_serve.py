"""Serving operators on the GPU against plain 64-bit implementations (``serve_ref``).

Tolerances, from the arithmetic:
* store, load, copy: none (every rounding is defined);
* tokens: none; logprob: 2^-28 for the weights' fixed point (2^-30 each, sums of them), and of itself 6 x 2^-24: it is
  -log1p(a / b), whose relative error is at most a / b's, with two conversions, a quotient (2^-24 each) and log1pf (2^-23);
* attend, out: bf16's half step 2^-8 |out|, plus 2^-11 (a probability's f16 form) + delta, relative to sum_j p_j |v_j|,
  plus 2^-39 max|v| per visible token (f16's least step, 2^-24 / 2^14, halved) -- where delta bounds a score's error: fp32
  sums of products whose magnitudes add to S <= scale D max|q| max|k| (2^-22 S), query elements far below their row's
  largest (f16's least step against 2^14: 2^-39 S, within the same 2^-22 S), and 2^-20 for exp2;
* lse: delta, and fp32's rounding of it and of the running maximum in log2 units, 2^-21 |lse|.
"""
import math
import random

import numpy as np
import pytest
import torch

import serve_ref as ref
from persistent_megakernel_decode_gb300 import kvcache
from persistent_megakernel_decode_gb300 import runtime as rt
from persistent_megakernel_decode_gb300 import synth

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]
DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def both(L, N, H, P, D, poison=False):
    """A Kv8Cache and its 64-bit counterpart; poison: pages full of NaN codes and NaN scales, as freed ones may be."""
    c = kvcache.Kv8Cache.empty(L, N, H, D, P, DEV)
    if poison:
        for t in (c.k, c.v):
            t.view(torch.uint8).fill_(0x7F)
        for t in (c.k_scale, c.v_scale):
            t.fill_(math.nan)
    return c, ref.RefCache(L, N, H, P, D)


def codes(c, name):
    """The cache's codes as fp64 values [L, N, Hkv, P, D]."""
    x = ref.e4m3_values(getattr(c, name).view(torch.uint8).cpu())
    return x.transpose(3, 4) if name == "v" else x


def table_of(pages, width=None):
    width = width or max(1, max(map(len, pages)))
    return i32([p + [-1] * (width - len(p)) for p in pages])


def deal(lens, P, N, rng, extra=0):
    ids = rng.sample(range(N), sum(-(-(n + extra) // P) for n in lens))
    out = []
    for n in lens:
        k = -(-(n + extra) // P)
        out.append(ids[:k])
        ids = ids[k:]
    return out


def gen(*shape, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def fill(c, r, pages, lens, seed, layers):
    """Store lens[b] tokens of every sequence in both."""
    H, D, T = c.kv_heads, c.head_dim, max(max(lens), 1)
    kv = {n: gen(layers, len(lens), T, H, D, seed=seed + i, scale=1.0 + i) for i, n in enumerate("kv")}
    c.store(kv["k"].to(DEV), kv["v"].to(DEV), table_of(pages), i32([0] * len(lens)), i32(lens))
    for n in "kv":
        for b, m in enumerate(lens):
            if m:
                r.store(n, kv[n][:, b, :m], pages[b], 0)
    return kv


def check_attend(r, got, q, pages, lens, layer, window, scale=None):
    """q: list of [T_b, Hq, D] on the CPU; got = (out, lse) lists in the same order."""
    D = q[0].shape[-1]
    sc = D ** -0.5 if scale is None else scale
    for b, x in enumerate(q):
        want, lse = r.attend(x, layer, pages[b], lens[b], window, scale)
        out, far = got[0][b].double().cpu(), got[1][b].double().cpu()
        if not x.numel():
            continue
        if lens[b] == 0:
            assert (out == 0).all() and (far == -math.inf).all()
            continue
        k, v = (torch.stack([r.token(n, layer, pages[b], j) for j in range(lens[b])]) for n in "kv")
        S = sc * D * x.abs().max().item() * k.abs().max().item()
        delta = 2.0 ** -21 * S + 2.0 ** -20
        mag = ref_abs(r, x, layer, pages[b], lens[b], window, scale)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + delta) * mag + lens[b] * 2.0 ** -39 * v.abs().max()
        assert torch.equal(far == -math.inf, lse == -math.inf)
        fin = lse > -math.inf
        assert (out[~fin] == 0).all()
        assert ((out - want).abs() <= tol).all(), (b, ((out - want).abs() / tol).max())
        assert ((far - lse).abs()[fin] <= delta + 2.0 ** -21 * lse.abs()[fin]).all(), (b, (far - lse).abs()[fin].max())


def ref_abs(r, x, layer, pages, n, window, scale):
    """sum_j p_j |v_j|."""
    v = r.code["v"]
    r.code["v"] = v.abs()
    try:
        return r.attend(x, layer, pages, n, window, scale)[0]
    finally:
        r.code["v"] = v


# ---- store and load ----
@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("H, L", [(1, 1), (3, 2)])
def test_store_then_append_then_load(P, D, H, L):
    rng = random.Random(P + D + H)
    lens, more = [0, 1, P - 1, P, P + 1, 3 * P + 5], [1, 2, 1, 1, 2 * P, 0]
    N = 40
    c, r = both(L, N, H, P, D, poison=True)
    pages = deal([a + b for a, b in zip(lens, more)], P, N, rng)
    tab = table_of(pages)
    fill(c, r, pages, lens, 5, L)
    c.check()
    # appended tokens, larger, so that partly filled pages are rounded to a larger scale; three calls
    T = 2 * P
    for step, grow in enumerate((1.0, 40.0, 0.01)):
        kv = {n: gen(L, len(lens), T, H, D, seed=70 + i + 10 * step, scale=grow * (1 + i)) for i, n in enumerate("kv")}
        cnt = more if step == 0 else [min(m, 1) for m in more]
        start = lens if step == 0 else [n + m - min(m, 1) for n, m in zip(lens, more)]  # the last token again
        c.store(kv["k"].to(DEV), kv["v"].to(DEV), tab, i32(start), i32(cnt))
        for n in "kv":
            for b, m in enumerate(cnt):
                if m:
                    r.store(n, kv[n][:, b, :m], pages[b], start[b])
    c.check()
    total = [a + b for a, b in zip(lens, more)]
    for n in "kv":
        got, scale = codes(c, n), getattr(c, n + "_scale").double().cpu()
        for b, t in enumerate(total):
            for j, page in enumerate(pages[b]):
                assert torch.equal(scale[:, page], r.scale[n][:, page])
                m = min(P, t - j * P)
                assert torch.equal(got[:, page, :, :m], r.code[n][:, page, :, :m])
    # load a part back, at a row offset; the rest of the rows stays
    start, cnt, row0 = [n // 3 for n in total], [n - n // 3 for n in total], [b % 3 for b in range(len(total))]
    rows = max(cnt) + 3
    out = {n: torch.full((L, len(lens), H, rows, D), 7.0, dtype=torch.bfloat16, device=DEV) for n in "kv"}
    c.load(out["k"].transpose(2, 3), out["v"].transpose(2, 3), tab, i32(start), i32(cnt), row0=i32(row0))
    c.check()
    for n in "kv":
        want = torch.full((L, len(lens), H, rows, D), 7.0, dtype=torch.bfloat16)
        for b in range(len(lens)):
            for i in range(cnt[b]):
                for l in range(L):
                    want[l, b, :, row0[b] + i] = r.token(n, l, pages[b], start[b] + i).to(torch.bfloat16)
        assert torch.equal(out[n].cpu(), want)


def test_store_opens_pages_clean_and_keeps_special_values():
    c, r = both(1, 4, 1, 32, 64, poison=True)
    x = gen(1, 1, 5, 1, 64, seed=1)
    x[0, 0, 0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 3.0e38, -0.0, 1e-38])
    y = torch.zeros_like(x)
    c.store(x.to(DEV), y.to(DEV), i32([[2]]), i32([0]), i32([5]))
    r.store("k", x[0, 0][None], [2], 0)
    k = codes(c, "k")[0, 2, 0]
    assert torch.equal(k[:5].nan_to_num(nan=1e9), r.code["k"][0, 2, 0, :5].nan_to_num(nan=1e9))
    assert k[0, 0] == 448 and k[0, 1] == -448 and math.isnan(k[0, 2]) and (k[5:] == 0).all()
    assert c.v_scale[0, 2, 0] == 0 and (codes(c, "v")[0, 2] == 0).all()  # all zeros: scale 0
    # the same for the pages that were not touched: as they were
    assert (c.k.view(torch.uint8)[0, [0, 1, 3]] == 0x7F).all() and torch.isnan(c.k_scale[0, [0, 1, 3]]).all()
    # a zero scale gives way to the first real value
    c.store(x.to(DEV), gen(1, 1, 5, 1, 64, seed=2, scale=1e-3).to(DEV), i32([[2]]), i32([5]), i32([1]))
    assert 0 < c.v_scale[0, 2, 0] <= 2.0 ** -14


def test_store_takes_packed_rows_and_fused_strides():
    """Packed ragged tokens, K and V slices of one fused projection."""
    H, D, P, cnt = 2, 64, 32, [3, 0, 40]
    c, r = both(1, 8, H, P, D)
    fused = gen(sum(cnt), 3 * H, D, seed=9)
    k, v = fused[:, H: 2 * H].to(DEV), fused[:, 2 * H:]
    big = fused.to(DEV)
    k, v = big[:, H: 2 * H], big[:, 2 * H:]
    pages = [[5], [], [1, 7]]
    e = lambda x: x[None, None].expand(1, 3, -1, -1, -1)  # noqa: E731
    c.store(e(k), e(v), table_of(pages), i32([0, 0, 0]), i32(cnt), row0=i32([0, 3, 3]), max_count=40)
    c.check()
    for n, x in (("k", k), ("v", v)):
        r.store(n, x[:3].cpu()[None], pages[0], 0)
        r.store(n, x[3:].cpu()[None], pages[2], 0)
        assert torch.equal(codes(c, n), r.code[n])


# ---- attention ----
@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("H, G, T, window", [(1, 1, 1, 0), (2, 4, 1, 0), (2, 8, 1, 40), (1, 3, 5, 0), (2, 4, 9, 33),
                                             (1, 16, 1, 0), (1, 16, 3, 1), (1, 5, 29, 0), (1, 8, 17, 100)])
def test_attend(P, D, H, G, T, window):
    rng = random.Random(P + D + G + T)
    lens = [T, P, P + 1, 2 * P - 1, 0, 333, T + P]
    lens = [max(n, T) if n else 0 for n in lens]
    N = 60
    c, r = both(2, N, H, P, D, poison=True)
    pages = deal(lens, P, N, rng)
    fill(c, r, pages, lens, 20, 2)
    q = gen(len(lens), T, H * G, D, seed=33)
    out, lse = c.attend(q.to(DEV), table_of(pages), i32(lens), layer=1, window=window)
    c.check()
    check_attend(r, (out, lse), q, pages, lens, 1, window)
    again = c.attend(q.to(DEV), table_of(pages), i32(lens), layer=1, window=window)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("P, D, H, G", [(64, 128, 2, 4), (32, 64, 3, 2)])
def test_attend_packed_queries_leave_other_rows(P, D, H, G):
    rng = random.Random(7)
    lens, cnt = [70, 5, 0, 200, 64, 31], [3, 0, 0, 70, 1, 31]
    c, r = both(1, 30, H, P, D, poison=True)
    pages = deal(lens, P, 30, rng)
    fill(c, r, pages, lens, 40, 1)
    total, off = sum(cnt), 2
    qs = [off]
    for n in cnt:
        qs.append(qs[-1] + n)
    rows = total + off + 3  # rows before the first and behind the last sequence
    fused = gen(rows, 3 * H * G, D, seed=3).to(DEV)
    q = fused[:, H * G: 2 * H * G]
    out = torch.full((rows, 2 * H * G, D), 9.0, dtype=torch.bfloat16, device=DEV)[:, :H * G]
    lse = torch.full((rows, H * G), 9.0, device=DEV)
    for most in (None, 1, 70):
        got = c.attend(q, table_of(pages), i32(lens), q_start=i32(qs), max_tokens=most, window=90, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        c.check()
        cut = [slice(qs[b], qs[b + 1]) for b in range(len(cnt))]
        check_attend(r, ([out[s] for s in cut], [lse[s] for s in cut]), [q[s].cpu() for s in cut], pages, lens, 0, 90)
        for t in (out, lse):
            assert (t[:off] == 9).all() and (t[off + total:] == 9).all()


def test_attend_wide_scores_and_zero_scale():
    """Peaked softmax (scores over +-200), a scale of 0 (uniform), query rows of zeros and of very unequal elements."""
    P, D, H, G, lens = 64, 64, 1, 4, [500]
    c, r = both(1, 10, H, P, D)
    pages = deal(lens, P, 10, random.Random(1))
    fill(c, r, pages, lens, 50, 1)
    q = gen(1, 3, G, D, seed=4, scale=20.0)
    q[0, 0, 0] = 0
    q[0, 1, 1, :] *= torch.logspace(0, -6, D).to(torch.bfloat16)
    for scale in (None, 1.0, 0.0):
        got = c.attend(q.to(DEV), table_of(pages), i32(lens), scale=scale)
        check_attend(r, got, q, pages, lens, 0, 0, scale)


def test_attend_nan_only_where_it_is_seen():
    P, D, H, G, T = 32, 64, 2, 2, 6
    lens = [70]
    c, r = both(1, 4, H, P, D, poison=True)
    pages = [[3, 0, 1]]
    kv = {n: gen(1, 1, 70, H, D, seed=60 + i) for i, n in enumerate("kv")}
    kv["v"][0, 0, 67, 1, 5] = math.nan   # V of position 67, kv head 1
    kv["k"][0, 0, 68, 0, 9] = math.nan   # K of position 68, kv head 0
    c.store(kv["k"].to(DEV), kv["v"].to(DEV), table_of(pages), i32([0]), i32(lens))
    q = gen(1, T, H * G, D, seed=61)
    q[0, 2, 1, 3] = math.inf
    out, lse = (x[0].cpu() for x in c.attend(q.to(DEV), table_of(pages), i32(lens)))
    for i in range(T):
        pos = 64 + i
        for h in range(H * G):
            nan = torch.zeros(D, dtype=torch.bool)
            if h // G == 0 and pos >= 68 or (i, h) == (2, 1):
                nan[:] = True
            elif h // G == 1 and pos >= 67:
                nan[5] = True
            assert torch.equal(torch.isnan(out[i, h]), nan), (i, h)
            assert math.isnan(lse[i, h]) == bool(nan.all())


@pytest.mark.parametrize("P, D, G, T", [(32, 64, 2, 1), (64, 128, 4, 12)])
def test_attend_as_many_sequences_as_a_call_takes(P, D, G, T):
    rng = random.Random(T)
    lens = [rng.choice([0, T, T + 1, 45]) for _ in range(1024)]
    c, r = both(1, 2100, 1, P, D)
    pages = deal(lens, P, 2100, rng)
    fill(c, r, pages, lens, 110, 1)
    q = gen(1024, T, G, D, seed=111)
    got = c.attend(q.to(DEV), table_of(pages), i32(lens))
    c.check()
    some = rng.sample(range(1024), 60) + [0, 1023]
    check_attend(r, (got[0][some], got[1][some]), q[some], [pages[b] for b in some], [lens[b] for b in some], 0, 0)
    with pytest.raises(rt.MkError):
        c.attend(gen(1025, 1, G, D, seed=1).to(DEV), i32([[0]] * 1025), i32([1] * 1025))


@pytest.mark.parametrize("P, D, G, T", [(64, 128, 4, 1), (32, 64, 2, 1), (32, 128, 4, 3), (64, 64, 8, 7)])
@pytest.mark.parametrize("sms", [1, 2, 5])
def test_attend_many_pages_per_cta(P, D, G, T, sms):
    """Few CTAs, so that every slot of the page ring is filled many times."""
    lens, H = [2300, 0, 700, 1500], 2
    lens = [max(n, T) if n else 0 for n in lens]
    N = 160
    c, r = both(1, N, H, P, D, poison=True)
    pages = deal(lens, P, N, random.Random(sms))
    fill(c, r, pages, lens, 100, 1)
    q = gen(len(lens), T, H * G, D, seed=101)
    c.num_sms = sms
    got = c.attend(q.to(DEV), table_of(pages), i32(lens))
    c.check()
    check_attend(r, got, q, pages, lens, 0, 0)
    for _ in range(20):  # which page lands first changes; the sums' order does not
        again = c.attend(q.to(DEV), table_of(pages), i32(lens))
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_attend_one_long_sequence_split_over_every_sm():
    P, D, H, G, n = 64, 128, 1, 4, 20011
    c, r = both(1, 320, H, P, D)
    pages = deal([n], P, 320, random.Random(2))
    kv = fill(c, r, pages, [n], 80, 1)
    assert kv["k"].shape[2] == n
    q = gen(1, 1, G, D, seed=5)
    got = c.attend(q.to(DEV), table_of(pages), i32([n]))
    check_attend(r, got, q, pages, [n], 0, 0)


def test_failed_checks_are_recorded_and_harmless():
    P, D, H, G = 32, 64, 1, 2
    lens = [40, 40, 40]
    c, r = both(1, 6, H, P, D)
    pages = [[0, 1], [2, 3], [4, 5]]
    fill(c, r, pages, lens, 90, 1)
    before = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    q = gen(3, 1, G, D, seed=6)

    def expect(seq):
        with pytest.raises(rt.MkError, match=f"sequence {seq} ") as e:
            c.check()
        assert e.value.code == rt.MK_ERR_DEVICE_CHECK
        c.check()  # cleared

    # pages out of range: their tokens count as masked, the other sequences are right
    tab = i32([[0, 1], [2, 6], [4, -7]])
    out, lse = c.attend(q.to(DEV), tab, i32(lens))
    with pytest.raises(rt.MkError):
        c.check()
    check_attend(r, (out[:1], lse[:1]), q[:1], pages[:1], lens[:1], 0, 0)
    want, far = r.attend(q[1], 0, [2], 32)  # sees the first page only
    assert (out[1].cpu().double() - want).abs().max() < 0.05 and (lse[1].cpu() - far).abs().max() < 1e-4
    # lengths beyond the table, negative ones
    for bad in (65, -1):
        out, lse = c.attend(q.to(DEV), table_of(pages), i32([40, bad, 40]))
        expect(1)
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
        check_attend(r, (out[2:], lse[2:]), q[2:], pages[2:], lens[2:], 0, 0)
    # offsets that leave q
    out = torch.full((3, G, D), 9.0, dtype=torch.bfloat16, device=DEV)
    c.attend(q[:, 0].to(DEV), table_of(pages), i32(lens), q_start=i32([0, 1, 2, 4]), out=out)
    expect(2)
    assert (out[2] == 9).all()
    # store and load: nothing moves for the sequences concerned
    x = gen(1, 3, 8, H, D, seed=7).to(DEV)
    y = x.clone()
    for start, count, tab in (([40, 60, 40], [0, 8, 0], table_of(pages)), ([-1, 0, 0], [2, 0, 0], table_of(pages)),
                              ([0, 0, 0], [0, 0, 9], table_of(pages)), ([0, 0, 0], [-1, 0, 0], table_of(pages)),
                              ([0, 0, 0], [4, 0, 0], i32([[6, 1], [2, 3], [4, 5]]))):
        for f in (c.store, c.load):
            f(x, x, tab, i32(start), i32(count))
            with pytest.raises(rt.MkError):
                c.check()
    c.store(x, x, table_of(pages), i32([0, 0, 0]), i32([4, 0, 0]), row0=i32([5, 0, 0]))
    expect(0)
    assert torch.equal(x, y)
    for a, b in zip(before, (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)):
        assert torch.equal(a, b)


# ---- pages ----
@pytest.mark.parametrize("P, D, H, L, n", [(32, 64, 1, 1, 1), (64, 128, 8, 2, 5), (32, 64, 3, 3, 40), (32, 64, 1, 1, 700)])
def test_copy_pages_and_rename(P, D, H, L, n):
    N = 2 * n + 3
    g = torch.Generator(device=DEV).manual_seed(n)
    c = kvcache.Kv8Cache.empty(L, N, H, D, P, DEV)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.rand(t.shape, generator=g, device=DEV))
    rng = random.Random(n)
    ids = rng.sample(range(N), 2 * n)
    src, dst = ids[:n], ids[n:]
    if n == 5:
        src[3] = src[1]  # one page to two places: renamed to the first
    tab = torch.randint(-1, N, (7, 50), generator=g, device=DEV, dtype=torch.int32)
    want = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    for w in want:
        w[:, dst] = w[:, src]
    name = {}
    for s, d in zip(src, dst):
        name.setdefault(s, d)
    renamed = [[name.get(e, e) for e in row] for row in tab.tolist()]
    c.copy_pages(src, dst, table=tab)
    for w, t in zip(want, (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)):
        assert torch.equal(w.view(torch.uint8), t.view(torch.uint8))
    assert tab.tolist() == renamed
    c.copy_pages([], [], table=tab)
    with pytest.raises(rt.MkError):
        c.copy_pages([0], [N])


# ---- sampling ----
def check_sample(z, u, got, settings):
    tokens, logprob = got[0].cpu(), got[1].double().cpu()
    # the settings are fp32 numbers to the call: 0.4 is 0.40000000596, which of 20,000 equal logits keeps not 8,000 but
    # the 8,001 that first sum to at least 8,000.00012
    settings = [{k: v if k == "top_k" else float(np.float32(v)) for k, v in s.items()} for s in settings]
    for b in range(z.shape[0]):
        t, lp = ref.sample_row(z[b], float(u[b]), **settings[b])
        assert int(tokens[b]) == t, (b, settings[b])
        if math.isinf(lp):
            assert logprob[b] == lp
        else:
            assert abs(float(logprob[b]) - lp) <= 6 * 2.0 ** -24 * abs(lp) + 2.0 ** -28, (b, lp, float(logprob[b]))


def settings_of(b, seed):
    rng = random.Random(seed)
    pick = lambda off, f: off if rng.random() < 0.35 else f()  # noqa: E731
    return [dict(temperature=float(np.float32(pick(1.0, lambda: rng.choice([0.0, 0.05, 0.6, 1.7, 30.0])))),
                 top_k=pick(0, lambda: rng.choice([1, 2, 5, 50, 3000])),
                 top_p=float(np.float32(pick(1.0, lambda: rng.choice([0.0, 0.1, 0.9, 0.999])))),
                 min_p=float(np.float32(pick(0.0, lambda: rng.choice([1e-4, 0.05, 1.0]))))) for _ in range(b)]


def tensors_of(s):
    return {k: torch.tensor([x[k] for x in s], dtype=torch.int32 if k == "top_k" else torch.float32, device=DEV) for k in s[0]}


@pytest.mark.parametrize("V", [1, 2, 7, 128, 1000, 4099, 32000, 128256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_settings(V, dtype):
    B = 24
    z = (torch.randn(B, V, generator=torch.Generator().manual_seed(V)) * 3).to(dtype)
    u = torch.rand(B, generator=torch.Generator().manual_seed(V + 1))
    s = settings_of(B, V)
    check_sample(z, u, rt.sample(z.to(DEV), u.to(DEV), **tensors_of(s)), s)
    # the same settings for all rows, as numbers; one row at a time
    one = dict(temperature=0.75, top_k=min(V, 40), top_p=0.75, min_p=0.0625)
    check_sample(z[:3], u[:3], rt.sample(z[:3].to(DEV), u[:3].to(DEV), **one), [one] * 3)
    check_sample(z[5:6], u[5:6], rt.sample(z[5:6].to(DEV), u[5:6].to(DEV)), [{}])


@pytest.mark.parametrize("B", [1, 9, 17, 41, 130])
def test_sample_batches_and_strides(B):
    V = 5003
    z = torch.randn(B, V + 11, generator=torch.Generator().manual_seed(B)) * 2
    u = torch.rand(B, generator=torch.Generator().manual_seed(B))
    s = settings_of(B, B)
    check_sample(z[:, 3: V + 3], u, rt.sample(z.to(DEV)[:, 3: V + 3], u.to(DEV), **tensors_of(s)), s)


def test_sample_ties_masks_and_ends():
    V = 20000
    inf = math.inf
    z = torch.zeros(14, V)                     # 0, 1: all equal
    z[2] = torch.randn(V, generator=torch.Generator().manual_seed(0)).round()  # many ties
    z[3] = z[2]
    z[4] = -inf
    z[4, 17777] = -5.0                         # a grammar's single choice
    z[5] = -inf                                # nothing left
    z[6] = math.nan
    z[6, 3] = 1.0
    z[7, 100] = inf
    z[8] = -1e38
    z[8, 9] = 3e38
    z[9, ::2] = -0.0                           # -0 and 0 are the same logit
    z[10] = torch.randn(V, generator=torch.Generator().manual_seed(1)) * 1e-30
    z[11] = -inf
    z[11, [5, 4000, 19999]] = torch.tensor([1.0, 1.0, 0.5])
    z[12] = torch.linspace(0, -30, V)
    z[13] = z[12].flip(0)
    u = torch.tensor([0.0, 0.999999940395, 0.3, 0.7, 0.5, 0.5, 0.2, 0.9, 0.9, 0.66, 0.41, 0.5, 0.37, 0.92])
    for s in (dict(), dict(top_k=7), dict(top_p=0.4), dict(top_k=5000, top_p=0.75), dict(top_p=0.9, min_p=0.5),
              dict(temperature=0.5, min_p=1.0), dict(top_k=2, temperature=2.0), dict(temperature=0.0), dict(top_p=1e-30)):
        check_sample(z, u, rt.sample(z.to(DEV), u.to(DEV), **s), [s] * len(z))


def test_sample_frequencies():
    """u on a grid: every token comes out as often as its probability says, within one grid step either way."""
    n, V = 4096, 37
    z = torch.randn(1, V, generator=torch.Generator().manual_seed(5)).expand(n, V).contiguous()
    u = (torch.arange(n) + 0.5) / n
    tokens, _ = rt.sample(z.to(DEV), u.to(DEV), temperature=0.8)
    share = torch.bincount(tokens.cpu().long(), minlength=V).double() / n
    want = torch.softmax(z[0].double() / float(np.float32(0.8)), 0)
    assert (share - want).abs().max() <= 1.0 / n + 1e-9


def test_sample_refuses_wrong_tensors():
    z, u = torch.zeros(2, 64, device=DEV), torch.zeros(2, device=DEV)
    for args, kw in (((z.half(), u), {}), ((z.t(), u), {}), ((z, u.double()), {}), ((z, u[:1]), {}), ((z, u.cpu()), {}),
                     ((z, u), dict(top_k=u)), ((z, u), dict(temperature=u[:1])), ((z, u), dict(tokens=u))):
        with pytest.raises(ValueError):
            rt.sample(*args, **kw)


# ---- streams and graphs ----
def test_streams_and_graphs():
    P, D, H, G = 64, 64, 2, 4
    lens = [300, 129, 64]
    c, r = both(1, 16, H, P, D)
    pages = deal(lens, P, 16, random.Random(4), extra=1)
    tab = table_of(pages)
    fill(c, r, pages, lens, 70, 1)
    q, n = gen(3, 1, H * G, D, seed=8).to(DEV), i32(lens)
    want = c.attend(q, tab, n)
    # two streams at once, each call with a workspace of its own
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [c.attend(q, tab, n, stream=st[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    # a decode step of the cache captured: store the new token, attend, sample; replayed with other inputs
    new = [torch.zeros(1, 3, 1, H, D, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    z, u = torch.zeros(3, 5000, device=DEV), torch.zeros(3, device=DEV)
    one, after = i32([1, 1, 1]), i32([x + 1 for x in lens])

    def step():
        c.store(new[0], new[1], tab, n, one)
        return c.attend(q, tab, after) + rt.sample(z, u, temperature=0.8, top_p=0.9)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
        assert graphs[-1][0] is graph
    c.check()
    for k in range(4):
        for t, s in zip(new, (200 + k, 300 + k)):
            t.copy_(gen(1, 3, 1, H, D, seed=s))
        z.copy_(torch.randn(5000, generator=torch.Generator().manual_seed(k)).expand(3, -1))
        u.copy_(torch.rand(3, generator=torch.Generator().manual_seed(k)))
        graph, out = graphs[k % 2]
        graph.replay()
        torch.cuda.synchronize()
        for name, t in zip("kv", new):
            for b in range(3):
                r.store(name, t[:, b].cpu(), pages[b], lens[b])
        check_attend(r, out[:2], q.cpu(), pages, [x + 1 for x in lens], 0, 0)
        s = dict(temperature=float(np.float32(0.8)), top_p=float(np.float32(0.9)))
        check_sample(z.cpu(), u.cpu(), out[2:], [s] * 3)


# ---- the operators together with the decoder ----
def test_session_samples_parks_forks_and_restores():
    """Decode with sampling; park a sequence in the 8-bit cache; fork it; go on from the fork in another session; the
    fork's K/V are the dequantised ones and its next logits those of a decoder whose cache holds exactly them."""
    shape = synth.TINY
    P, steps, lens = 32, 3, [40, 21]
    w = synth.make_weights(shape, 31, device=DEV)
    kc, vc = synth.make_cache(shape, 2, 80, 131, device=DEV)
    a = rt.Session(shape, w, kc, vc, lens, steps)
    a.tokens[0] = i32([5, 900])
    u = torch.rand(steps, 2, generator=torch.Generator().manual_seed(1)).to(DEV)
    s = dict(temperature=0.875, top_k=200, top_p=0.9375)
    tokens, logprob = a.generate(0, steps, u, **s)
    a.sync()
    assert tokens.shape == (steps, 2) and (logprob <= 0).all()
    check_sample(a.logits.cpu(), u[-1].cpu(), (tokens[-1], logprob[-1]), [s] * 2)
    # step by step gives the same
    kc2, vc2 = synth.make_cache(shape, 2, 80, 131, device=DEV)
    b = rt.Session(shape, w, kc2, vc2, lens, steps)
    b.tokens[0] = i32([5, 900])
    for i in range(steps):
        b.run(i, 1, host_tokens=True)
        b.sample(i, u[i], **s)
    b.sync()
    assert torch.equal(b.tokens[1:], tokens)
    # park both sequences
    done = [n + steps for n in lens]
    pool = kvcache.PagePool(8)
    c = kvcache.Kv8Cache.empty(shape.L, 8, shape.Hkv, shape.D, P, DEV)
    pages = [pool.alloc(-(-n // P)) for n in done]
    a.store_kv(c, table_of(pages), i32([0, 0]), i32(done))
    r = ref.RefCache(shape.L, 8, shape.Hkv, P, shape.D)
    for n, t in (("k", kc), ("v", vc)):
        for i, m in enumerate(done):
            r.store(n, t[:, i, :, :m].transpose(1, 2).cpu(), pages[i], 0)
    # fork sequence 0, then let the parent go on over its own last page
    child, src, dst = pool.fork(pages[0], done[0], P)
    c.copy_pages(src, dst)
    new = gen(shape.L, 1, 1, shape.Hkv, shape.D, seed=77).to(DEV)
    c.store(new, new, table_of(pages[:1]), i32([done[0]]), i32([1]))
    pool.release(pages[1])
    # the pool packed: pages move, the child's table follows
    tab = table_of([child])
    moves = pool.compact()
    c.copy_pages(*moves, table=tab)
    c.check()
    moved = tab[0].tolist()[:len(child)]
    q = gen(1, 1, shape.Hq, shape.D, seed=78)
    check_attend(r, c.attend(q.to(DEV), tab, i32(done[:1]), layer=1), q, [pages[0]], done[:1], 1, 0)
    assert moved == [dict(zip(*moves)).get(x, x) for x in child]
    # restore the fork into a fresh decoder
    kd, vd = (torch.zeros((shape.L, 1, shape.Hkv, 80, shape.D), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    d = rt.Session(shape, w, kd, vd, done[:1], 2)
    d.load_kv(c, tab, i32([0]), i32(done[:1]))
    d.sync()
    ke, ve = kd.clone(), vd.clone()
    for n, t in (("k", kd), ("v", vd)):
        want = torch.stack([torch.stack([r.token(n, l, pages[0], j) for j in range(done[0])], 1) for l in range(shape.L)])
        assert torch.equal(t[:, 0, :, :done[0]].cpu(), want.to(torch.bfloat16))
        assert (t[:, 0, :, done[0]:] == 0).all()
    e = rt.Session(shape, w, ke, ve, done[:1], 2)
    for x in (d, e):
        x.tokens[0] = tokens[-1, :1]
        x.run(0, 1, host_tokens=True)
        x.sync()
    assert torch.equal(d.logits, e.logits)
    with pytest.raises(ValueError):
        a.sample(steps, u[0])


# ---- far and short ----
def test_offsets_beyond_32_bits():
    """Pages, token rows and logits whose byte (and element) offsets pass 2^31 and 2^32."""
    P, D, H, N, n = 64, 128, 8, 70000, 70     # 4.6 GB of K codes
    c = kvcache.Kv8Cache.empty(1, N, H, D, P, DEV)
    ids = [N - 1, 40000]
    r = ref.RefCache(1, 2, H, P, D)
    far = 2 ** 31 + 4096                      # elements between the two token blocks of the buffer
    buf = torch.zeros(far + n * H * D + 64, dtype=torch.bfloat16, device=DEV)
    rows = {k: gen(1, n, H, D, seed=150 + i) for i, k in enumerate("kv")}
    for i, k in enumerate("kv"):
        buf.as_strided((1, 1, n, H, D), (0, 0, H * D, D, 1), far * i).copy_(rows[k][:, None])
        r.store(k, rows[k], [0, 1], 0)
    k, v = (buf.as_strided((1, 1, n, H, D), (8, 8, H * D, D, 1), far * i) for i in range(2))
    tab = i32([ids])
    c.store(k, v, tab, i32([0]), i32([n]))
    for name in "kv":
        for j, page in enumerate(ids):
            x = ref.e4m3_values(getattr(c, name).view(torch.uint8)[0, page].cpu())
            x = x.transpose(1, 2) if name == "v" else x
            assert torch.equal(x, r.code[name][0, j])
    q = gen(1, 1, 2 * H, D, seed=152)
    check_attend(r, c.attend(q.to(DEV), tab, i32([n])), q, [[0, 1]], [n], 0, 0)
    c.copy_pages(ids, [7, 60000], table=tab)
    assert tab.tolist() == [[7, 60000]]
    check_attend(r, c.attend(q.to(DEV), tab, i32([n])), q, [[0, 1]], [n], 0, 0)
    back = buf.as_strided((2, 1, n, H, D), (far, 8, H * D, D, 1))  # both blocks as two rows far apart
    buf.zero_()
    c.load(back[:1], back[1:], tab, i32([0]), i32([n]))
    for i, name in enumerate("kv"):
        want = torch.stack([r.token(name, 0, [0, 1], j) for j in range(n)]).to(torch.bfloat16)
        assert torch.equal(back[i, 0].cpu(), want)
    c.check()
    z = buf.as_strided((2, 1000), (far, 1))
    x = torch.randn(2, 1000, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    z.copy_(x)
    u = torch.tensor([0.3, 0.8])
    check_sample(x, u, rt.sample(z, u.to(DEV), top_p=0.9), [dict(top_p=0.9)] * 2)


def test_attend_more_queries_than_tokens_and_spread_rows():
    """A sequence shorter than its new tokens: the first queries see nothing. One new token a sequence taken out of longer
    rows, the output into such rows."""
    P, D, H, G, T = 32, 64, 2, 2, 7
    lens = [3, 40]
    c, r = both(1, 4, H, P, D, poison=True)
    pages = [[3], [0, 2]]
    fill(c, r, pages, lens, 160, 1)
    q = gen(2, T, H * G, D, seed=161)
    for window in (0, 2):
        got = c.attend(q.to(DEV), table_of(pages), i32(lens), window=window)
        assert (got[0][0, :4] == 0).all() and (got[1][0, :4] == -math.inf).all()
        check_attend(r, got, q, pages, lens, 0, window)
    long, out = q.to(DEV), torch.full((2, 5, H * G, D), 9.0, dtype=torch.bfloat16, device=DEV)
    got = c.attend(long[:, 6:], table_of(pages), i32(lens), out=out[:, 2:3])
    check_attend(r, got, q[:, 6:], pages, lens, 0, 0)
    assert (out[:, :2] == 9).all() and (out[:, 3:] == 9).all()
    with pytest.raises(ValueError, match="evenly spaced"):
        c.attend(long[:, 5:], table_of(pages), i32(lens))
    c.check()


# ---- arguments ----
def test_load_into_packed_rows_and_parts_of_a_session():
    """Packed ragged rows of load; a session's positions from the middle on, stored and brought back."""
    H, D, P, cnt = 2, 64, 32, [5, 0, 33]
    c, r = both(1, 8, H, P, D)
    pages = [[3], [], [6, 0]]
    fill(c, r, pages, cnt, 120, 1)
    flat = [torch.full((sum(cnt) + 2, H, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    e = lambda x: x[None, None].expand(1, 3, -1, -1, -1)  # noqa: E731
    c.load(e(flat[0]), e(flat[1]), table_of(pages), i32([0, 0, 0]), i32(cnt), row0=i32([1, 6, 6]), max_count=33)
    c.check()
    for n, t in zip("kv", flat):
        want = torch.full((sum(cnt) + 2, H, D), 7.0, dtype=torch.bfloat16)
        for b, at in ((0, 1), (2, 6)):
            for i in range(cnt[b]):
                want[at + i] = r.token(n, 0, pages[b], i).to(torch.bfloat16)
        assert torch.equal(t.cpu(), want)
    with pytest.raises(ValueError, match="overlap"):
        c.load(e(flat[0]), e(flat[1]), table_of(pages), i32([0, 0, 0]), i32(cnt))
    shape = synth.TINY
    w = synth.make_weights(shape, 41, device=DEV)
    kc, vc = synth.make_cache(shape, 2, 90, 141, device=DEV)
    s = rt.Session(shape, w, kc, vc, [80, 60], 1)
    c = kvcache.Kv8Cache.empty(shape.L, 8, shape.Hkv, shape.D, P, DEV)
    r = ref.RefCache(shape.L, 8, shape.Hkv, P, shape.D)
    tab = i32([[0, 1, 2], [3, 4, -1]])
    s.store_kv(c, tab, i32([40, 0]), i32([40, 60]))
    k0 = kc.clone()
    kc.zero_()
    s.load_kv(c, tab, i32([50, 10]), i32([30, 20]), max_count=30)
    s.sync()
    c.check()
    r.store("k", k0[:, 0, :, 40:80].transpose(1, 2).cpu(), [0, 1, 2], 40)
    r.store("k", k0[:, 1, :, :60].transpose(1, 2).cpu(), [3, 4], 0)
    for b, pages, lo, hi in ((0, [0, 1, 2], 50, 80), (1, [3, 4], 10, 30)):
        for j in range(90):
            want = torch.stack([r.token("k", l, pages, j) for l in range(shape.L)]) if lo <= j < hi else 0.0
            assert (kc[:, b, :, j].double().cpu() == want).all()


def test_attend_arguments():
    c, r = both(1, 4, 1, 32, 64)
    pages = [[2, 1]]
    fill(c, r, pages, [50], 130, 1)
    tab, n, q = table_of(pages), i32([50]), gen(1, 1, 2, 64, seed=131).to(DEV)
    size = c.attend_workspace(1, 2)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    want = c.attend(q, tab, n)
    got = c.attend(q, tab, n, workspace=ws, out=torch.empty_like(q))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # in the place of the queries
    p = q.clone()
    assert torch.equal(c.attend(p, tab, n, out=p)[0], want[0])
    bad = [dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(tab=tab.long()), dict(tab=tab[0]),
           dict(tab=tab.cpu()), dict(n=n.long()), dict(n=i32([50, 50])), dict(max_tokens=2), dict(out=q.float()),
           dict(lse=q), dict(workspace=q), dict(q_start=i32([0, 1]))]
    for kw in bad:
        a = dict(q=q, tab=tab, n=n)
        a.update({k: kw[k] for k in a if k in kw})
        with pytest.raises(ValueError):
            c.attend(a["q"], a["tab"], a["n"], **{k: v for k, v in kw.items() if k not in a})
    for kw in (dict(workspace=ws[:16]), dict(layer=1), dict(layer=-1), dict(window=-1), dict(scale=-1.0)):
        with pytest.raises(rt.MkError):
            c.attend(q, tab, n, **kw)
    with pytest.raises(rt.MkError):  # 3 query heads over 2 kv heads
        d, _ = both(1, 4, 2, 32, 64)
        d.attend(gen(1, 1, 3, 64, seed=1).to(DEV), tab, n)
    x = gen(1, 1, 5, 1, 64, seed=2).to(DEV)
    for args in ((x.float(), x, tab, n, n), (x[:, :, :, :, :32], x, tab, n, n), (x, x[:, :, :4], tab, n, n),
                 (x, x, tab, n.long(), n), (x, x, tab.cpu(), n, n), (x[..., ::2], x[..., ::2], tab, n, n)):
        with pytest.raises(ValueError):
            c.store(*args)
    with pytest.raises(ValueError):
        kvcache.Kv8Cache(c.k, c.k, c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        kvcache.Kv8Cache(c.k[:, ::2], c.v[:, ::2], c.k_scale[:, ::2], c.v_scale[:, ::2])
    with pytest.raises(ValueError):
        c.copy_pages([0, 1], [2])
    c.check()


def test_no_sequences_and_no_tokens():
    c, _ = both(1, 4, 1, 32, 64)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out, lse = c.attend(torch.zeros((0, 1, 2, 64), dtype=torch.bfloat16, device=DEV), none.view(0, 1), none)
    assert out.shape == (0, 1, 2, 64) and lse.shape == (0, 1, 2)
    out, lse = c.attend(torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV), i32([[0]]), i32([5]), q_start=i32([0, 0]))
    assert out.shape == (0, 2, 64)
    x = torch.zeros((1, 0, 3, 1, 64), dtype=torch.bfloat16, device=DEV)
    c.store(x, x, none.view(0, 1), none, none)
    c.load(x, x, none.view(0, 1), none, none)
    t, lp = rt.sample(torch.zeros((0, 10), device=DEV), torch.zeros(0, device=DEV))
    assert t.shape == (0,) and lp.shape == (0,)
    c.check()
