"""Cache attention where tiles pass pages they do not load: prompts of many new tokens, windows, page numbers out of range
in the middle of long sequences.  Compared with a plain fp64 attention over the dequantised cache; the tolerances are those
derived in ``test_gpu_serve``."""
import math
import random

import pytest
import torch

import serve_ref as ref
from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_serve import DEV, both, deal, gen, i32, table_of

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def filled(lens, P, D, H, seed, spare=3):
    """A cache with random tokens, the sequences' pages, the rest of it NaN."""
    N = sum(-(-n // P) for n in lens) + spare
    c, _ = both(1, N, H, P, D, poison=True)
    pages = deal(lens, P, N, random.Random(seed))
    k, v = (gen(1, len(lens), max(lens), H, D, seed=seed + i).to(DEV) for i in range(2))
    c.store(k, v, table_of(pages), i32([0] * len(lens)), i32(lens))
    c.check()
    return c, pages


def dense(c, name, pages, n):
    """The sequence's values, fp64 [n, Hkv, D]."""
    x = ref.e4m3_values(getattr(c, name)[0, pages].view(torch.uint8).cpu())
    x = x.transpose(2, 3) if name == "v" else x
    x = x * getattr(c, name + "_scale")[0, pages].double().cpu()[..., None, None]
    return x.transpose(1, 2).reshape(-1, c.kv_heads, c.head_dim)[:n].to(DEV)


def check(c, out, lse, q, pages, n, window=0, there=None):
    """One sequence: q [T, Hq, D]; there [n]: tokens whose pages exist (all)."""
    T, hq, D = q.shape
    k, v = dense(c, "k", pages, n), dense(c, "v", pages, n)
    pos = torch.arange(n - T, n, device=DEV)[:, None]
    j = torch.arange(n, device=DEV)
    seen = j <= pos
    if window:
        seen &= j > pos - window
    if there is not None:
        seen &= there
    g = hq // c.kv_heads
    S = D ** 0.5 * q.abs().max().double() * k.abs().max()
    delta = 2.0 ** -21 * S + 2.0 ** -20
    least = n * 2.0 ** -39 * v.abs().max()
    for h in range(hq):
        z = (q[:, h].double() @ k[:, h // g].T) * D ** -0.5
        z = z.masked_fill(~seen, -math.inf)
        far = torch.logsumexp(z, 1)
        none = ~seen.any(1)
        p = torch.exp(z - torch.where(none, 0.0, far)[:, None])
        want, mag = p @ v[:, h // g], p @ v[:, h // g].abs()
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + delta) * mag + least
        assert (out[none, h] == 0).all() and (lse[none, h] == -math.inf).all()
        off = (out[:, h].double() - want).abs() / tol
        assert (off <= 1).all(), (h, float(off.max()), int(off.amax(1).argmax()))
        off = ((lse[:, h].double() - far).abs() / (delta + 2.0 ** -21 * far.abs()))[~none]
        assert (off <= 1).all(), (h, float(off.max()))


@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("T, H, G, window, sms", [(700, 2, 4, 0, 0), (1100, 1, 2, 0, 3), (1100, 2, 1, 90, 0), (2000, 1, 4, 0, 0),
                                                  (2000, 1, 3, 513, 2)])
def test_prompts(P, D, T, H, G, window, sms):
    """Whole prompts, one over an earlier context: a tile sees the pages up to its last row only."""
    lens = [T, T + 777]
    c, pages = filled(lens, P, D, H, T + P)
    c.num_sms = sms
    q = gen(2, T, H * G, D, seed=T + 5).to(DEV)
    out, lse = c.attend(q, table_of(pages), i32(lens), window=window)
    c.check()
    for b in range(2):
        check(c, out[b], lse[b], q[b], pages[b], lens[b], window)
    again = c.attend(q, table_of(pages), i32(lens), window=window)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
def test_prompts_and_single_tokens_in_one_call(P, D):
    H, G, cnt, lens = 2, 2, [1, 900, 0, 1, 333, 1300], [3000, 900, 50, 1, 1000, 1300]
    c, pages = filled(lens, P, D, H, D)
    start = [sum(cnt[:b]) for b in range(len(cnt) + 1)]
    q = gen(start[-1], H * G, D, seed=77).to(DEV)
    for sms, most in ((0, None), (5, 1300), (0, 1)):
        c.num_sms = sms
        out, lse = c.attend(q, table_of(pages), i32(lens), q_start=i32(start), max_tokens=most)
        c.check()
        for b in range(len(cnt)):
            if cnt[b]:
                at = slice(start[b], start[b + 1])
                check(c, out[at], lse[at], q[at], pages[b], lens[b])


@pytest.mark.parametrize("P, D", [(32, 64), (64, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("T, G, sms", [(1, 4, 2), (1, 16, 0), (5, 4, 1), (9, 8, 3)])
def test_bad_page_numbers_in_long_sequences(P, D, T, G, sms):
    """They are skipped as if masked and recorded; what is around them is right."""
    H, lens = 2, [6000, 4100]
    c, pages = filled(lens, P, D, H, T + G)
    c.num_sms = sms
    rng = random.Random(P + T)
    named, there = [list(p) for p in pages], []
    for b, n in enumerate(lens):
        bad = rng.sample(range(len(pages[b])), len(pages[b]) // 7) + [11, 12, 13]
        for j in bad:
            named[b][j] = rng.choice([-1, -9, c.pages, c.pages + 5, 2 ** 31 - 1])
        there.append(torch.tensor([j // P not in bad for j in range(n)], device=DEV))
    q = gen(2, T, H * G, D, seed=T).to(DEV)
    for _ in range(3):
        out, lse = c.attend(q, table_of(named), i32(lens))
        with pytest.raises(rt.MkError) as e:
            c.check()
        assert e.value.code == rt.MK_ERR_DEVICE_CHECK
        for b in range(2):
            check(c, out[b], lse[b], q[b], pages[b], lens[b], there=there[b])
