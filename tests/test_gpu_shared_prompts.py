"""Prompts on the GPU: hundreds of new tokens a sequence behind a shared prefix, and through a window with sinks; sequences that
share nothing beside groups that do; one large group beside many of one.

Tolerances as in ``test_gpu_beams``: those of ``test_gpu_serve``, and for tiles of 128 rows 2^-30 max|v| a token in the place
of 2^-39 (``check_rows`` takes it for all).
"""
import math
import random

import pytest
import torch

from test_gpu_beams import (DEV, both, built, check_attend, check_sinks, codes, deal, fill, gen, i32, shared_case,  # noqa: F401
                            table_of)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


def check_rows(c, got, q, pages, n, some, heads):
    """Rows `some` of one sequence's new tokens q [T, hq, D], of the given q heads, in 64 bits."""
    out, lse = got
    T, hq, D = q.shape
    P = c.page_tokens
    hkv = c.kv_heads
    val = {}
    for x in "kv":
        y = codes(c, x)[0][pages] * getattr(c, x + "_scale")[0].double().cpu()[pages][:, :, None, None]  # [pages, hkv, P, D]
        val[x] = y.transpose(0, 1).reshape(hkv, -1, D)[:, :n]
    for i in some:
        pos = n - T + i
        for h in heads:
            k, v = val["k"][h // (hq // hkv)][: pos + 1], val["v"][h // (hq // hkv)][: pos + 1]
            z = k @ q[i, h].double() * D ** -0.5
            far = torch.logsumexp(z, 0)
            p = torch.exp(z - far)
            S = D ** 0.5 * q[i, h].double().abs().max() * k.abs().max()
            delta = 2.0 ** -21 * S + 2.0 ** -20
            want = p @ v
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + delta) * (p @ v.abs()) + (pos + 1) * 2.0 ** -30 * v.abs().max()
            assert ((out[i, h].double().cpu() - want).abs() <= tol).all(), (i, h)
            assert (lse[i, h].double().cpu() - far).abs() <= delta + 2.0 ** -21 * far.abs()


@pytest.mark.parametrize("P, D", [(32, 64), (64, 128)])
@pytest.mark.parametrize("T", [512, 2048])
def test_prompts_behind_a_shared_prefix(P, D, T):
    """Three conversations' prompts behind one instruction, the second shorter, and one that is by itself."""
    hq, hkv, prefix = 4, 2, 11 * P + 7
    counts = [T, T // 3 + 1, T - 5, 77]
    lens = [prefix + n for n in counts[:3]] + [300]
    c, r, pages = shared_case(P, D, hq, hkv, [0, 3], [prefix], lens, seed=T, N=20 + sum(-(-n // P) for n in lens), poison=False)
    start = [sum(counts[:b]) for b in range(5)]
    q = gen(start[-1], hq, D, seed=1)
    ask = lambda f, *a: f(q.to(DEV), table_of(pages), i32(lens), *a, q_start=i32(start), max_tokens=T)  # noqa: E731
    out, lse = ask(c.attend_shared, i32([0, 3]), i32([prefix]))
    plain = ask(c.attend)
    c.check()
    for b, n in enumerate(counts):
        x = slice(start[b], start[b + 1])
        some = sorted({0, 1, n // 2, n - P, n - 2, n - 1})
        check_rows(c, (out[x], lse[x]), q[x], pages[b], lens[b], some, (0, hq - 1))
    assert (out.double() - plain[0].double()).norm() <= 2.0 ** -8 * plain[0].double().norm()
    assert (lse - plain[1]).abs().max() <= 2.0 ** -12


@pytest.mark.parametrize("T, window, sinks", [(600, 200, 70), (1500, 64, 4), (700, 5000, 9), (515, 1, 1)])
def test_prompts_through_a_window_with_sinks(T, window, sinks):
    P, D, hq, hkv = 32, 64, 6, 2
    lens, counts = [T, T + 333, 40], [T, T - 9, 40]
    start = [sum(counts[:b]) for b in range(4)]
    N = sum(-(-n // P) for n in lens) + 3
    c, r = both(1, N, hkv, P, D)
    pages = deal(lens, P, N, random.Random(T))
    fill(c, r, pages, lens, seed=2, layers=1)
    q = gen(start[-1], hq, D, seed=3)
    out, lse = c.attend(q.to(DEV), table_of(pages), i32(lens), q_start=i32(start), max_tokens=T, window=window, sinks=sinks)
    c.check()
    for b, n in enumerate(counts):
        x = slice(start[b], start[b + 1])
        check_sinks(r, (out[None, x], lse[None, x]), [q[x]], [pages[b]], [lens[b]], 0, window, sinks)


@pytest.mark.parametrize("T, hq", [(1, 8), (3, 8), (40, 24)])
def test_sequences_that_share_nothing_are_as_without_groups(T, hq):
    """Groups of one, groups that share no whole page, and sequences in no group."""
    P, D, hkv, B = 64, 64, 2, 9
    lens = [T + 400 + 100 * b for b in range(B)]
    c, r, pages = shared_case(P, D, hq, hkv, [0, 3], [5 * P], lens, seed=5, poison=False)
    c.num_sms = 30
    q = torch.stack([gen(T, hq, D, seed=b) for b in range(B)]).to(DEV)
    args = q, table_of(pages), i32(lens)
    first = [0, 3, 4, 7]
    got = c.attend_shared(*args, i32(first), i32([5 * P, 5 * P, P - 1]))
    plain = c.attend(*args)
    c.check()
    check_attend(r, ([got[0][b] for b in (0, 2, 3, 5, 8)], [got[1][b] for b in (0, 2, 3, 5, 8)]), [q[b].cpu() for b in (0, 2, 3, 5, 8)],
                 [pages[b] for b in (0, 2, 3, 5, 8)], [lens[b] for b in (0, 2, 3, 5, 8)], 0, 0)
    assert (got[0].double() - plain[0].double()).norm() <= 2.0 ** -8 * plain[0].double().norm()
    assert (got[1] - plain[1]).abs().max() <= 2.0 ** -12


def test_one_large_group_beside_many_of_one():
    """A group of 32 and 32 sequences by themselves, listed as groups and not."""
    P, D, hq, hkv, B = 64, 128, 8, 2, 64
    prefix = 9 * P
    lens = [prefix + 1 + (5 * b) % 90 for b in range(32)] + [30 + 17 * b for b in range(32)]
    c, r, pages = shared_case(P, D, hq, hkv, [0, 32], [prefix], lens, seed=6, N=500)
    q = [gen(1, hq, D, seed=b) for b in range(B)]
    some = [0, 1, 31, 32, 50, 63]
    for first in ([0] + list(range(32, B + 1)), [0, 32]):
        shared = [prefix] * (len(first) - 1)
        got = c.attend_shared(torch.stack(q).to(DEV), table_of(pages), i32(lens), i32(first), i32(shared))
        c.check()
        check_attend(r, ([got[0][b] for b in some], [got[1][b] for b in some]), [q[b] for b in some], [pages[b] for b in some],
                     [lens[b] for b in some], 0, 0)


def test_large_workspaces_are_not_kept():
    """A prompt's workspace goes back to the allocator after the call; small ones stay for the next."""
    P, D, hq, hkv, T = 64, 128, 32, 8, 4096
    c, r = both(1, 2 * T // P, hkv, P, D)
    table, lens = i32([list(range(T // P)), list(range(T // P))]), i32([T, T])
    q = torch.zeros((2, T // 2, hq, D), dtype=torch.bfloat16, device=DEV)
    groups, shared = i32([0, 2]), i32([T // 2])
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    assert c.attend_shared_workspace(2, hq, 1, T // 2) > 128 << 20
    out = c.attend_shared(q, table, lens, groups, shared)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated() - before - sum(x.numel() * x.element_size() for x in out)
    assert held <= 64 << 20
    c.check()
    assert not math.isnan(float(out[1].sum()))
