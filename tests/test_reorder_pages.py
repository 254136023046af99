"""How the accounting of pages follows the reordering of beams, on the CPU: the plain implementation's tables and the pool."""
import collections
import random

import pytest

import beam_ref
from persistent_megakernel_decode_gb300 import kvcache


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()


def entries(table):
    return [x for row in table for x in row if x >= 0]


@pytest.mark.parametrize("every", [1, 7, 1000])
@pytest.mark.parametrize("w", [1, 2, 5])
def test_pool_follows_by_sharing_the_new_and_releasing_the_old(w, every):
    rng, P, B, prompt, steps = random.Random(w + every), 32, 2, 70, 90
    pool = kvcache.PagePool(100)
    table = []
    for _ in range(B):
        common = pool.alloc(prompt // P)
        for i in range(w):
            if i:
                pool.share(common)
            table.append(common + pool.alloc(-(-(prompt + steps) // P) - len(common)) + [-1])
    old, lost = table, False
    for n in range(prompt, prompt + steps):
        parents = [[rng.randrange(-1, w) for _ in range(w)] for _ in range(B)]
        table, _ = beam_ref.reorder(table, [n] * (B * w), parents, P)
        # from the page being filled on the pages stay the same ones, each in one row; before, some are lost to all rows
        for b in range(B):
            rows = range(b * w, (b + 1) * w)
            assert sorted(x for r in rows for x in table[r][n // P:]) == sorted(x for r in rows for x in old[r][n // P:])
        lost = lost or set(entries(table)) != set(entries(old))
        if (n - prompt) % every == 0:
            pool.share(entries(table))
            pool.release(entries(old))
            old = table
            count = collections.Counter(entries(table))
            assert pool.refs().tolist() == [count[i] for i in range(100)]
    assert lost or w == 1
    pool.share(entries(table))
    pool.release(entries(old))
    pool.release(entries(table))
    assert pool.free_pages == 100
