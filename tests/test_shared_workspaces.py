"""Workspaces of attention over shared prefixes on the CPU: one sized for the most is enough for less, of everything."""
import ctypes as C
import random

import pytest

from persistent_megakernel_decode_gb300 import runtime as rt
from test_serve_args import A, attend, desc


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()


def need(batch, groups, most, width, q_heads, sms, tokens=None):
    a = attend(batch=batch, tokens=batch * most if tokens is None else tokens, max_tokens=most, table_width=width,
               q_heads=q_heads, num_sms=sms, q_start=A)
    n, s = C.c_uint64(), rt.SharedDesc(A, A, groups)
    assert rt.load().mk_cache_attend_shared_workspace(C.byref(desc()), C.byref(a), C.byref(s), C.byref(n)) == rt.MK_OK
    return n.value


def test_a_workspace_for_many_groups_is_enough_when_they_become_one():
    """64 sequences of 32 groups have tiles of 8 rows, of one group tiles of 128."""
    assert need(64, 32, 1, 300, 32, 152) >= need(64, 1, 1, 300, 32, 152) >= need(64, 0, 1, 300, 32, 152)


@pytest.mark.parametrize("seed", range(20))
def test_a_workspace_for_the_most_is_enough_for_less(seed):
    rng = random.Random(seed)
    for _ in range(50):
        batch, most, width = rng.randrange(1, 600), rng.choice((1, 1, 2, 5, 40, 700)), rng.choice((1, 3, 40, 1000))
        groups, heads, sms = rng.randrange(0, min(batch, 1024 - batch) + 1), 4 * rng.randrange(1, 9), rng.choice((1, 3, 20, 152))
        size = need(batch, groups, most, width, heads, sms)
        for _ in range(20):
            b, m, w = rng.randrange(1, batch + 1), rng.randrange(1, most + 1), rng.randrange(1, width + 1)
            g = rng.randrange(0, min(b, groups) + 1)
            assert need(b, g, m, w, heads, sms, tokens=rng.choice((b * m, rng.randrange(b * m + 1)))) <= size, (b, g, m, w)
