"""Attention of one sequence with one kv head over thousands of tokens on the GPU: ranges of one page a CTA, rows merged from
hundreds of parts; by itself, in a group of one and in none.  Tolerances as in ``test_gpu_serve``."""
import pytest
import torch

from test_gpu_beams import DEV, both, built, check_attend, fill, gen, i32, table_of  # noqa: F401  (built is a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.mark.parametrize("P, D", [(32, 64), (64, 128)])
@pytest.mark.parametrize("n, T, hq", [(1000, 1, 4), (9999, 1, 8), (16384, 2, 1), (12001, 5, 8)])
def test_one_sequence_one_kv_head(P, D, n, T, hq):
    pages = [list(range(-(-n // P)))[::-1]]
    c, r = both(1, len(pages[0]), 1, P, D)
    fill(c, r, pages, [n], seed=n, layers=1)
    q = gen(T, hq, D, seed=T, scale=2.0)
    args = q[None].to(DEV), table_of(pages), i32([n])
    plain = c.attend(*args)
    for got in (plain, c.attend_shared(*args, i32([0, 1]), i32([n])), c.attend_shared(*args, i32([0]), i32([]))):
        c.check()
        check_attend(r, got, [q], pages, [n], 0, 0)
