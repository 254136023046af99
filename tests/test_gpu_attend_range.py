"""Cache attention at the ends of its arguments' ranges: large values, windows beyond any length.  Tolerances as derived in
``test_gpu_serve``."""
import random

import pytest
import torch

from test_gpu_serve import DEV, both, check_attend, deal, fill, gen, i32, table_of

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("P, D, T", [(64, 128, 1), (32, 64, 9)])
@pytest.mark.parametrize("power", [118, -100])
def test_values_near_the_ends_of_bf16(P, D, T, power):
    """|v| up to 2^120, several hundred tokens of like weight: the sums stay within fp32."""
    H, G, lens = 2, 4, [300, 77]
    c, r = both(1, 20, H, P, D, poison=True)
    pages = deal(lens, P, 20, random.Random(power))
    kv = [gen(1, 2, 300, H, D, seed=220 + i, scale=s) for i, s in enumerate((1.0, 2.0 ** power))]
    c.store(*(x.to(DEV) for x in kv), table_of(pages), i32([0, 0]), i32(lens))
    for n, x in zip("kv", kv):
        for b, m in enumerate(lens):
            r.store(n, x[:, b, :m], pages[b], 0)
    q = gen(2, T, H * G, D, seed=222)
    got = c.attend(q.to(DEV), table_of(pages), i32(lens))
    c.check()
    check_attend(r, got, q, pages, lens, 0, 0)


@pytest.mark.parametrize("P, D", [(32, 64), (64, 128)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3])
def test_windows_beyond_any_length(P, D, window):
    """They are no windows, also for sequences shorter than their new tokens."""
    H, G, T, lens = 2, 2, 17, [3, 40, 16, 150]
    c, r = both(1, 20, H, P, D, poison=True)
    pages = deal(lens, P, 20, random.Random(7))
    fill(c, r, pages, lens, 230, 1)
    q = gen(4, T, H * G, D, seed=231)
    got = c.attend(q.to(DEV), table_of(pages), i32(lens), window=window)
    c.check()
    check_attend(r, got, q, pages, lens, 0, 0)
    for a, b in zip(got, c.attend(q.to(DEV), table_of(pages), i32(lens))):
        assert torch.equal(a, b)
