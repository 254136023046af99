"""Serving operators called from several threads and on streams other than the current one."""
import random
import threading

import pytest
import torch

from test_gpu_serve import DEV, both, deal, fill, gen, i32, table_of

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_threads_on_one_cache():
    """Calls of different sizes, most of whose units are cut by CTA boundaries, from four threads."""
    P, D, H, G, lens = 64, 128, 2, 4, [2500, 64, 1111, 3000]
    c, r = both(1, 120, H, P, D)
    pages = deal(lens, P, 120, random.Random(3))
    fill(c, r, pages, lens, 200, 1)
    work = []
    for n, T in ((1, 1), (4, 1), (3, 5), (2, 20)):
        a = (gen(n, T, H * G, D, seed=n + T).to(DEV), table_of(pages[:n]), i32(lens[:n]))
        work.append((a, c.attend(*a)))
    torch.cuda.synchronize()
    wrong, go = [], threading.Barrier(len(work))

    def calls(a, want):
        go.wait()
        got = [c.attend(*a) for _ in range(200)]
        torch.cuda.synchronize()
        wrong.append(sum(not torch.equal(x, y) for g in got for x, y in zip(g, want)))
    threads = [threading.Thread(target=calls, args=w) for w in work]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert wrong == [0] * len(work)
    c.check()
