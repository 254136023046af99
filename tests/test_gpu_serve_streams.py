"""Serving operators called from several threads and on streams other than the current one."""
import random
import threading

import pytest
import torch

from persistent_megakernel_decode_gb300 import kvcache
from persistent_megakernel_decode_gb300 import runtime as rt
from persistent_megakernel_decode_gb300 import synth
from test_gpu_serve import DEV, both, check_sample, deal, fill, gen, i32, table_of

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def hold(ms=60):
    """Keep the current stream busy, so that what is queued behind this has not run when another stream's work has."""
    torch.cuda._sleep(int(ms * 2e6))


def recycled(shape, dtype, value):
    """Free a block of memory to the current stream's pool while its filling is still queued there."""
    hold()
    torch.empty(shape, dtype=dtype, device=DEV).fill_(value)


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


def test_sample_beside_a_busy_current_stream():
    """Strided uniforms and settings, and results in recycled memory, while the current stream is behind."""
    B, V = 6, 9000
    z = torch.randn(B, V, generator=torch.Generator().manual_seed(1)) * 2
    u = torch.rand(B, 3, generator=torch.Generator().manual_seed(2))
    p = torch.rand(3, B, generator=torch.Generator().manual_seed(3)) * 0.5 + 0.5
    k = torch.randint(5, 4000, (B, 2), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    zd, ud, pd, kd = z.to(DEV), u.to(DEV), p.to(DEV).t().contiguous().t(), k.to(DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(3):
        recycled((B,), torch.int32, -5)
        recycled((B,), torch.float32, 5.0)
        got = rt.sample(zd, ud[:, i], top_k=kd[:, i % 2], top_p=pd[i], stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        check_sample(z, u[:, i], got, [dict(top_k=int(k[b, i % 2]), top_p=float(p[i, b])) for b in range(B)])


def test_session_of_another_stream_samples_transposed_uniforms():
    shape, steps, lens = synth.TINY, 3, [40, 21]
    w = synth.make_weights(shape, 31, device=DEV)
    u = torch.rand(2, steps, generator=torch.Generator().manual_seed(1)).to(DEV)  # [B, steps]
    got = []
    for stream in (None, torch.cuda.Stream()):
        kc, vc = synth.make_cache(shape, 2, 80, 131, device=DEV)
        s = rt.Session(shape, w, kc, vc, lens, steps, stream=stream)
        s.tokens[0] = i32([5, 900])
        torch.cuda.synchronize()
        if stream is not None:
            hold()
        tokens, logprob = s.generate(0, steps, u.t(), temperature=0.875, top_k=200)
        s.sync()
        torch.cuda.synchronize()
        got.append((tokens.clone(), logprob.clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_attend_beside_a_busy_current_stream():
    """Results and workspace in recycled memory of which the current stream still has work queued."""
    P, D, H, G, lens = 64, 128, 2, 4, [2500, 64, 1111]
    c, r = both(1, 120, H, P, D)
    pages = deal(lens, P, 120, random.Random(5))
    fill(c, r, pages, lens, 210, 1)
    a = (gen(3, 2, H * G, D, seed=9).to(DEV), table_of(pages), i32(lens))
    want = c.attend(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    size = c.attend_workspace(3, H * G, 2, a[1].shape[1])
    for _ in range(3):
        recycled(want[0].shape, torch.bfloat16, -5)
        recycled(want[1].shape, torch.float32, 5.0)
        recycled((size,), torch.uint8, 77)
        got = c.attend(*a, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_new_cache_on_another_stream():
    """The status words of a cache made behind queued work, in recycled memory."""
    side = torch.cuda.Stream()
    c = kvcache.Kv8Cache.empty(1, 4, 1, 64, 32, DEV)
    q, n = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device=DEV), i32([3])
    tabs = i32([[2]]), i32([[4]])
    torch.cuda.synchronize()
    recycled((4,), torch.int32, 7)
    d = kvcache.Kv8Cache(c.k, c.v, c.k_scale, c.v_scale)
    d.check(side)
    d.attend(q, tabs[0], n, stream=side)
    d.check(side)
    d.attend(q, tabs[1], n, stream=side)
    with pytest.raises(rt.MkError, match="page 4"):
        d.check(side)


def test_forked_streams_and_two_graphs_at_once():
    """Two graphs, each with load, page copy, attention and sampling on a stream forked inside the capture, replayed at the
    same time on two streams."""
    P, D, H, G, lens = 32, 64, 2, 4, [700, 90]
    c, r = both(1, 80, H, P, D)
    pages = deal(lens, P, 60, random.Random(8))
    fill(c, r, pages, lens, 240, 1)
    free = sorted(set(range(80)) - {x for p in pages for x in p})
    tab, n = table_of(pages), i32(lens)
    z, u = torch.randn(2, 4000, generator=torch.Generator().manual_seed(5)).to(DEV), torch.rand(2, 3, device=DEV)
    lo, count = i32([5, 6]), i32([40, 33])
    graphs, kept = [], []
    for i in range(2):
        q = gen(2, 3 + i, H * G, D, seed=241 + i).to(DEV)
        rows = [torch.zeros((1, 2, 40, H, D), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        kept.append(q)  # the graphs read it
        src, dst = [pages[0][i]], [free[i]]

        def step(stream=None):
            c.load(rows[0], rows[1], tab, lo, count, stream=stream)
            c.copy_pages(src, dst, stream=stream)
            return c.attend(q, tab, n, stream=stream) + rt.sample(z, u[:, i], top_p=0.9, stream=stream)
        want = [t.clone() for t in step()]
        loaded = [t.clone() for t in rows]
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            out = step(side)
            torch.cuda.current_stream().wait_stream(side)
        graphs.append((graph, out, want, rows, loaded, src, dst))
    on = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for _, out, _, rows, _, _, dst in graphs:
            for t in rows:
                t.zero_()
            c.k.view(torch.uint8)[:, dst] = 0
        torch.cuda.synchronize()
        for s, (graph, *_) in zip(on, graphs):
            with torch.cuda.stream(s):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for _, out, want, rows, loaded, src, dst in graphs:
            assert all(torch.equal(a, b) for a, b in zip([*out, *rows], want + loaded))
            assert torch.equal(c.k.view(torch.uint8)[:, dst], c.k.view(torch.uint8)[:, src])
    c.check()
