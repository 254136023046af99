"""A beam search on the GPU (store, attention over a shared prompt, selection, reordering), each step against what the beams'
kept tokens give by themselves: their K and V, quantised in the order in which they were stored, attention over those in 64
bits, the selection from its definition.  And the pages: none is lost or counted twice.

Tolerances: none for codes and scales (every rounding is defined), beams and tokens; attention as in ``test_gpu_serve``.
"""
import collections
import copy
import math

import pytest
import torch

import serve_ref as ref
from persistent_megakernel_decode_gb300 import kvcache
from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_beams import DEV, built, check_attend, check_select, codes, gen, i32, table_of  # noqa: F401  (built is a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.mark.parametrize("P, D, W, steps", [(32, 64, 4, 40), (64, 128, 3, 20), (32, 128, 1, 5), (32, 64, 7, 36)])
def test_each_step_from_the_kept_tokens(P, D, W, steps):
    hq, hkv, V, B, N = 4, 2, 301, 2, 200
    rng = torch.Generator().manual_seed(P + W)
    prompts = [torch.randint(0, V, (n,), generator=rng).tolist() for n in (70, 45)]
    emb = {n: gen(V, h, D, seed=i, scale=1.5) for i, (n, h) in enumerate((("q", hq), ("k", hkv), ("v", hkv)))}
    emb["k"] *= torch.exp2(torch.randint(-3, 4, (V, 1, 1), generator=rng)).to(torch.bfloat16)  # scales that grow inside a page
    head = (torch.randn(hq * D, V, generator=rng) * 0.2).to(DEV)
    pool, c = kvcache.PagePool(N), kvcache.Kv8Cache.empty(1, N, hkv, D, P, DEV)
    rows, beams = [], []  # beams: a cache of each beam's own, in which its pages are 0, 1, ...
    for tokens in prompts:
        n, full = len(tokens), len(tokens) // P * P
        common = pool.alloc(full // P)
        for w in range(W):
            if w:
                pool.share(common)
            rows.append(common + pool.alloc(-(-(n + steps) // P) - len(common)))
            r = ref.RefCache(1, len(rows[-1]), hkv, P, D)
            for x in "kv":
                r.store(x, emb[x][tokens][None], list(range(len(rows[-1]))), 0)
            beams.append(r)
        kv = {x: emb[x][tokens].to(DEV)[None, None] for x in "kv"}
        c.store(kv["k"], kv["v"], table_of([rows[-W]]), i32([0]), i32([n]))
        for w in range(1, W):  # the rest behind the shared pages, for every beam
            c.store(*(kv[x][:, :, full:].contiguous() for x in "kv"), table_of([rows[w - W]]), i32([full]), i32([n - full]))
    table, held = table_of(rows), rows
    lens = [len(t) for t in prompts for _ in range(W)]
    first, shared = i32([0, W, 2 * W]), i32([len(t) for t in prompts])
    score = torch.full((B, W), -math.inf)
    score[:, 0] = 0
    done = torch.zeros((B, W), dtype=torch.bool)
    last = torch.tensor([t[-1] for t in prompts for _ in range(W)])
    for step in range(steps):
        q = emb["q"][last][:, None]
        got = c.attend_shared(q.to(DEV), table, i32(lens), first, shared)
        if step % 3 == 0 or step == steps - 1:
            for x in "kv":  # every slot that holds a token, and the scales
                have, scale = codes(c, x)[0], getattr(c, x + "_scale").double().cpu()[0]
                for b, row in enumerate(table.tolist()):
                    for j in range(-(-lens[b] // P)):
                        n = min(P, lens[b] - j * P)
                        assert torch.equal(have[row[j], :, :n], beams[b].code[x][0, j, :, :n]), (step, x, b, j)
                        assert torch.equal(scale[row[j]], beams[b].scale[x][0, j])
            for b in range(B * W):
                own = list(range(-(-lens[b] // P)))
                check_attend(beams[b], ([got[0][b]], [got[1][b]]), [q[b]], [own], [lens[b]], 0, 0)
        z = got[0].float().reshape(-1, hq * D) @ head
        pick = rt.beam_select(z, score.to(DEV), finished=done.to(DEV), end=1)
        check_select(z.cpu(), score, W, done, 1, pick)
        score, parent, token = (x.cpu() for x in pick)
        table = c.reorder(table, i32(lens), pick[1])
        source = [b * W + (w if parent[b, w] < 0 else int(parent[b, w])) for b in range(B) for w in range(W)]
        beams = [copy.deepcopy(beams[s]) for s in source]
        done = done.gather(1, parent.clamp(min=0).long()) | (token == 1)
        last = token.flatten().clamp(min=0).long()
        kv = {x: emb[x][last] for x in "kv"}
        c.store(*(kv[x].to(DEV)[None, :, None] for x in "kv"), table, i32(lens), i32([1] * (B * W)))
        for b, r in enumerate(beams):
            for x in "kv":
                r.store(x, kv[x][b][None, None], list(range(len(rows[b]))), lens[b])
        lens = [n + 1 for n in lens]
        if step % 7 == 0 or step == steps - 1:  # the pool follows
            now = table.tolist()
            flat = lambda t: [x for r in t for x in r if x >= 0]  # noqa: E731
            pool.share(flat(now))
            pool.release(flat(held))
            held = now
            count = collections.Counter(flat(now))
            assert pool.refs().tolist() == [count[i] for i in range(N)]
    c.check()
    pool.release(flat(held))
    assert pool.free_pages == N
