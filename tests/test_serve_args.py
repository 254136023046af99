"""Serving operators on the CPU: what the calls refuse before any launch, the page accounting, and the 64-bit
implementations the GPU tests compare with."""
import ctypes as C
import random

import numpy as np
import pytest
import torch

import serve_ref as ref
from persistent_megakernel_decode_gb300 import kvcache
from persistent_megakernel_decode_gb300 import runtime as rt


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()


A = 1 << 20  # an aligned address that no refused call may touch


def desc(**kw):
    d = rt.CacheDesc(A, A, A, A, A, 2, 16, 4, 64, 128)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def rows(**kw):
    r = rt.CacheRows(A, A, *[8] * 8, 100, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def attend(**kw):
    a = rt.AttendDesc()
    a.q = a.out = a.lse = a.table = a.lens = A
    a.q_token_stride = a.out_token_stride = 1024
    a.q_head_stride = a.out_head_stride = 128
    a.batch, a.table_width, a.q_heads, a.tokens, a.max_tokens, a.scale, a.num_sms = 3, 8, 8, 3, 1, 0.1, 152
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad, code", [
    (dict(layers=0), rt.MK_ERR_INVALID), (dict(pages=-1), rt.MK_ERR_INVALID), (dict(kv_heads=0), rt.MK_ERR_INVALID),
    (dict(page_tokens=16), rt.MK_ERR_UNSUPPORTED), (dict(page_tokens=128), rt.MK_ERR_UNSUPPORTED),
    (dict(head_dim=96), rt.MK_ERR_UNSUPPORTED), (dict(k_codes=0), rt.MK_ERR_INVALID), (dict(status=0), rt.MK_ERR_INVALID),
    (dict(v_codes=A + 8), rt.MK_ERR_INVALID), (dict(k_scales=A + 2), rt.MK_ERR_INVALID)])
def test_cache_descriptor_refusals(bad, code):
    lib = rt.load()
    d = desc(**bad)
    ids = np.array([1], np.int32), np.array([2], np.int32)
    for rc in (lib.mk_cache_store(C.byref(d), C.byref(rows()), A, 8, A, A, 3, 5, None),
               lib.mk_cache_load(C.byref(d), C.byref(rows()), A, 8, A, A, 3, 5, None),
               lib.mk_cache_attend(C.byref(d), 0, C.byref(attend()), A, 1 << 30, None),
               lib.mk_cache_copy(C.byref(d), ids[0].ctypes.data, ids[1].ctypes.data, 1, None, 0, None),
               lib.mk_cache_status(C.byref(d), 0, None, None)):
        assert rc == code
        assert lib.mk_last_error()


@pytest.mark.parametrize("kw, args", [
    (dict(k=0), {}), (dict(v=A + 2), {}), (dict(k_stride_token=4), {}), (dict(rows=-1), {}),
    ({}, dict(batch=-1)), ({}, dict(width=0)), ({}, dict(count=-1)), ({}, dict(table=0)), ({}, dict(start=0)),
    ({}, dict(batch=70000))])
def test_store_and_load_refusals(kw, args):
    lib = rt.load()
    a = dict(table=A, width=8, start=A, batch=3, count=5)
    a.update(args)
    for f in (lib.mk_cache_store, lib.mk_cache_load):
        rc = f(C.byref(desc()), C.byref(rows(**kw)), a["table"] or None, a["width"], a["start"] or None, A, a["batch"],
               a["count"], None)
        assert rc in (rt.MK_ERR_INVALID, rt.MK_ERR_UNSUPPORTED)
        # nothing to do is no error
        assert f(C.byref(desc()), C.byref(rows()), A, 8, A, A, 0, 5, None) == rt.MK_OK
        assert f(C.byref(desc()), C.byref(rows()), A, 8, A, A, 3, 0, None) == rt.MK_OK


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(out=A + 8), dict(lens=0), dict(batch=-1), dict(batch=1025), dict(q_heads=6), dict(q_heads=0),
    dict(tokens=4), dict(max_tokens=-1), dict(window=-1), dict(scale=-0.5), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(table_width=0), dict(lse=A + 1), dict(q_head_stride=4),
    dict(out_token_stride=1020), dict(table_width=1 << 26)])
def test_attend_refusals(bad):
    lib = rt.load()
    assert lib.mk_cache_attend(C.byref(desc()), 0, C.byref(attend(**bad)), A, 1 << 30, None) in (
        rt.MK_ERR_INVALID, rt.MK_ERR_UNSUPPORTED)


def test_attend_refuses_layers_and_workspaces():
    lib, a, need = rt.load(), attend(), C.c_uint64()
    assert lib.mk_cache_attend_workspace(C.byref(desc()), C.byref(a), C.byref(need)) == rt.MK_OK and need.value > 0
    for layer, ws, n in ((-1, A, need.value), (2, A, need.value), (0, None, need.value), (0, A + 4, need.value),
                         (0, A, need.value - 1)):
        assert lib.mk_cache_attend(C.byref(desc()), layer, C.byref(a), ws, n, None) == rt.MK_ERR_INVALID
    for kw in (dict(batch=0, tokens=0), dict(tokens=0, max_tokens=0)):  # nothing to do
        assert lib.mk_cache_attend(C.byref(desc()), 0, C.byref(attend(**kw)), A, 1 << 30, None) == rt.MK_OK


@pytest.mark.parametrize("src, dst", [([1], [16]), ([-1], [2]), ([1, 2], [3, 3]), ([1, 2], [2, 3]), ([2, 1], [3, 2]),
                                      ([4], [4]), ([1, 5], [5, 1])])
def test_copy_refusals(src, dst):
    s, d = np.array(src, np.int32), np.array(dst, np.int32)
    rc = rt.load().mk_cache_copy(C.byref(desc()), s.ctypes.data, d.ctypes.data, len(src), None, 0, None)
    assert rc == rt.MK_ERR_INVALID
    assert rt.load().mk_cache_copy(C.byref(desc()), s.ctypes.data, d.ctypes.data, 0, None, 0, None) == rt.MK_OK
    assert rt.load().mk_cache_copy(C.byref(desc()), s.ctypes.data, d.ctypes.data, -1, None, 0, None) == rt.MK_ERR_INVALID
    assert rt.load().mk_cache_copy(C.byref(desc()), None, None, 1, None, 0, None) == rt.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(logits=0), dict(u=0), dict(tokens=0), dict(batch=-1), dict(vocab=0),
                                 dict(vocab=622593, row_stride=622593), dict(row_stride=999), dict(logits=A + 2),
                                 dict(tokens=A + 1)])
def test_sample_refusals(bad):
    d = rt.SampleDesc()
    d.logits = d.u = d.tokens = d.logprob = A
    d.row_stride, d.batch, d.vocab = 1000, 2, 1000
    for k, v in bad.items():
        setattr(d, k, v)
    assert rt.load().mk_sample(C.byref(d), None) in (rt.MK_ERR_INVALID, rt.MK_ERR_UNSUPPORTED)
    d.batch, d.vocab, d.row_stride = 0, 1000, 1000
    assert rt.load().mk_sample(C.byref(d), None) == rt.MK_OK
    assert rt.load().mk_sample(None, None) == rt.MK_ERR_INVALID


def test_binding_refuses_cpu_tensors():
    z = torch.zeros((1, 1, 1, 32, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.Kv8Cache(z, z.transpose(3, 4).contiguous(), torch.zeros(1, 1, 1), torch.zeros(1, 1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        rt.sample(torch.zeros(2, 8), torch.zeros(2))


# ---- page accounting ----
def test_pool_takes_the_lowest_free_pages_and_refuses_the_rest():
    p = kvcache.PagePool(8)
    assert p.alloc(3) == [0, 1, 2] and p.alloc(2) == [3, 4] and p.free_pages == 3
    p.release([1, 3])
    assert p.alloc(3) == [1, 3, 5]
    with pytest.raises(rt.MkError, match="out of pages"):
        p.alloc(3)
    assert p.free_pages == 2 and p.alloc(0) == []
    for bad in ([8], [-1], [6]):
        with pytest.raises(rt.MkError):
            p.share(bad)
        with pytest.raises(rt.MkError):
            p.release([0] + bad)
    assert p.refs().tolist() == [1, 1, 1, 1, 1, 1, 0, 0]
    with pytest.raises(rt.MkError, match="more often"):  # the same page twice: undone as a whole
        p.release([2, 0, 0])
    assert p.refs().tolist() == [1, 1, 1, 1, 1, 1, 0, 0] and p.free_pages == 2
    p.share([0, 0])
    p.release([0, 0, 0])
    assert p.refs()[0] == 0 and p.alloc(1) == [0]
    with pytest.raises(rt.MkError):
        kvcache.PagePool(0)


def test_fork_shares_full_pages():
    p = kvcache.PagePool(6)
    a = p.alloc(3)
    assert p.fork(a, 70, 32) == ([0, 1, 3], [2], [3])
    assert p.refs().tolist() == [2, 2, 1, 1, 0, 0]
    assert p.fork(a, 64, 32) == ([0, 1], [], [])  # full pages only
    assert p.fork(a, 0, 32) == ([], [], [])
    with pytest.raises(ValueError):
        p.fork(a, 97, 32)
    p.alloc(2)
    with pytest.raises(rt.MkError):
        p.fork(a, 70, 32)
    assert p.refs().tolist() == [3, 3, 1, 1, 1, 1]


def test_pool_against_a_plain_model():
    rng = random.Random(3)
    p, refs = kvcache.PagePool(40), [0] * 40
    for _ in range(600):
        held = [i for i, r in enumerate(refs) if r]
        what = rng.random()
        if what < 0.4:
            n = rng.randrange(0, 6)
            free = [i for i, r in enumerate(refs) if not r]
            if n <= len(free):
                assert p.alloc(n) == free[:n]
                for i in free[:n]:
                    refs[i] = 1
        elif what < 0.55 and held:
            ids = rng.choices(held, k=3)
            p.share(ids)
            for i in ids:
                refs[i] += 1
        elif what < 0.95 and held:
            ids = rng.sample(held, min(len(held), 4))
            p.release(ids)
            for i in ids:
                refs[i] -= 1
        else:
            src, dst = p.compact()
            assert not set(src) & set(dst) and len(set(dst)) == len(dst)
            for s, d in zip(src, dst):
                assert refs[s] and not refs[d]
                refs[s], refs[d] = 0, refs[s]
            used = sum(r > 0 for r in refs)
            assert all(refs[:used]) and not any(refs[used:])
        assert p.refs().tolist() == refs and p.free_pages == refs.count(0)


# ---- the 64-bit implementations themselves ----
def test_reference_rounding_is_torchs_cast():
    x = torch.cat([torch.linspace(-500, 500, 20001), torch.linspace(-0.04, 0.04, 20001)]).double()
    got = ref.round_e4m3(x)
    want = x.float().clamp(-448, 448).to(ref.F8).double()
    assert torch.equal(got, want)
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    assert torch.equal(ref.e4m3_values(codes).nan_to_num(nan=1e9), codes.view(ref.F8).double().nan_to_num(nan=1e9))


def test_reference_sampling_by_hand():
    z = torch.tensor([1.0, 3.0, 3.0, -float("inf"), 2.0])
    w = torch.exp(z.double() - 3)
    assert ref.sample_row(z, 0.0, temperature=0)[0] == 1
    t, lp = ref.sample_row(z, 0.0)
    assert t == 0 and abs(lp - float(torch.log(w[0] / w.sum()))) < 1e-12
    assert ref.sample_row(z, 0.999999)[0] == 4
    assert ref.sample_row(z, 0.6, top_k=2) == (2, pytest.approx(-np.log(2)))
    assert ref.sample_row(z, 0.99, top_p=0.3)[0] == 1      # one token is enough: the lower index of the tie
    assert ref.sample_row(z, 0.99, top_p=0.0)[0] == 1
    assert ref.sample_row(z, 0.99, min_p=0.5)[0] == 2
    assert ref.sample_row(torch.full((4,), -float("inf")), 0.5) == (0, -float("inf"))


def test_generate_refuses_steps_that_were_not_planned():
    """Before any step runs: the cache and the tokens stay as they are."""
    s = object.__new__(rt.Session)
    s.max_steps, s.B, s.logits, s.torch = 4, 2, torch.zeros(2, 8), torch
    s.run = lambda *a, **k: pytest.fail("a step ran")
    for first, n in ((3, 2), (-1, 2), (0, 5), (5, 0), (1, -1)):
        with pytest.raises(ValueError, match="outside the planned 4"):
            s.generate(first, n, torch.zeros(max(n, 0), 2))
