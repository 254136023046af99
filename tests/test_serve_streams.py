"""Which stream, workspace and numbers a call of the serving operators passes on, on the CPU: the library's calls and torch's
streams are replaced by records."""
import contextlib
import sys
import threading
import time
from types import SimpleNamespace

import pytest
import torch

from persistent_megakernel_decode_gb300 import kvcache
from persistent_megakernel_decode_gb300 import runtime as rt

BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()


class Stream:
    """A stand-in for a torch stream."""

    def __init__(self, handle):
        self.cuda_stream, self.device_index, self.synced = handle, 0, 0

    def synchronize(self):
        self.synced += 1


@pytest.fixture
def machine(monkeypatch):
    """Current streams per thread (default: handle 0), launches [(stream handle, arguments)] and what tensors went through."""
    m = SimpleNamespace(local=threading.local(), launches=[], made=[], recorded=[], default=Stream(0), during=lambda *a: None)
    m.current = lambda *a: getattr(m.local, "stream", m.default)

    @contextlib.contextmanager
    def under(stream):
        before, m.local.stream = m.current(), stream
        try:
            yield
        finally:
            m.local.stream = before

    def launch(index, stream, call, *args):
        m.during(args)
        m.launches.append(((stream or m.current()).cuda_stream, call, args))

    empty, contiguous = torch.empty, torch.Tensor.contiguous

    def made(t):
        m.made.append((t.data_ptr(), m.current().cuda_stream))
        return t

    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: m.current().cuda_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", m.current)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: m.recorded.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made(empty(*a, **k)))
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda t: made(contiguous(t)))
    monkeypatch.setattr(rt, "launch", launch)
    m.under = under
    return m


def cache(monkeypatch):
    """A Kv8Cache of CPU tensors."""
    k, v = (torch.zeros((1, 8, 1) + s, dtype=torch.uint8) for s in ((32, 64), (64, 32)))
    c = kvcache.Kv8Cache(k, v, torch.zeros(1, 8, 1), torch.zeros(1, 8, 1))
    monkeypatch.setattr(c, "_workspace", lambda a: 4096 * a.batch)
    return c


def ask(c, b, **kw):
    return c.attend(torch.zeros((b, 1, 2, 64), dtype=BF16), torch.zeros((b, 3), dtype=I32), torch.ones(b, dtype=I32), **kw)


def test_threads_do_not_share_a_workspace_in_use(machine, monkeypatch):
    """A call of attention is two launches: another thread's must not come between them with the same workspace."""
    c = cache(monkeypatch)
    held, lock, clashes = {}, threading.Lock(), []

    def during(args):
        at, size = args[3], args[4]
        with lock:
            clashes.extend(x for x in held.items() if x[0] < at + size and at < x[0] + x[1])
            held[at] = size
        time.sleep(0.002)
        with lock:
            held.pop(at, None)
    machine.during = during
    threads = [threading.Thread(target=lambda n=n: [ask(c, n) for _ in range(10)]) for n in (1, 2, 3, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(machine.launches) == 40 and not clashes


def test_default_stream_keeps_one_workspace(machine, monkeypatch):
    c = cache(monkeypatch)
    ask(c, 2)
    ask(c, 1)
    ask(c, 2)
    assert len({a[3] for _, _, a in machine.launches}) == 1
    with machine.under(Stream(7)):  # another stream: a workspace of the call's own
        ask(c, 2)
    assert machine.launches[-1][0] == 7 and machine.launches[-1][2][3] != machine.launches[0][2][3]


def test_sample_works_on_its_own_stream(machine):
    """The copies of strided arguments and the results are made on the stream that the launch is on."""
    z, s = torch.zeros(4, 100), Stream(9)
    u, k = torch.zeros(4, 2)[:, 1], torch.zeros((4, 3), dtype=I32)[:, 1]
    out = rt.sample(z, u, top_k=k, stream=s)
    (handle, _, _), = machine.launches
    assert handle == 9 and len(machine.made) == 4 and {h for _, h in machine.made} == {9}
    for t in (z, u, k):  # may be dropped after the call
        assert (t.data_ptr(), 9) in machine.recorded
    for t in out:        # may be dropped while the caller's stream reads them
        assert (t.data_ptr(), 0) in machine.recorded
    machine.made.clear(), machine.recorded.clear()
    rt.sample(z, u, top_k=k, stream=machine.default)
    assert machine.launches[-1][0] == 0 and {h for _, h in machine.made} == {0} and not machine.recorded
    other = Stream(9)
    other.device_index = 1
    with pytest.raises(ValueError, match="stream of cuda:1"):
        rt.sample(z, u, stream=other)


def test_attend_works_on_its_own_stream(machine, monkeypatch):
    """Results and workspace come from the memory of the stream that the launches are on."""
    c, s = cache(monkeypatch), Stream(9)
    machine.made.clear()
    out = ask(c, 2, stream=s)
    (handle, _, args), = machine.launches
    assert handle == 9 and len(machine.made) == 3 and {h for _, h in machine.made} == {9}
    assert args[3] in [at for at, _ in machine.made]
    for t in out:
        assert (t.data_ptr(), 0) in machine.recorded
    machine.recorded.clear()
    ask(c, 2, stream=machine.default)
    assert machine.launches[-1][0] == 0 and not machine.recorded


def test_attend_keeps_arguments_of_another_stream(machine, monkeypatch):
    c, s = cache(monkeypatch), Stream(9)
    a = [torch.zeros((2, 2, 64), dtype=BF16), torch.zeros((1, 3), dtype=I32), torch.ones(1, dtype=I32)]
    kw = dict(q_start=torch.tensor([0, 2], dtype=I32), out=torch.zeros((2, 2, 64), dtype=BF16), lse=torch.zeros(2, 2),
              workspace=torch.zeros(8192, dtype=torch.uint8))
    c.attend(*a, stream=s, **kw)
    for t in [*a, *kw.values()]:
        assert (t.data_ptr(), 9) in machine.recorded


def test_moves_keep_arguments_of_another_stream(machine, monkeypatch):
    c, s = cache(monkeypatch), Stream(9)
    k, v = (torch.zeros((1, 2, 5, 1, 64), dtype=BF16) for _ in "kv")
    tab, ints = torch.zeros((2, 3), dtype=I32), [torch.zeros(2, dtype=I32) for _ in range(3)]
    for f in (c.store, c.load):
        machine.recorded.clear()
        f(k, v, tab, ints[0], ints[1], row0=ints[2], stream=s)
        assert machine.launches[-1][0] == 9
        for t in (k, v, tab, *ints, c.k, c.v, c.k_scale, c.v_scale, c.status):
            assert (t.data_ptr(), 9) in machine.recorded
    machine.recorded.clear()
    c.copy_pages([0], [1], table=tab, stream=s)
    assert machine.launches[-1][0] == 9 and (tab.data_ptr(), 9) in machine.recorded


def test_a_new_cache_may_be_used_on_any_stream(machine, monkeypatch):
    """Its status words are zero before the first call can run, whatever stream that is on."""
    cache(monkeypatch)
    assert machine.default.synced == 1


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 1, sys.maxsize])
def test_numbers_beyond_32_bits_are_not_wrapped(machine, monkeypatch, big):
    c, most = cache(monkeypatch), 2 ** 31 - 1
    last = lambda: machine.launches[-1][2]  # noqa: E731
    rt.sample(torch.zeros(2, 100), torch.zeros(2), top_k=big)
    assert last()[0]._obj.top_k == most
    ask(c, 1, window=big)
    assert last()[2]._obj.window == most
    ask(c, 1, layer=big)
    assert last()[1] == most  # which the library refuses
    c.attend(torch.zeros((2, 2, 64), dtype=BF16), torch.zeros((1, 3), dtype=I32), torch.ones(1, dtype=I32),
             q_start=torch.tensor([0, 2], dtype=I32), max_tokens=big)
    assert last()[2]._obj.max_tokens == most
    x, n = torch.zeros((1, 1, 5, 1, 64), dtype=BF16), torch.zeros(1, dtype=I32)
    c.store(x, x, torch.zeros((1, 3), dtype=I32), n, n, max_count=big)
    assert last()[-1] == most
    asked = []
    monkeypatch.setattr(c, "_workspace", lambda a: asked.append((a.batch, a.tokens, a.max_tokens)))
    c.attend_workspace(4, 2, max_tokens=big)
    assert asked == [(4, most, most)]


def test_attend_refuses_an_output_of_overlapping_rows(machine, monkeypatch):
    c, q = cache(monkeypatch), torch.zeros((3, 1, 2, 64), dtype=BF16)
    for out in (q[:1].expand(3, 1, 2, 64), q[:, :, :1].expand(3, 1, 2, 64)):
        with pytest.raises(ValueError, match="overlap"):
            ask(c, 3, out=out)
    ask(c, 3, out=q)
    assert len(machine.launches) == 1
