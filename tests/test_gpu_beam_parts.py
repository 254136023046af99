"""Beam selection on the GPU where the parts of a row follow from how many lists an SM holds: many continuations, few and many
prompts.  Tolerances as in ``test_gpu_beams``."""
import ctypes as C

import pytest
import torch

from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_beams import DEV, built, check_select, logits_of, scores_of  # noqa: F401  (built is a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.mark.parametrize("num", [32, 33, 66, 67, 99, 100, 128])
@pytest.mark.parametrize("b, w, v", [(1, 2, 40000), (1, 64, 4100), (12, 5, 20001), (160, 1, 5000)])
def test_select_many_continuations(b, w, v, num):
    check_select(logits_of(b * w, v, seed=num + b), scores_of(b, w, seed=num), num)


def test_workspace_query_is_enough_for_the_call():
    """A workspace of exactly that size, with nothing written behind it."""
    for b, w, v, num in ((1, 1, 622592, 1), (3, 64, 33000, 128), (2, 4, 151936, 100), (700, 2, 9000, 3), (1, 8, 151936, 16)):
        z, s = logits_of(b * w, v, seed=1).to(DEV), scores_of(b, w, seed=2).to(DEV)
        out = [torch.empty(b, num, device=DEV, dtype=t) for t in (torch.float32, torch.int32, torch.int32)]
        d = rt.BeamDesc(z.data_ptr(), v, b, w, v, 0, num, 0, s.data_ptr(), 0, *(x.data_ptr() for x in out))
        need = C.c_uint64()
        assert rt.load().mk_beam_select_workspace(C.byref(d), C.byref(need)) == rt.MK_OK
        room = torch.full((need.value + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        rt.launch(0, None, rt.load().mk_beam_select, C.byref(d), room.data_ptr(), need.value)
        want = rt.beam_select(z, s, num)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert (room[need.value:] == 0xA5).all()
