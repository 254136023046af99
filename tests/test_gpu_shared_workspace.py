"""Attention over shared prefixes on the GPU with a workspace of the caller's, sized once for the most groups: the call writes
nothing behind it, whatever the groups are.  Tolerances as in ``test_gpu_serve``."""
import pytest
import torch

from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_beams import DEV, built, check_attend, gen, i32, shared_case, table_of  # noqa: F401  (built is a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.mark.parametrize("P, D", [(32, 64), (64, 128)])
def test_one_workspace_for_any_groups(P, D):
    B, hq, hkv = 64, 8, 2
    c, r, pages = shared_case(P, D, hq, hkv, [0, B], [5 * P], [5 * P + 1 + (3 * b) % (2 * P) for b in range(B)], seed=1)
    lens = [5 * P + 1 + (3 * b) % (2 * P) for b in range(B)]
    q = [gen(1, hq, D, seed=b) for b in range(B)]
    need = c.attend_shared_workspace(B, hq, 32, table_width=max(map(len, pages)))
    room = torch.empty(need + 65536, dtype=torch.uint8, device=DEV)
    for n, first in ((B, list(range(0, B + 1, 2))), (B, [0, B]), (B, [0, 10, 20, 64]), (9, [0, 9]), (2, [0, 2]), (B, [0])):
        room.fill_(0xA5)
        args = [torch.stack(q[:n]).to(DEV), table_of(pages[:n]), i32(lens[:n]), i32(first), i32([5 * P] * (len(first) - 1))]
        got = c.attend_shared(*args, workspace=room[:need])
        c.check()
        some = sorted({0, n // 2, n - 1})
        check_attend(r, ([got[0][b] for b in some], [got[1][b] for b in some]), [q[b] for b in some], [pages[b] for b in some],
                     [lens[b] for b in some], 0, 0)
        assert (room[need:] == 0xA5).all()
    with pytest.raises(rt.MkError, match="workspace"):
        c.attend_shared(*args, workspace=room[:64])
