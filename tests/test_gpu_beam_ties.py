"""Beam selection on the GPU where very many totals are equal: right, and in a time of the same order as otherwise.

Tolerances: none for beams and tokens; scores as in ``test_gpu_beams``.
"""
import math

import pytest
import torch

from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_beams import DEV, built, check_select  # noqa: F401  (built is a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.mark.parametrize("w, v, num", [(64, 300, 128), (8, 40000, 128), (4, 151936, 128), (16, 9001, 32), (3, 70001, 100), (2, 20, 30)])
@pytest.mark.parametrize("scores", ["equal", "apart", "some equal"])
def test_rows_of_one_value(w, v, num, scores):
    sc = {"equal": torch.zeros(1, w) - 5, "apart": -5 - torch.arange(w).float()[None], "some equal": -5 - (torch.arange(w) // 3).float()[None]}
    check_select(torch.zeros(w, v), sc[scores], num)
    check_select(torch.full((w, v), -0.0, dtype=torch.bfloat16), sc[scores], num)


def test_rows_of_one_value_with_others_above_and_ended_beams():
    w, v, num = 8, 40000, 128
    z = torch.zeros(2 * w, v)
    for r in range(2 * w):
        z[r, 777 * r % v: 777 * r % v + 9] = 1.5
    sc = torch.full((2, w), -3.0)
    fin = torch.zeros(2, w, dtype=torch.bool)
    fin[0, 2] = fin[1, 0] = fin[1, 7] = True
    check_select(z, sc, num, fin, 5)
    check_select(z[:, :200].contiguous(), sc, num, fin, 5)


def test_equal_totals_of_different_logits():
    """Differences that 64-bit totals do not show: by beam, and within a beam by the logits."""
    w, v = 6, 30000
    z = torch.randn(1, v, generator=torch.Generator().manual_seed(3)).expand(w, v) * 1e-30
    check_select(z.contiguous(), torch.zeros(1, w) - 1, 100)
    check_select(z.contiguous(), torch.zeros(1, w) - 1, 7)


@pytest.mark.parametrize("w, v, num", [(64, 300, 128), (4, 151936, 128), (8, 151936, 16)])
def test_equal_totals_take_no_time_of_another_order(w, v, num):
    """A millisecond for what other rows take up to a tenth of (it was 9 to 36, each candidate compared with each)."""
    z, sc = torch.zeros(w, v, device=DEV), torch.full((1, w), -5.0, device=DEV)
    rt.beam_select(z, sc, num)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = math.inf
    for _ in range(5):
        a.record()
        rt.beam_select(z, sc, num)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    assert best < 1.0
