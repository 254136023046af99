"""Beam selection's sum of exponentials on the GPU, where rows repeat values, so that errors of single terms add up.

The bound, 2^-27 of the sum, from the arithmetic of a term below the bound of the listed logits: the argument's fraction
2^-30.5, a polynomial 2^-30, and the products' rounding 2^-30 make 2^-28.6 at most, the same for equal logits; chains of eight
such products in fp32 2^-28.7 of their thread's sum; the listed logits' weights 2^-30; the unit of the joined sums, 2^-44 of a
number between a half and one a thread and piece, 2^-29 for 622592 logits.  Were all of one sign: 2^-27.1.
"""
import math

import pytest
import torch

from persistent_megakernel_decode_gb300 import runtime as rt

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def lse_of(z):
    z = z.double()
    return torch.logsumexp(torch.where(torch.isnan(z), -math.inf, z), 1), z.max(1).values


def error_of(z):
    """Errors of the log sums of z's rows, each a prompt with one beam whose score all but cancels the rest of the total: the
    total is then so small that its own rounding (2^-24 of it) is nothing."""
    lse, top = lse_of(z)
    score = (lse - top).float()
    got = rt.beam_select(z.to(DEV), score[:, None].to(DEV), 1)[0][:, 0].double().cpu()
    want = score.double() + top - lse
    return (got - want).abs() - 2.0 ** -24 * want.abs()


def rows_of(kind, n, v, seed):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    z = (rand(n, 1) * 16 - 8).expand(n, v).clone()
    if kind == "flat tail":
        z[:, :: max(1, v // 7)] += 5 + 3 * rand(n, 1)
    elif kind == "flat tail far below":  # 2^-19 of the largest, as many: half of the sum
        z[:, 7] += 13 + 0.2 * rand(n)
    elif kind == "three values":
        z += (torch.randn(n, 3, generator=g) * 2).gather(1, torch.randint(0, 3, (n, v), generator=g))
    elif kind == "two in turn":
        z[:, ::2] -= 12 * rand(n, 1)
        z[:, 1] += 8
    elif kind == "one of sixteen":  # one large value in sixteen places of a thread's, the others small
        z[:, 4:] -= 4 + 8 * rand(n, 1)
        z.view(n, -1)[:, : v // 4096 * 4096].view(n, -1, 4, 1024)[:, :, 0, ::4] += 4
        z[:, 3] += 9
    elif kind == "masked tail":  # a mask's lowest value, as fp32 and bf16 have it, and -inf
        z = torch.randn(n, v, generator=g) * 3
        z[:, v // 3:] = torch.tensor([-1e4, -3.3e38, -math.inf, -80.0, -44.0])[torch.arange(n) % 5][:, None]
        z[:, 0] = 4
    elif kind == "all equal":
        pass
    elif kind == "steps":  # values an 8th apart
        z += torch.round(torch.randn(n, v, generator=g) * 20) / 8
    elif kind == "normal":
        z += torch.randn(n, v, generator=g) * (0.5 + 4 * rand(n, 1))
    return z


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [17, 1000, 8192, 32003, 151936, 622592])
@pytest.mark.parametrize("kind", ["flat tail", "flat tail far below", "three values", "two in turn", "one of sixteen", "masked tail",
                                  "all equal", "steps", "normal"])
def test_sum_of_rows_that_repeat_values(kind, v, dtype):
    n = 6 if v > 200000 else 20
    z = rows_of(kind, n, v, seed=v).to(dtype)
    e = error_of(z)
    assert (e <= 2.0 ** -27).all(), math.log2(e.max())


@pytest.mark.parametrize("offset", [-9e4, -3000.5, 3000.5, 99000.0])
def test_sum_of_rows_far_from_zero(offset):
    """Where the argument's reduction has the most to take off."""
    g = torch.Generator().manual_seed(int(abs(offset)))
    z = torch.full((16, 40000), offset) - torch.rand(16, 1, generator=g) * 10
    z[:, :3] = offset + 1 + torch.rand(16, 3, generator=g)
    z[8:] += torch.randn(8, 40000, generator=g)
    assert (error_of(z) <= 2.0 ** -27).all()


@pytest.mark.parametrize("v", [3000, 50257, 151936])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams_of_different_constants_in_the_order_of_their_totals(v, dtype):
    """Two beams, each a few large logits and a tail of one value, another one in each; totals 2^-25 apart, either way."""
    g = torch.Generator().manual_seed(v)
    wrong = []
    for i in range(24):
        z = torch.zeros(2, v)
        z[0] = 1.5 * torch.rand((), generator=g)
        z[1] = z[0, 0] + 2.0 ** -7 * (1 + torch.rand((), generator=g))
        z[:, 11:15] = 7 + torch.rand(1, 4, generator=g)
        z = z.to(dtype)
        lse, top = lse_of(z)
        best = top - lse
        score = torch.zeros(1, 2)
        score[0, 1] = (best[0] - best[1] + (1 if i % 2 else -1) * 2.0 ** -25).float()  # near 2^-7: its steps are 2^-31
        total = best + score[0].double()
        assert 2.0 ** -26 < (total[0] - total[1]).abs() < 2.0 ** -24
        got = rt.beam_select(z.to(DEV), score.to(DEV), 1)[1].item()
        wrong += [i] if got != int(total[1] > total[0]) else []
    assert not wrong
