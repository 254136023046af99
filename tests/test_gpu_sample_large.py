"""Sampling over vocabularies up to the largest that a call takes, in batches on both sides of the rule for the number of
CTAs a row gets; against the 64-bit implementation, with the tolerance derived in ``test_gpu_serve``."""
import math

import pytest
import torch

from persistent_megakernel_decode_gb300 import runtime as rt
from test_gpu_serve import DEV, check_sample, settings_of, tensors_of

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from persistent_megakernel_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("B, V", [(1, 622592), (5, 622591), (17, 622592), (18, 155649), (17, 311297), (3, 262145)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_vocabularies(B, V, dtype):
    g = torch.Generator().manual_seed(V + B)
    z = (torch.randn(B, V, generator=g) * 2).to(dtype)
    z[0] = 0.0                                  # all equal: the largest sums
    if B > 2:
        z[1, ::2] = -math.inf
        z[2, 5:] = z[2, 4]                      # ties over the end of every CTA's share
    u = torch.rand(B, generator=g)
    s = settings_of(B, V + B)
    check_sample(z, u, rt.sample(z.to(DEV), u.to(DEV), **tensors_of(s)), s)
    for one in (dict(), dict(top_k=V // 3, top_p=0.75)):
        check_sample(z[:3], u[:3], rt.sample(z[:3].to(DEV), u[:3].to(DEV), **one), [one] * min(B, 3))
