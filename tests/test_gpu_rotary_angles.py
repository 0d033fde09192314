"""gdn_rotary's angles, by themselves: the pair (1, 0) turns into cosine and sine, with no other
arithmetic between them and the result."""
import math

import pytest
import torch

from test_gpu_rotary import gdn  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [0, 1_000_000, 2**31 - 5000])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("what", ["every turn", "near half a turn", "near quarters"])
def test_sine_and_cosine(gdn, what, inverse, start):  # noqa: F811
    """The bound: the angle off by 2^-50 of itself and by 2^-31 turns; its rounding to fp32 moves
    sine and cosine by less than 2^-24 of themselves, the functions have two units in the last
    place (2^-22); in all 1.25 times 2^-22 of the value."""
    N, half = 4000, 64
    i = torch.arange(half, dtype=torch.float64)
    if what == "every turn":
        f = 1e4 ** (-i / half)
    elif what == "near half a turn":
        f = math.pi * (1 + 2.0 ** -21 * (i - 32))
    else:
        f = math.pi / 2 * (1 + 2.0 ** -20 * (i - 32))
    f = f.float()
    pos = torch.arange(start, start + N, dtype=torch.int64)
    x = torch.zeros(N, 1, 2 * half, device="cuda")
    x[..., 0::2] = 1
    y = gdn.gdn_rotary(x, pos.to(torch.int32).cuda(), f.cuda(), pairs=True, inverse=inverse).cpu().double()[:, 0]
    # (the product in 64 bits is off by 2^-53 of itself)
    angle = pos.double()[:, None] * f.double()
    slack = 2 * math.pi * 2.0 ** -31 + 2.0 ** -50 * angle
    for got, ref in ((y[:, 0::2], torch.cos(angle)), (y[:, 1::2], torch.sin(-angle if inverse else angle))):
        far = (got - ref).abs() - slack - 1.25 * 2.0 ** -22 * ref.abs()
        assert bool((far <= 0).all()), f"{float(far.max()):.3g} beyond the bound, at {(far == far.max()).nonzero()[0].tolist()}"
