"""The rotation's cosines and sines against float64, where the output's own rounding does not hide them.

An angle is a whole number of 2^-32 turns (cut off: up to 2 pi 2^-32 rad) that becomes fp32 in half turns below 1 (half
of a step of 2^-24, pi 2^-25 rad); cosine and sine are off by two of their own steps, 2^-23, at most.  A result
a cos - b sin is off by that of |a| + |b|, three roundings of 2^-24 of a cos and b sin, and its rounding to 16 bits,
u |out| or half of the smallest step.  (The fast functions, 2^-21 by their documentation, are past this by a fifth.)
"""
import numpy as np
import pytest

from .test_longctx_gpu import sv, torch   # noqa: F401  (fixtures)
pytestmark = pytest.mark.gpu


COSINE = np.pi * 2.0 ** -25 + 2 * np.pi * 2.0 ** -32 + 2.0 ** -23


@pytest.mark.parametrize("base", [300.0, 1.0, 1e6])
@pytest.mark.parametrize("n,interleaved", [(300, False), (300, True), (400000, False), (400000, True)])
def test_cosines_and_sines(torch, sv, n, interleaved, base):
    """Heads of (1, 0) and (0, 1) pairs: the outputs are cosines and sines, those near 0 with all their bits."""
    g = torch.Generator(device="cuda").manual_seed(n)
    pos = torch.randint(-131072, 131072, (n,), device="cuda", generator=g, dtype=torch.int32)
    rope = sv.Rope.from_base(64, base, interleaved=interleaved)
    x = torch.zeros((n, 2, 64), dtype=torch.float16, device="cuda")
    first = slice(0, 64, 2) if interleaved else slice(0, 32)
    second = slice(1, 64, 2) if interleaved else slice(32, 64)
    x[:, 0, first] = 1
    x[:, 1, second] = 1
    got = sv.qk_norm_rope(x, None, pos, rope)[0].double()
    # in float64 an angle of 2^17 rad is off by 2^-36
    angle = pos.double()[:, None] * torch.tensor([base ** (-i / 32) for i in range(32)], dtype=torch.float64, device="cuda")
    c, s = torch.cos(angle), torch.sin(angle)
    for y, want in ((got[:, 0, first], c), (got[:, 0, second], s), (got[:, 1, first], -s), (got[:, 1, second], c)):
        tol = COSINE + (2.0 ** -11 * want.abs()).clamp(min=2.0 ** -25) + 3 * 2.0 ** -24 * want.abs()
        worst = float(((y - want).abs() / tol).max())
        assert worst <= 1, worst
