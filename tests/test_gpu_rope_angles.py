"""The angles of pa_rope_and_cache at the farthest positions, against rational arithmetic."""
import math
from fractions import Fraction

import pytest
import torch

from tests.test_gpu_rope import DEV, pa  # noqa: F401

pytestmark = pytest.mark.gpu
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")  # 62 digits


def turn(position, freq):
    """position * freq radians, as the rest of a whole number of turns, in [-1/2, 1/2]."""
    t = position * Fraction(freq) / (2 * PI)
    return float(t - round(t))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("largest", [1e-3, 2.0, 300.0, 2.0 ** 53])
def test_every_position_is_as_exact_as_the_first(pa, largest, interleaved):
    """Bound: the angle is off by 2^-25 half turns for the conversion to fp32, 2^-31 for the bits
    dropped before it and 2^-32 for the fixed-point frequency, pi times as many radians (1.62 u,
    u = 2^-24); the sine and cosine of it by up to 2 ulp, at most 2 u of values up to 1; this test's
    own, in fp64, by far less.  Rows of (1, 0) pairs make the products exact."""
    gen = torch.Generator().manual_seed(5)
    R, T = 128, 24
    inv = torch.rand(R // 2, generator=gen, dtype=torch.float64) * largest
    inv[0], inv[1], inv[2], inv[3] = 0.0, 1e-300, -0.7, 5e-324
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=gen)
    pos[:5] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1, 0])
    k = torch.zeros(T, 1, R, device=DEV)
    a = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    b = a + 1 if interleaved else a + R // 2
    k[..., a.to(DEV)] = 1.0
    kb, vb = (torch.zeros(2, 16, 1, R, device=DEV) for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache(None, k, k, None, kb, vb, pos.int().to(DEV), slots, inv.to(DEV),
                         interleaved=interleaved)
    assert pa.pa_device_status() == pa.PA_OK
    got = kb.view(32, R)[:T].cpu().double()
    t = torch.tensor([[turn(p, f) for f in inv.tolist()] for p in pos.tolist()],
                     dtype=torch.float64) * (2 * math.pi)
    assert (got[:, a] - t.cos()).abs().max() <= 3.7 * 2.0 ** -24
    assert (got[:, b] - t.sin()).abs().max() <= 3.7 * 2.0 ** -24
