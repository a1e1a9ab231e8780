"""GPU: rotary positions at frequencies of many turns a position, against angles reduced in exact arithmetic."""
import math
from fractions import Fraction

import numpy as np
import pytest

from layer_ops_util import U, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def _arctan_of_one_over(n, bits):
    total, k = Fraction(0), 0
    while True:
        term = Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1))
        total += term
        k += 1
        if abs(term) < Fraction(1, 1 << bits):
            return total


# 1 / (2 pi) within 2^-250, by Machin's formula
OVER_TWO_PI = 1 / (8 * (4 * _arctan_of_one_over(5, 260) - _arctan_of_one_over(239, 260)))


@pytest.mark.parametrize("far", [1000, 2 ** 20, 2 ** 31 - 1])
@pytest.mark.parametrize("scale", [1.0, 6.2831855, 100.5, 1000.3, 1e6, 3e9, 1e15])
def test_angles_of_many_turns(la, scale, far):
    """x0 cos - x1 sin and x1 cos + x0 sin of an angle that is off by pi 2^-25 (its fp32 rounding, half a unit of
    u pi) and 2 pi |position| (2^-63 + 2^-106 |freq|); cos and sin within one step (2 u each), two roundings of
    products and sum: (pi / 2 + 2 + 2) u and the second term, times |x0| + |x1|."""
    g = torch.Generator().manual_seed(int(scale) % 1000 + far % 97)
    T, P = 40, 8
    x = torch.randn(T, 1, 2 * P, generator=g)
    freq = (scale * (1 + torch.rand(P, generator=g)) * torch.where(torch.rand(P, generator=g) < 0.5, -1.0, 1.0))
    pos = torch.randint(-far, far + 1, (T,), generator=g).to(torch.int32)
    angle = np.empty((T, P))
    for t in range(T):
        for p in range(P):
            turns = Fraction(float(freq[p])) * int(pos[t]) * OVER_TWO_PI
            angle[t, p] = 2 * math.pi * float(turns - round(turns))
    c, s = np.cos(angle), np.sin(angle)
    x0, x1 = x[:, 0, :P].double().numpy(), x[:, 0, P:].double().numpy()
    ref = np.concatenate([x0 * c - x1 * s, x1 * c + x0 * s], 1)
    off = 2 * math.pi * np.abs(pos.double().numpy())[:, None] * (2.0 ** -63 + 2.0 ** -106 * np.abs(freq.double().numpy()))
    bound = ((math.pi / 2 + 4) * U + off) * (np.abs(x0) + np.abs(x1))
    got = la.la_rotary(x.cuda(), None, freq.cuda(), pos.cuda(), [P]).cpu().double().numpy()[:, 0]
    check(got, ref, np.concatenate([bound, bound], 1), "f32", "rotary")


@pytest.mark.parametrize("far", [1000, 1 << 20])
@pytest.mark.parametrize("inverse", [False, True])
def test_what_fp32_rounds_of_an_angle(la, far, inverse):
    """The pair (1, 0) turns into cos and sin themselves.  An angle is rounded beside whole quarters of a turn: by pi 2^-27,
    (pi / 8) u; each value is within a step of it, 2 u of itself.  So where one of them is almost zero it is within
    (pi / 8) u, not within the rounding of a whole turn.  (fp64 angles here are off by 2^20 2^-53 radians, 2^-9 u.)"""
    g = torch.Generator().manual_seed(far)
    T, P = 20000, 32
    x = torch.cat([torch.ones(T, 1, P), torch.zeros(T, 1, P)], -1)
    freq = (10000.0 ** (-torch.arange(P, dtype=torch.float64) / P)).float()
    pos = torch.randint(-far, far, (T,), generator=g).to(torch.int32)
    angle = pos.double()[:, None] * freq.double() * (-1 if inverse else 1)
    ref = np.concatenate([angle.cos().numpy(), angle.sin().numpy()], 1)
    bound = (math.pi / 8 + 2 ** -8) * U + 2 * U * np.abs(ref)
    got = la.la_rotary(x.cuda(), None, freq.cuda(), pos.cuda(), [P], inverse=inverse).cpu().double().numpy()[:, 0]
    check(got, ref, bound, "f32", "rotary")
