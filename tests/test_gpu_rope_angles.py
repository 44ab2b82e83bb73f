"""Angles of kvq_norm_rope at positions up to 2^31 and frequencies of any size, against fractions of a turn to 700 digits.

Tolerance of a pair of size m: the angle is cut to 2^-32 turns and rounded to fp32, at most pi: 2^-32 2 pi + pi 2^-24; cos
and sin are off by 2 u, the products and their sum by 3 u (u = 2^-24): less than 12 u m.  At 2^31 positions the turn's
fraction is off by 2^31 2^-64 turns, 2^-30 rad, and beyond 2^38 by up to 2^31 2^-102 |f| turns."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

from gpu_util import kvq_lib, torch_cuda

pytestmark = pytest.mark.gpu

getcontext().prec = 700


def _arctan_of_one_over(n):
    total = term = Decimal(1) / n
    k = 1
    while abs(term) > Decimal(10) ** -690:
        term, k = -term / (n * n), k + 2
        total += term / k
    return total


TURN = 8 * (4 * _arctan_of_one_over(5) - _arctan_of_one_over(239))  # 2 pi (Machin)
FREQS = [1.0, -1.0, 1e-4, 10000.0 ** -0.5, 40.0, -40.0, 1e3, -1e3, 1e6, 12345678.9, 2.0 ** 38, 3e13, -7e17, 2 * math.pi,
         -2 * math.pi, math.pi, 1e-9, 0.0, 5e-324, -1e-300, 0.7071067811865476, 6.02e23, 1e-5, 999.999, -3.3e4, 17.0, 1e9, 1e10,
         -1e-7, 2.5, 250.0, 8e5]


@pytest.mark.parametrize("side", [False, True])
def test_angles(side):
    torch, kvq = torch_cuda(), kvq_lib()
    pos = [0, 1, -1, 131071, 2 ** 24 + 1, 10 ** 9 + 7, -(10 ** 9) - 9, 2 ** 31 - 1, -2 ** 31, 1999999999]
    n, half = len(pos), len(FREQS)
    rng = np.random.default_rng(3)
    x = rng.normal(size=(n, 2, 128)).astype(np.float32)
    qkv = torch.from_numpy(x.reshape(n, 256)).cuda()
    q = torch.empty(n, 2, 128, device="cuda")
    none = torch.empty(n, 0, 128, device="cuda")
    rope = kvq.Rope(FREQS, interleaved=side)
    kvq.kvq_norm_rope(qkv, torch.tensor([pos], dtype=torch.int32, device="cuda"), rope, None, None, 0.0, q, none, None)
    got = q.cpu().numpy().astype(np.float64)
    for i, f in enumerate(FREQS):
        a, b = (2 * i, 2 * i + 1) if side else (i, i + half)
        for t, p in enumerate(pos):
            turns = Decimal(f) * p / TURN
            angle = float((turns - turns.to_integral_value()) * TURN)
            c, s = math.cos(angle), math.sin(angle)
            u, v = x[t, :, a].astype(np.float64), x[t, :, b].astype(np.float64)
            off = 12 * 2.0 ** -24 + 2 * math.pi * abs(p) * max(2.0 ** -64, 2.0 ** -102 * abs(f))
            tol = off * np.hypot(u, v)
            assert (np.abs(got[t, :, a] - (u * c - v * s)) <= tol).all(), (f, p)
            assert (np.abs(got[t, :, b] - (u * s + v * c)) <= tol).all(), (f, p)
    assert (got[:, :, 2 * half:] == x[:, :, 2 * half:]).all()
