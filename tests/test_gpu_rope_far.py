"""Rotary positions against angles taken in 60 decimal digits: the rotation's error does
not grow with the position."""
import decimal
import math

import numpy as np
import pytest
import torch

from rows_ref import HALF, U, close, f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
D = decimal.Context(prec=60)


def two_pi():
    """2 pi = 8 (4 atan(1/5) - atan(1/239)) (Machin), from the series in integers."""
    one = 10 ** 70

    def atan_inv(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-term if k % 2 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total
    return D.divide(decimal.Decimal(8 * (4 * atan_inv(5) - atan_inv(239))), decimal.Decimal(one))


def cos_sin(positions, inv_freq):
    """[positions, frequencies] each, from the exact products reduced by whole turns."""
    turn = two_pi()
    c, s = (np.empty((len(positions), len(inv_freq))) for _ in range(2))
    for i, p in enumerate(positions):
        for j, f in enumerate(inv_freq):
            a = D.multiply(decimal.Decimal(int(p)), decimal.Decimal(float(f)))
            t = D.divide(a, turn)
            a = float(D.multiply(D.subtract(t, t.to_integral_value(context=D)), turn))
            c[i, j], s[i, j] = math.cos(a), math.sin(a)
    return c, s


FAR = [0, 99991, (1 << 29) + 3, (1 << 40) + 12345, (1 << 45) - 7, (1 << 50) + 1, (1 << 53) - 64,
       -(1 << 52) + 5]


@pytest.mark.parametrize("il", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [64, 20, 6])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_error_does_not_grow_with_the_position(dtype, rot, il):
    """The reduced half-turn is off by U of at most 1, pi U radians, wherever the position is;
    sincospif by 2 ulp, 4 U; the products with the magnitude and x and the sum by 4 U; the
    output's rounding by half a step.  rot 64, 20 and 6: 8, 2 and 1 pairs at a time."""
    from fp8_gemms_b200 import api
    freq, _ = api.rope_frequencies(rot)
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(1, len(FAR), 3, rot, generator=gen).to(dtype).cuda()
    positions = torch.tensor([FAR], device="cuda")
    c, s = (t[None, :, None, :] for t in cos_sin(FAR, f64(freq)))
    i1, i2 = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if il
              else (np.arange(rot // 2), np.arange(rot // 2, rot)))
    x64 = f64(x)
    for call, sine in ((api.rope, s), (api.rope_backward, -s)):
        want, size = np.empty_like(x64), np.empty_like(x64)
        want[..., i1] = x64[..., i1] * c - x64[..., i2] * sine
        want[..., i2] = x64[..., i2] * c + x64[..., i1] * sine
        size[..., i1] = size[..., i2] = np.abs(x64[..., i1]) + np.abs(x64[..., i2])
        bound = size * (math.pi + 8) * U
        bound += HALF[dtype] * (np.abs(want) + bound) + 1e-38
        close(f64(call([x], freq, positions=positions, interleaved=il)[0]), want, bound, "rope")
        # counted from `start`: the same angles
        for k, p in enumerate(FAR):
            one = call([x[:, k:k + 1]], freq, start=p, interleaved=il)[0]
            close(f64(one), want[:, k:k + 1], bound[:, k:k + 1], f"start {p}")
