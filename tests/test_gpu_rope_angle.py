"""Cosines and sines of the rotation, read off fp32 unit vectors, to a few ulp of themselves:
also where the angle is near a multiple of a quarter turn and one of them is small."""
import numpy as np
import pytest
import torch

from rows_ref import U, close, f64
from test_gpu_rope_far import cos_sin

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("il", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 20, 6])
def test_small_coefficients_keep_their_digits(rot, il):
    """sincospif is good to 2 ulp of its value, 4 U, at an angle held in fp32; what that leaves
    of the angle, at most 2^-24 of a half-turn, is brought in by one product and sum, U; the
    magnitude of 1 and the sum with the other element's 0 are exact.  The rest's own roundings
    and its square, 3 U and 2^-24 of it, are below 4e-14, the fp64 angle's below 1e-15."""
    from fp8_gemms_b200 import api
    freq, _ = api.rope_frequencies(rot, theta=10000.0)
    # positions whose first angles (frequency 1) are near quarter turns, and others
    pos = [1, 2, 3, 11, 22, 33, 44, 333, 344, 355, 710, 51819, 52174, 103993, 104348, 208341, 312689,
           833719, 77, 1000, 4097, 65537]
    c, s = cos_sin(pos, f64(freq))
    half = rot // 2
    x = torch.zeros(1, len(pos), 1, rot, device="cuda")
    x[..., 0::2 if il else 1][..., :half] = 1.0        # (1, 0): turns to (cos, sin)
    y = f64(api.rope([x], freq, positions=torch.tensor([pos], device="cuda"), interleaved=il)[0])
    y = y[0, :, 0]
    got_c, got_s = (y[:, 0::2], y[:, 1::2]) if il else (y[:, :half], y[:, half:])
    for name, got, want in (("cos", got_c, c), ("sin", got_s, s)):
        close(got, want, 5 * U * np.abs(want) + 4e-14, name)
