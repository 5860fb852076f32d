"""Layer norm at the ends of its documented range: rows whose centred values have squares
that just fit fp32."""
import pytest
import torch

import rows_ref as ref
from rows_ref import close, f64, vector

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# one, a few and many warps a row, with and without whole chunks
@pytest.mark.parametrize("rows,cols", [(3, 512), (3, 2048), (701, 2048), (701, 2049), (3, 8192),
                                       (331, 8192), (61, 32768), (2, 40000)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_squares_that_just_fit(dtype, rows, cols):
    """The first half of each row is +a, the rest -a, but for a few columns: the sum of the
    squares is 1e38.  A warp's sum of centred values, squared, would be up to a thousand
    times that."""
    a = (1e38 / cols) ** 0.5
    x = torch.full((rows, cols), a, dtype=dtype)
    x[:, cols // 2:] = -a
    x[:, ::97] *= 0.25
    x = x.cuda()
    w, b = vector(cols, dtype, 1, 0.3, 1.0), vector(cols, dtype, 2, 0.2)
    args = (f64(x), f64(w), f64(b), 1e-5)
    from fp8_gemms_b200 import api
    for name, got, want, bound in zip(("y", "mean", "rstd"), api.layernorm(x, w, b),
                                      ref.norm(*args), ref.norm_bounds(*args, dtype)):
        close(f64(got), want, bound, name)


@pytest.mark.parametrize("rows,cols", [(3, 512), (701, 2048), (701, 2049), (61, 32768)])
@pytest.mark.parametrize("sigma", [1e-17, 3e17 / 32768 ** 0.5])
def test_gradients_of_small_and_large_rows(rows, cols, sigma):
    """Variances of 1e-34 (with eps of 1e-37) and 1e30."""
    from fp8_gemms_b200 import api
    x, dy = ref.draw((rows, cols), F32, 3, sigma), ref.draw((rows, cols), F32, 4)
    w = vector(cols, F32, 5, 0.3, 1.0)
    y, mean, rstd = api.layernorm(x, w, None, eps=1e-37)
    args = (f64(x), f64(w), None, 1e-37)
    close(f64(y), ref.norm(*args)[0], ref.norm_bounds(*args, F32)[0], "y")
    args = (f64(dy), f64(x), f64(w), f64(mean), f64(rstd))
    got = api.layernorm_backward(dy, x, w, mean, rstd)
    for name, g, want, bound in zip(("dx", "dweight", "dbias"), got, ref.norm_grads(*args),
                                    ref.norm_grad_bounds(*args, F32, F32)):
        close(f64(g), want, bound, name)
