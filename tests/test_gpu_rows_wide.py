"""The row operators at the widths and sizes where their kernels' plans end: the fused fp32
calls from 4,097 to 32,768 columns, and tensors past 2^31 elements in the kernels that go over
them row by row."""
import numpy as np
import pytest
import torch

import rows_ref as ref
from rows_ref import close, draw, f64, vector

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SEED, OFFSET, P = 77, 5, 0.2


def rng():
    from fp8_gemms_b200 import api
    return api.dropout_rng(SEED, OFFSET)


# 24 warps a forward row and more; the backward's one group with two rows in shared memory, up
# to all of it (8192), its largest odd width, and the first widths of the kernels that read the
# row again
WIDE = [(311, 4104, F32), (311, 4097, F32), (301, 5120, F32), (207, 8184, F32), (201, 8192, F32),
        (31, 8200, F32), (121, 12288, F32), (121, 12296, F32), (61, 16384, F32), (40, 16385, F32),
        (31, 32760, F32), (31, 32768, F32), (9, 32776, F32), (40, 8193, BF), (40, 16383, BF),
        (31, 16392, BF), (31, 32760, BF)]
IDS = [f"{r}x{c}-{'bf16' if d is BF else 'fp32'}" for r, c, d in WIDE]


@pytest.mark.parametrize("rows,cols,dtype", WIDE, ids=IDS)
def test_fused_forward_and_backward(rows, cols, dtype):
    from fp8_gemms_b200 import api
    x, r = draw((rows, cols), dtype, 1, 1.0, 0.1), draw((rows, cols), dtype, 2, 2.0, -0.1)
    dy, ds = draw((rows, cols), dtype, 3, 0.1), draw((rows, cols), dtype, 4, 0.1)
    w, b = vector(cols, dtype, 5, 0.3, 1.0), vector(cols, dtype, 6, 0.2)
    amax = torch.zeros(1, device="cuda")
    s, y, mean, rstd = api.dropout_add_layernorm(x, r, w, b, P, rng(), 3, amax_out=amax)
    keep, scale = ref.keep_mask(rows, cols, P, SEED, OFFSET + 3)
    host = lambda t: t.float().cpu().numpy()
    want = torch.from_numpy(host(r) + ref.dropped(host(x), keep, scale)).to(dtype).cuda()
    assert torch.equal(s, want)
    args = (f64(s), f64(w), f64(b), 1e-5)
    for name, got, one, bound in zip(("y", "mean", "rstd"), (y, mean, rstd), ref.norm(*args),
                                     ref.norm_bounds(*args, dtype)):
        close(f64(got), one, bound, name)
    assert amax.item() == y.float().abs().max().item()
    args = (f64(dy), f64(s), f64(w), f64(mean), f64(rstd))
    grads, bounds = ref.norm_grads(*args), ref.norm_grad_bounds(*args, F32, dtype)
    total = grads[0] + f64(ds)
    dx, dr, dw, db = api.dropout_add_layernorm_backward(dy, ds, s, w, mean, rstd, P, rng(), 3)
    inner = bounds[0] + 2 * ref.U * np.abs(total)
    close(f64(dr), total, inner + ref.HALF[dtype] * (np.abs(total) + inner), "dresidual")
    want = np.where(keep, total * float(scale), 0.0)
    inner = (inner + 2 * ref.U * np.abs(total)) * float(scale) * keep
    close(f64(dx), want, inner + ref.HALF[dtype] * (np.abs(want) + inner), "dx")
    close(f64(dw), grads[1], bounds[1], "dweight")
    close(f64(db), grads[2], bounds[2], "dbias")
    # the same sums by the call without dropout, and the same bits again
    again = api.dropout_add_layernorm_backward(dy, ds, s, w, mean, rstd, P, rng(), 3)
    for a, c in zip(again, (dx, dr, dw, db)):
        assert torch.equal(a, c)


def picked(rows):
    """Rows at both ends, in the middle and about 2^31 elements."""
    return sorted({0, 1, 147, 148, rows // 3, rows // 2, rows - 149, rows - 3, rows - 2, rows - 1})


def large(rows, cols, seed, sigma=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(rows, cols, dtype=BF, device="cuda").normal_(0.0, sigma, generator=gen)


# 4096: rows through asynchronous copies; 4095: by scalar loads; 2^31 is passed by both
@pytest.mark.parametrize("rows,cols", [(524300, 4096), (524500, 4095)])
def test_gradients_past_two_to_the_31_elements(rows, cols):
    """Every row of x is another; dy is zero but for a few rows, so that dx is zero in the
    others and the weight gradients are the sums of those few: a row that reads another's
    operand, mean or rstd shows in each of them."""
    from fp8_gemms_b200 import api
    x, at = large(rows, cols, 1, 2.0), picked(rows)
    w = vector(cols, BF, 2, 0.3, 1.0)
    y, mean, rstd = api.layernorm(x, w, None)
    some = draw((len(at), cols), BF, 3)
    index = torch.tensor(at, device="cuda")
    args = (f64(x[index]), f64(w), None, 1e-5)
    for got, want, bound in zip((y, mean, rstd), ref.norm(*args), ref.norm_bounds(*args, BF)):
        close(f64(got[index]), want, bound, "forward")
    dy = y.zero_()
    dy[index] = some
    args = (f64(some), f64(x[index]), f64(w), f64(mean[index]), f64(rstd[index]))
    want, bounds = ref.norm_grads(*args), ref.norm_grad_bounds(*args, BF, BF)
    dx, dw, db = api.layernorm_backward(dy, x, w, mean, rstd)
    close(f64(dx[index]), want[0], bounds[0], "dx")
    close(f64(dw), want[1], bounds[1], "dweight")
    close(f64(db), want[2], bounds[2], "dbias")
    dx[index] = 0
    assert not dx.any()


@pytest.mark.parametrize("rows,cols", [(524300, 4096), (524500, 4095)])
def test_fused_past_two_to_the_31_elements(rows, cols):
    from fp8_gemms_b200 import api
    x, at = large(rows, cols, 4), picked(rows)
    res = large(rows, cols, 5, 2.0)
    w, b = vector(cols, BF, 6, 0.3, 1.0), vector(cols, BF, 7, 0.2)
    s, y, mean, rstd = api.dropout_add_layernorm(x, res, w, b, P, rng())
    assert torch.equal(s, api.dropout_add(x, P, rng(), residual=res))
    index = torch.tensor(at, device="cuda")
    keep, scale = (np.concatenate([ref.keep_mask(1, cols, P, SEED, OFFSET, r)[0] for r in at]),
                   ref.keep_mask(1, 1, P, SEED, OFFSET)[1])
    host = lambda t: t.float().cpu().numpy()
    want = torch.from_numpy(host(res[index]) + ref.dropped(host(x[index]), keep, scale)).to(BF)
    assert torch.equal(s[index].cpu(), want)
    args = (f64(s[index]), f64(w), f64(b), 1e-5)
    for got, one, bound in zip((y, mean, rstd), ref.norm(*args), ref.norm_bounds(*args, BF)):
        close(f64(got[index]), one, bound, "forward")
    del res
    # backward: dy is zero but for those rows, ds everywhere
    ds, dy = x, y.zero_()
    dy[index] = draw((len(at), cols), BF, 8, 0.1)
    dx, dr, dw, db = api.dropout_add_layernorm_backward(dy, ds, s, w, mean, rstd, P, rng())
    args = (f64(dy[index]), f64(s[index]), f64(w), f64(mean[index]), f64(rstd[index]))
    grads, bounds = ref.norm_grads(*args), ref.norm_grad_bounds(*args, F32, BF)
    total = grads[0] + f64(ds[index])
    inner = bounds[0] + 2 * ref.U * np.abs(total)
    close(f64(dr[index]), total, inner + ref.HALF[BF] * (np.abs(total) + inner), "dresidual")
    want = np.where(keep, total * float(scale), 0.0)
    inner = (inner + 2 * ref.U * np.abs(total)) * float(scale) * keep
    close(f64(dx[index]), want, inner + ref.HALF[BF] * (np.abs(want) + inner), "dx")
    close(f64(dw), grads[1], bounds[1], "dweight")
    close(f64(db), grads[2], bounds[2], "dbias")
    # the other rows: dresidual is ds as it is, dx its dropout
    plain = api.dropout_add_backward(ds, P, rng())
    for got, one in ((dr, ds), (dx, plain)):
        got[index] = one[index]
        assert torch.equal(got, one)


@pytest.mark.parametrize("residual", [False, True])
def test_dropout_of_odd_widths_past_two_to_the_31_elements(residual):
    from fp8_gemms_b200 import api
    rows, cols = 524500, 4095
    x = large(rows, cols, 9)
    res = large(rows, cols, 10) if residual else None
    got = api.dropout_add(x, P, rng(), residual=res)
    host = lambda t: t.float().cpu().numpy()
    for r in picked(rows):
        keep, scale = ref.keep_mask(1, cols, P, SEED, OFFSET, r)
        want = ref.dropped(host(x[r:r + 1]), keep, scale)
        if residual:
            want = host(res[r:r + 1]) + want
        assert torch.equal(got[r:r + 1].cpu(), torch.from_numpy(want).to(BF)), r
    # every row against the same rows as tensors of their own cannot be told by the mask, which
    # goes by the row's number; but by what a kept element is: x scale (+ residual) or residual
    rest = res if residual else torch.zeros((), dtype=BF, device="cuda")
    for k in range(0, rows, 65536):
        part = slice(k, k + 65536)
        base = rest[part].float() if residual else rest.float()
        kept = (base + x[part].float() * float(scale)).to(BF)
        assert ((got[part] == kept) | (got[part] == base.to(BF))).all(), k
