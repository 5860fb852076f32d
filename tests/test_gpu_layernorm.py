"""Layer norm on the GPU against the 64-bit forms of rows_ref, at the widths, strides
and alignments where its kernels change, with the bounds derived there."""
import numpy as np
import pytest
import torch

import rows_ref as ref
from rows_ref import close, draw, f64, vector

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# rows, cols, type, columns between rows, first element's place in the buffer
SHAPES = [(1, 1, BF, 0, 0), (3, 1, F32, 2, 1), (5, 7, BF, 0, 0), (2, 8, BF, 0, 0), (9, 8, F32, 8, 8),
          (33, 257, BF, 0, 3), (33, 256, BF, 8, 16), (17, 256, F32, 4, 4), (16, 1024, BF, 0, 0),
          (130, 264, F32, 0, 0), (7, 1000, BF, 1, 0), (150, 1032, BF, 0, 0), (40, 1537, F32, 0, 0),
          (301, 2048, BF, 0, 0), (19, 4096, BF, 0, 8), (5, 4104, F32, 0, 0), (6, 8191, BF, 0, 0),
          (4, 12288, BF, 0, 0), (3, 16384, F32, 0, 0), (2, 20001, BF, 0, 0), (3, 32768, BF, 0, 0),
          (2, 33000, F32, 0, 0), (2, 40008, BF, 8, 0), (1, 70001, F32, 0, 0)]
# many rows: the forward's kernels for a row a warp and a row a block, with and without
# whole warps of columns, and the backward's groups, each at its first and last widths
SHAPES += [(5001, 256, BF, 0, 0), (5001, 248, F32, 0, 0), (2601, 512, BF, 0, 0),
           (2601, 504, F32, 0, 0), (1301, 1024, BF, 0, 0), (1301, 1024, F32, 0, 0),
           (1301, 1000, BF, 0, 0), (1301, 1001, BF, 0, 0), (1001, 1032, F32, 0, 0),
           (701, 2048, BF, 8, 8), (701, 2056, BF, 0, 0), (701, 2049, F32, 0, 0),
           (331, 4096, F32, 0, 0), (331, 4104, BF, 0, 0), (311, 5120, BF, 0, 0),
           (201, 8192, BF, 0, 0), (181, 8191, F32, 0, 0), (151, 12288, BF, 0, 0),
           (121, 12296, BF, 0, 0), (101, 16384, BF, 0, 0), (99, 16385, BF, 0, 0),
           (61, 32768, F32, 0, 0), (61, 32760, BF, 0, 0)]
IDS = [f"{r}x{c}-{'bf16' if d is BF else 'fp32'}-{p}-{s}" for r, c, d, p, s in SHAPES]


def run_fwd(x, w, b, eps, **kw):
    from fp8_gemms_b200 import api
    return api.layernorm(x, w, b, eps=eps, **kw)


@pytest.mark.parametrize("rows,cols,dtype,pad,shift", SHAPES, ids=IDS)
def test_forward(rows, cols, dtype, pad, shift):
    x = draw((rows, cols), dtype, 1, 2.0, 0.5, pad, shift)
    w, b = vector(cols, dtype, 2, 0.3, 1.0), vector(cols, dtype, 3, 0.2)
    amax = torch.zeros(1, device="cuda")
    y, mean, rstd = run_fwd(x, w, b, 1e-5, amax_out=amax)
    assert y.dtype == dtype and y.shape == x.shape
    ry, rm, rr = ref.norm(f64(x), f64(w), f64(b), 1e-5)
    by, bm, br = ref.norm_bounds(f64(x), f64(w), f64(b), 1e-5, dtype)
    close(f64(mean), rm, bm, "mean")
    close(f64(rstd), rr, br, "rstd")
    close(f64(y), ry, by, "y")
    assert amax.item() == y.float().abs().max().item()
    # without the weight, the bias or either
    for wi, bi in [(None, b), (w, None), (None, None)]:
        got = run_fwd(x, wi, bi, 1e-5)[0]
        args = (f64(x), None if wi is None else f64(wi), None if bi is None else f64(bi), 1e-5)
        close(f64(got), ref.norm(*args)[0], ref.norm_bounds(*args, dtype)[0], "y")


@pytest.mark.parametrize("rows,cols,dtype,pad,shift", SHAPES, ids=IDS)
def test_backward(rows, cols, dtype, pad, shift):
    from fp8_gemms_b200 import api
    x = draw((rows, cols), dtype, 11, 2.0, 0.5, pad, shift)
    dy = draw((rows, cols), dtype, 12, 0.1, 0.01, pad, shift)
    w = vector(cols, dtype, 13, 0.3, 1.0)
    _, mean, rstd = run_fwd(x, w, None, 1e-5)
    got = api.layernorm_backward(dy, x, w, mean, rstd)
    args = (f64(dy), f64(x), f64(w), f64(mean), f64(rstd))
    want, bounds = ref.norm_grads(*args), ref.norm_grad_bounds(*args, dtype, dtype)
    for name, g, r, bd in zip(("dx", "dweight", "dbias"), got, want, bounds):
        assert g.dtype == dtype
        close(f64(g), r, bd, name)
    # added to fp32 accumulators, one at a time too; and without the weight
    acc_w, acc_b = vector(cols, F32, 14), vector(cols, F32, 15)
    w0, b0 = f64(acc_w), f64(acc_b)
    bounds = ref.norm_grad_bounds(*args, dtype, F32)
    dx, dw, db = api.layernorm_backward(dy, x, w, mean, rstd, dweight=acc_w, dbias=None,
                                        accumulate=True)
    assert db is None and torch.equal(dx, got[0])
    api.layernorm_backward(dy, x, w, mean, rstd, dbias=acc_b, accumulate=True)
    # the sum as computed, plus one fp32 addition
    close(f64(acc_w), w0 + want[1], bounds[1] + ref.U * (np.abs(w0) + np.abs(want[1])), "dw sum")
    close(f64(acc_b), b0 + want[2], bounds[2] + ref.U * (np.abs(b0) + np.abs(want[2])), "db sum")
    args = (f64(dy), f64(x), None, f64(mean), f64(rstd))
    dx = api.layernorm_backward(dy, x, None, mean, rstd)[0]
    close(f64(dx), ref.norm_grads(*args)[0], ref.norm_grad_bounds(*args, dtype, dtype)[0], "dx")


def test_large_mean_costs_no_digits():
    """x = 1000 + N(0, 1): a variance from E[x^2] - m^2 in fp32 would be off by several
    percent; the bound allows about 1e-4 of h (the mean's last digits)."""
    x = draw((64, 2000), F32, 21, 1.0, 1000.0)
    y, mean, rstd = run_fwd(x, None, None, 1e-5)
    args = (f64(x), None, None, 1e-5)
    for got, want, bound in zip((y, mean, rstd), ref.norm(*args), ref.norm_bounds(*args, F32)):
        close(f64(got), want, bound, "large mean")
    assert ref.norm_bounds(*args, F32)[0].max() < 0.05


@pytest.mark.parametrize("cols", [24, 37, 2048, 40000])
def test_constant_rows_and_rows_with_infinities_and_nan(cols):
    """A row's result depends on that row alone: one with a NaN or an infinity is NaN, a
    constant one gives the bias, the others are what they are without it.  With eps = 0
    a constant row is 0 / 0 = NaN, as the formula says."""
    x = draw((6, cols), BF, 22)
    w, b = vector(cols, BF, 23), vector(cols, BF, 24)
    want = run_fwd(x, w, b, 1e-5)[0].clone()
    x[1] = 3.0
    x[3, cols // 2] = float("inf")
    x[4, cols - 1] = float("nan")
    y, mean, rstd = run_fwd(x, w, b, 1e-5)
    assert torch.equal(y[1], b)
    assert mean[1].item() == 3.0
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    for r in (0, 2, 5):
        assert torch.equal(y[r], want[r])
    assert torch.isnan(run_fwd(x[1:2], w, b, 0.0)[0]).all()


def test_no_rows():
    from fp8_gemms_b200 import api
    x = torch.empty(0, 48, dtype=BF, device="cuda")
    w = vector(48, BF, 25)
    y, mean, rstd = run_fwd(x, w, None, 1e-5)
    assert y.shape == (0, 48) and mean.shape == rstd.shape == (0,)
    dx, dw, db = api.layernorm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 48) and not dw.any() and not db.any()
    acc = torch.ones(48, device="cuda")
    api.layernorm_backward(x, x, w, mean, rstd, dweight=acc, accumulate=True)
    assert torch.equal(acc, torch.ones_like(acc))


@pytest.mark.parametrize("cols,pad,dtype", [(136, 8, BF), (135, 1, BF), (264, 8, F32), (40001, 3, BF)])
def test_in_place_and_nothing_past_the_columns(cols, pad, dtype):
    """y over x, and dx over dy or x, give the same bits; the buffer between and behind
    the rows stays as it was."""
    from fp8_gemms_b200 import api
    rows = 21

    def fresh(seed, sigma=1.0):
        return draw((rows, cols), dtype, seed, sigma, 0.0, pad, 0)

    def edges_kept(t):
        whole = t.as_strided((rows * (cols + pad) + 64,), (1,))
        inner = torch.zeros_like(whole, dtype=torch.bool)
        inner[:rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True
        return bool(torch.isnan(whole[~inner]).all()) and bool(torch.isfinite(whole[inner]).all())

    w, b = vector(cols, dtype, 31), vector(cols, dtype, 32)
    x = fresh(33)
    y, mean, rstd = run_fwd(x, w, b, 1e-5)
    z = fresh(33)
    assert torch.equal(run_fwd(z, w, b, 1e-5, out=z)[0], y) and edges_kept(z)
    dy = fresh(34, 0.1)
    want = api.layernorm_backward(dy, x, w, mean, rstd)
    for over in ("dy", "x"):
        dyi, xi = fresh(34, 0.1), fresh(33)
        got = api.layernorm_backward(dyi, xi, w, mean, rstd, out=dyi if over == "dy" else xi)
        for g, r in zip(got, want):
            assert torch.equal(g, r), over
        assert edges_kept(dyi) and edges_kept(xi)


@pytest.mark.parametrize("rows,cols,dtype", [(3001, 520, BF), (777, 4096, BF), (513, 1537, F32)])
def test_repeats_and_replays_give_the_same_bits(rows, cols, dtype):
    """Eager again, on another stream, and replayed from two captured graphs."""
    from fp8_gemms_b200 import api
    x, dy = draw((rows, cols), dtype, 41), draw((rows, cols), dtype, 42)
    w, b = vector(cols, dtype, 43), vector(cols, dtype, 44)

    def step(**kw):
        y, mean, rstd = api.layernorm(x, w, b, **kw)
        return (y, mean, rstd, *api.layernorm_backward(dy, x, w, mean, rstd, **kw))

    eager = step()
    for a, c in zip(eager, step()):
        assert torch.equal(a, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(eager, other):
        assert torch.equal(a, c)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for _ in range(2):
        for g, outs in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for a, c in zip(eager, outs):
            assert torch.equal(a, c)
    # a replay reads what the inputs hold then
    x.mul_(0.5)
    graphs[0][0].replay()
    want = step()
    torch.cuda.synchronize()
    for a, c in zip(want, graphs[0][1]):
        assert torch.equal(a, c)


def test_gradients_against_differences_of_the_kernel():
    """<dL/dx, v> against (L(x + e v) - L(x - e v)) / 2 e of the kernel's own fp32 forward,
    L = sum(y dy): each L is off by the forward's bounds (triangle inequality over all
    outputs), so the quotient by that over e.  Rows have variance near 1 and v is +-1, so a
    third derivative of h is at most 3 |h| + 3 and its sixth, on average over a row, below
    1; 4 e^2 |dy|_1 covers the weight's spread too."""
    from fp8_gemms_b200 import api
    rows, cols, e = 8, 96, 2.0 ** -6
    x, dy, v = (draw((rows, cols), F32, s) for s in (51, 52, 53))
    w, b = vector(cols, F32, 54, 0.3, 1.0), vector(cols, F32, 55)
    v = torch.sign(v)
    _, mean, rstd = api.layernorm(x, w, b)
    dx, dw, db = api.layernorm_backward(dy, x, w, mean, rstd)

    def loss(x, w, b):
        err = (ref.norm_bounds(f64(x), f64(w), f64(b), 1e-5, F32)[0] * np.abs(f64(dy))).sum()
        return float((f64(api.layernorm(x, w, b)[0]) * f64(dy)).sum()), err

    third = 4 * e * e * np.abs(f64(dy)).sum()
    vc = torch.sign(vector(cols, F32, 56))
    for grad, direction, plus, minus in [
            (dx, v, (x + e * v, w, b), (x - e * v, w, b)),
            (dw, vc, (x, w + e * vc, b), (x, w - e * vc, b)),
            (db, vc, (x, w, b + e * vc), (x, w, b - e * vc))]:
        (lp, ep), (lm, em) = loss(*plus), loss(*minus)
        # x + e v itself is rounded to fp32: U |x| per element, of slope |grad|
        rounded = 2 * ref.U * 6 * np.abs(f64(grad)).sum() / e
        want = float((f64(grad) * f64(direction)).sum())
        assert abs((lp - lm) / (2 * e) - want) <= (ep + em) / (2 * e) + third + rounded


def test_refusals_with_device_tensors():
    from fp8_gemms_b200 import _lib, api
    x = draw((4, 32), BF, 61)
    w = vector(32, BF, 62)
    mean = torch.zeros(4, device="cuda")
    for call, status in [
            (lambda: api.layernorm(x.t()), 1),
            (lambda: api.layernorm(x[:1].expand(4, 32)), 1),
            (lambda: api.layernorm(x.half()), 4),
            (lambda: api.layernorm(x, w.float()), 1),
            (lambda: api.layernorm(x, w[:16]), 1),
            (lambda: api.layernorm(x, w, eps=-1.0), 1),
            (lambda: api.layernorm(x, w, out=x.float()), 1),
            (lambda: api.layernorm(x, w, out=x[:2]), 1),
            (lambda: api.layernorm(x, w, amax_out=w[:1]), 1),
            (lambda: api.layernorm_backward(x, x, w, mean[:3], mean), 1),
            (lambda: api.layernorm_backward(x, x, w, mean, mean.double()), 1),
            (lambda: api.layernorm_backward(x[:3], x, w, mean, mean), 1),
            (lambda: api.layernorm_backward(x, x, w, mean, mean, dweight=w, accumulate=True), 1),
            (lambda: api.layernorm_backward(x, x, w, mean, mean, dweight=w[:8]), 1)]:
        with pytest.raises(_lib.LmError) as err:
            call()
        assert err.value.status == status


def test_rows_past_two_to_the_31_elements():
    """131,080 rows of 16,392: 2^31 is passed in the last rows; those and the first are
    checked."""
    rows, cols = 131080, 16392
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    x[:4] = draw((4, cols), BF, 71)
    x[4:-4] = 0
    x[-4:] = draw((4, cols), BF, 72)
    w, b = vector(cols, BF, 73), vector(cols, BF, 74)
    y, mean, rstd = run_fwd(x, w, b, 1e-5)
    for part in (slice(0, 4), slice(rows - 4, rows)):
        args = (f64(x[part]), f64(w), f64(b), 1e-5)
        close(f64(y[part]), ref.norm(*args)[0], ref.norm_bounds(*args, BF)[0], "y")
    from fp8_gemms_b200 import api
    dx, dw, db = api.layernorm_backward(y, x, w, mean, rstd, out=y)
    assert torch.isfinite(dx[-4:]).all()
    # the rows between hold zeros: their h is 0 and their y the bias, so they add nothing
    # to dw, and b to db, each
    ends = torch.cat([x[:4], x[-4:]])
    ey, em, er = run_fwd(ends, w, b, 1e-5)
    _, want, _ = api.layernorm_backward(ey, ends, w, em, er)
    bound = (2 * ref.HALF[BF]) * np.abs(f64(want)) + 32 * ref.U * np.abs(f64(ey)).sum(0) * 8
    close(f64(dw), f64(want), bound, "dw")
