"""Dropout into the residual stream, alone and fused with the layer norm after it: the mask
bit for bit against the documented generator, the values against the documented
fp32 arithmetic, the fused calls against the separate ones."""
import numpy as np
import pytest
import torch

import rows_ref as ref
from rows_ref import close, draw, f64, vector

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SEED, OFFSET = 0x9E3779B97F4A7C15, 0xFFFFFFFFFFFFFFF0   # the offset wraps with the argument
SHAPES = [(1, 1, BF, 0, 0), (7, 3, F32, 0, 0), (33, 8, BF, 0, 0), (5, 24, F32, 8, 8),
          (64, 257, BF, 3, 1), (40, 1000, BF, 0, 0), (129, 1001, BF, 0, 0), (16, 2056, F32, 0, 0),
          (21, 4096, BF, 0, 0), (3, 12288, BF, 8, 8), (2, 40001, F32, 0, 0), (2000, 16, BF, 0, 0)]
# whole tiles of four (bf16) and two (fp32) times 256 columns; rows of 3, 9 and 16 groups
# of eight, several to a warp
SHAPES += [(301, 1024, BF, 0, 0), (300, 512, F32, 8, 8), (77, 3000, BF, 0, 0), (1001, 24, BF, 0, 0),
           (333, 72, F32, 0, 0), (129, 128, BF, 8, 0), (65, 136, BF, 0, 0)]
IDS = [f"{r}x{c}-{'bf16' if d is BF else 'fp32'}-{p}-{s}" for r, c, d, p, s in SHAPES]


def rng(seed=SEED, offset=OFFSET):
    from fp8_gemms_b200 import api
    return api.dropout_rng(seed, offset)


def expected(x, p, arg, residual=None):
    """The documented result, in x's type."""
    keep, scale = ref.keep_mask(x.shape[0], x.shape[1], p, SEED, OFFSET + arg)
    y = ref.dropped(x.float().cpu().numpy(), keep, scale)
    if residual is not None:
        y = residual.float().cpu().numpy() + y
    return torch.from_numpy(y).to(x.dtype).cuda(), keep


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("rows,cols,dtype,pad,shift", SHAPES, ids=IDS)
def test_bit_for_bit(rows, cols, dtype, pad, shift, p):
    from fp8_gemms_b200 import api
    x = draw((rows, cols), dtype, 1, 1.0, 0.0, pad, shift)
    r = draw((rows, cols), dtype, 2, 2.0, 0.0, pad, shift)
    for arg in (0, 3, 1000):
        assert torch.equal(api.dropout_add(x, p, rng(), arg, residual=r),
                           expected(x, p, arg, r)[0])
    assert torch.equal(api.dropout_add(x, p, rng()), expected(x, p, 0)[0])
    assert torch.equal(api.dropout_add_backward(x, p, rng(), 3), expected(x, p, 3)[0])
    if p == 0.0:
        assert torch.equal(api.dropout_add(x, p, rng()), x)
    if p == 1.0:
        assert not api.dropout_add(x, p, rng()).any()


# widths about a warp's 127 (bf16) and 63 (fp32) aligned eights of a row, and about one eight
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 15, 17, 248, 257, 497, 504, 505, 512, 1001, 1009, 1010,
                                  1016, 1017, 1024, 2033, 5001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_start_alike_between_the_eights(dtype, cols):
    """x, residual and output at one distance past an aligned eight, row by row: each first
    row's distance, with row strides that move it on (odd) and that keep it (a multiple of
    8); then one of the three lies elsewhere.  Bit for bit; what is between the rows stays."""
    from fp8_gemms_b200 import api
    rows = 11
    for shift in range(8):
        for pad in (1 + cols % 2, -cols % 8 + 8):
            x, r = draw((rows, cols), dtype, 1, pad=pad, shift=shift), draw((rows, cols), dtype, 2, 2.0,
                                                                            pad=pad, shift=shift)
            want = expected(x, 0.4, 7, r)[0]
            for other in (0, 3):
                ld = cols + pad
                buf = torch.full((shift + other + rows * ld + 64,), float("nan"), dtype=dtype,
                                 device="cuda")
                out = buf[shift + other:shift + other + rows * ld].view(rows, ld)[:, :cols]
                api.dropout_add(x, 0.4, rng(), 7, residual=r, out=out)
                assert torch.equal(out, want), (shift, pad, other)
                api.dropout_add_backward(x, 0.4, rng(), 7, out=out)
                assert torch.equal(out, expected(x, 0.4, 7)[0]), (shift, pad, other)
                out.fill_(float("nan"))
                assert torch.isnan(buf).all(), (shift, pad, other)


@pytest.mark.parametrize("p,drop", [(2.0 ** -18, 0), (2.0 ** -16, 1), (1.5 * 2.0 ** -16, 2),
                                    (1 - 2.0 ** -16, 65535), (1 - 2.0 ** -18, 65536)])
def test_probabilities_at_the_ends(p, drop):
    from fp8_gemms_b200 import api
    assert int(np.rint(p * 65536)) == drop
    x = draw((256, 4096), F32, 3)
    got, (want, keep) = api.dropout_add(x, p, rng()), expected(x, p, 0)
    assert torch.equal(got, want)
    assert bool(got.any()) == bool(keep.any())


@pytest.mark.parametrize("cols", [64, 77])
def test_dropped_elements_contribute_nothing_whatever_they_hold(cols):
    from fp8_gemms_b200 import api
    x, r = draw((50, cols), BF, 4), draw((50, cols), BF, 5)
    keep = torch.from_numpy(ref.keep_mask(50, cols, 0.5, SEED, OFFSET)[0]).cuda()
    want = api.dropout_add(x, 0.5, rng(), residual=r)
    for bad in (float("nan"), float("inf"), float("-inf")):
        z = torch.where(keep, x, torch.full_like(x, bad))
        assert torch.equal(api.dropout_add(z, 0.5, rng(), residual=r), want)
        # and a kept one reaches its own place only
        z = x.clone()
        z[keep] = bad
        got = api.dropout_add(z, 0.5, rng(), residual=r)
        assert torch.equal(got[~keep], want[~keep]) and not torch.isfinite(got[keep]).any()


@pytest.mark.parametrize("cols,pad", [(136, 8), (135, 1)])
def test_in_place_and_nothing_past_the_columns(cols, pad):
    from fp8_gemms_b200 import api
    rows = 19
    x, r = draw((rows, cols), BF, 6, pad=pad), draw((rows, cols), BF, 7, pad=pad)
    want = api.dropout_add(x, 0.3, rng(), residual=r)
    for over in ("x", "residual"):
        xi, ri = draw((rows, cols), BF, 6, pad=pad), draw((rows, cols), BF, 7, pad=pad)
        out = xi if over == "x" else ri
        api.dropout_add(xi, 0.3, rng(), residual=ri, out=out)
        assert torch.equal(out, want)
        whole = out.as_strided((rows * (cols + pad) + 64,), (1,))
        inner = torch.zeros_like(whole, dtype=torch.bool)
        inner[:rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True
        assert torch.isnan(whole[~inner]).all() and torch.isfinite(whole[inner]).all()


def test_a_replayed_graph_takes_a_new_mask():
    """The kernel reads {seed, offset} on the device: advancing the offset between replays
    gives the masks that eager calls at those offsets give."""
    from fp8_gemms_b200 import api
    x = draw((64, 512), BF, 8)
    state = rng(5, 0)
    api.dropout_add(x, 0.4, state)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = api.dropout_add(x, 0.4, state, 2)
        state[1] += 10
    seen = []
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        want = api.dropout_add(x, 0.4, rng(5, 10 * step), 2)
        assert torch.equal(y, want)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_no_rows_and_refusals():
    from fp8_gemms_b200 import _lib, api
    x = draw((4, 32), BF, 9)
    assert api.dropout_add(x[:0], 0.5, rng()).shape == (0, 32)
    for call, status in [(lambda: api.dropout_add(x, 1.5, rng()), 1),
                         (lambda: api.dropout_add(x, -0.1, rng()), 1),
                         (lambda: api.dropout_add(x, 0.1, rng()[:1]), 1),
                         (lambda: api.dropout_add(x, 0.1, rng().int()), 1),
                         (lambda: api.dropout_add(x, 0.1, rng().cpu()), 1),
                         (lambda: api.dropout_add(x, 0.1, rng(), -1), 1),
                         (lambda: api.dropout_add(x, 0.1, rng(), residual=x[:1].expand(4, 32)), 1),
                         (lambda: api.dropout_add(x, 0.1, rng(), residual=x.float()), 1),
                         (lambda: api.dropout_add(x.half(), 0.1, rng()), 4),
                         (lambda: api.dropout_add(x.t(), 0.1, rng()), 1)]:
        with pytest.raises(_lib.LmError) as err:
            call()
        assert err.value.status == status


def test_mask_past_two_to_the_31_elements():
    from fp8_gemms_b200 import api
    rows, cols = 131080, 16392
    x = torch.ones(rows, cols, dtype=BF, device="cuda")
    api.dropout_add(x, 0.5, rng(), out=x)
    for first in (0, rows - 8):
        keep, scale = ref.keep_mask(8, cols, 0.5, SEED, OFFSET, first)
        want = torch.from_numpy(np.where(keep, scale, np.float32(0))).to(BF).cuda()
        assert torch.equal(x[first:first + 8], want)


# ------------------------------------------------- fused with the layer norm
FUSED = SHAPES + [(150, 1032, BF, 0, 0), (300, 520, BF, 0, 0), (6, 8191, BF, 0, 0),
                  (3, 32768, BF, 0, 0), (2, 33000, F32, 0, 0), (5, 8192, BF, 0, 0),
                  (5001, 256, F32, 0, 0), (2601, 512, BF, 0, 0), (1301, 1000, F32, 0, 0),
                  (1301, 1001, BF, 0, 0), (701, 2048, BF, 8, 8), (701, 2049, F32, 0, 0),
                  (331, 4096, F32, 0, 0), (311, 5120, BF, 0, 0), (201, 8192, BF, 0, 0),
                  (181, 8191, BF, 0, 0), (151, 12296, BF, 0, 0), (101, 16384, BF, 0, 0)]
FUSED_IDS = [f"{r}x{c}-{'bf16' if d is BF else 'fp32'}-{p}-{s}" for r, c, d, p, s in FUSED]


@pytest.mark.parametrize("p", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("rows,cols,dtype,pad,shift", FUSED, ids=FUSED_IDS)
def test_fused_forward(rows, cols, dtype, pad, shift, p):
    from fp8_gemms_b200 import api
    x = draw((rows, cols), dtype, 21, 1.0, 0.1, pad, shift)
    r = draw((rows, cols), dtype, 22, 2.0, -0.1, pad, shift)
    w, b = vector(cols, dtype, 23, 0.3, 1.0), vector(cols, dtype, 24, 0.2)
    amax = torch.zeros(1, device="cuda")
    s, y, mean, rstd = api.dropout_add_layernorm(x, r, w, b, p, rng(), 3, amax_out=amax)
    assert torch.equal(s, expected(x, p, 3, r)[0])
    args = (f64(s), f64(w), f64(b), 1e-5)
    for name, got, want, bound in zip(("y", "mean", "rstd"), (y, mean, rstd), ref.norm(*args),
                                      ref.norm_bounds(*args, dtype)):
        close(f64(got), want, bound, name)
    assert amax.item() == y.float().abs().max().item()


@pytest.mark.parametrize("p", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("rows,cols,dtype,pad,shift", FUSED, ids=FUSED_IDS)
def test_fused_backward(rows, cols, dtype, pad, shift, p):
    from fp8_gemms_b200 import api
    s = draw((rows, cols), dtype, 31, 2.0, 0.1, pad, shift)
    dy, ds = (draw((rows, cols), dtype, k, 0.1, 0.0, pad, shift) for k in (32, 33))
    w = vector(cols, dtype, 34, 0.3, 1.0)
    _, mean, rstd = api.layernorm(s, w, None)
    args = (f64(dy), f64(s), f64(w), f64(mean), f64(rstd))
    grads, bounds = ref.norm_grads(*args), ref.norm_grad_bounds(*args, F32, dtype)
    keep, scale = ref.keep_mask(rows, cols, p, SEED, OFFSET + 3)
    for up in (ds, None):
        dx, dr, dw, db = api.dropout_add_layernorm_backward(dy, up, s, w, mean, rstd, p, rng(), 3)
        total = grads[0] + (0.0 if up is None else f64(up))
        inner = bounds[0] + 2 * ref.U * np.abs(total)          # the sum, in fp32
        close(f64(dr), total, inner + ref.HALF[dtype] * (np.abs(total) + inner), "dresidual")
        want = np.where(keep, total * float(scale), 0.0)
        inner = (inner + 2 * ref.U * np.abs(total)) * float(scale) * keep
        close(f64(dx), want, inner + ref.HALF[dtype] * (np.abs(want) + inner), "dx")
        assert not dx[torch.from_numpy(~keep).cuda()].any()
        close(f64(dw), grads[1], bounds[1], "dweight")
        close(f64(db), grads[2], bounds[2], "dbias")


def test_fused_no_rows_accumulators_and_refusals():
    from fp8_gemms_b200 import _lib, api
    x = draw((4, 32), BF, 41)
    w = vector(32, BF, 42)
    s, y, mean, rstd = api.dropout_add_layernorm(x[:0], x[:0], w, w, 0.1, rng())
    assert s.shape == y.shape == (0, 32)
    acc = torch.ones(32, device="cuda")
    out = api.dropout_add_layernorm_backward(x[:0], None, x[:0], w, mean, rstd, 0.1, rng(),
                                             dweight=acc, accumulate=True)
    assert out[3] is None and torch.equal(acc, torch.ones_like(acc))
    mean, rstd = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    for call, status in [
            (lambda: api.dropout_add_layernorm(x, None, w, w, 0.1, rng()), 1),
            (lambda: api.dropout_add_layernorm(x, x[:2], w, w, 0.1, rng()), 1),
            (lambda: api.dropout_add_layernorm(x, x, w, w, 2.0, rng()), 1),
            (lambda: api.dropout_add_layernorm(x, x, w.float(), w, 0.1, rng()), 1),
            (lambda: api.dropout_add_layernorm_backward(x, x[:2], x, w, mean, rstd, 0.1, rng()), 1),
            (lambda: api.dropout_add_layernorm_backward(x, x, x, w, mean[:2], rstd, 0.1, rng()), 1)]:
        with pytest.raises(_lib.LmError) as err:
            call()
        assert err.value.status == status
