"""Forms of the row operators' and rotary calls that are documented: outputs over inputs in the
fused calls, outputs laid out unlike the inputs, amax of values that are not finite, weights left
out, accumulators, the generator's state as unsigned integers, many heads and whole heads of
512."""
import itertools

import numpy as np
import pytest
import torch

import rows_ref as ref
from rows_ref import close, draw, f64, vector

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# few rows; a row a warp; whole and broken chunks; scalar accesses; rows read again
SHAPES = [(5, 768, BF), (301, 512, BF), (301, 504, F32), (700, 2048, BF), (150, 5120, BF),
          (65, 777, BF), (33, 1001, F32), (20, 8192, F32), (3, 40001, BF), (3, 40008, F32)]
IDS = [f"{r}x{c}-{'bf16' if d is BF else 'fp32'}" for r, c, d in SHAPES]


@pytest.mark.parametrize("rows,cols,dtype", SHAPES, ids=IDS)
def test_fused_outputs_over_inputs(rows, cols, dtype):
    """S over x or residual, Y over the one that S is not over: the same bits as apart."""
    from fp8_gemms_b200 import _lib, api
    w, b = vector(cols, dtype, 1, 0.3, 1.0), vector(cols, dtype, 2, 0.2)
    rng = api.dropout_rng(3)

    def inputs():
        return {"x": draw((rows, cols), dtype, 4), "res": draw((rows, cols), dtype, 5, 2.0)}
    t = inputs()
    want = api.dropout_add_layernorm(t["x"], t["res"], w, b, 0.3, rng)
    for s_at, y_at in itertools.product(("x", "res", None), repeat=2):
        if s_at == y_at:
            continue
        t = inputs()
        S = torch.empty_like(t["x"]) if s_at is None else t[s_at]
        Y = torch.empty_like(t["x"]) if y_at is None else t[y_at]
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        _lib.lm_dropout_add_layernorm_fwd(t["x"], t["res"], w, b, S, Y, 0.3, rng, 0, mean, rstd)
        for got, one in zip((S, Y, mean, rstd), want):
            assert torch.equal(got, one), (s_at, y_at)


@pytest.mark.parametrize("rows,cols,dtype", SHAPES, ids=IDS)
def test_fused_gradients_over_inputs(rows, cols, dtype):
    """dX and dR each over dY, dS or S, or apart."""
    from fp8_gemms_b200 import _lib, api
    w, rng = vector(cols, dtype, 1, 0.3, 1.0), api.dropout_rng(3)

    def inputs():
        return {"dy": draw((rows, cols), dtype, 4, 0.1), "ds": draw((rows, cols), dtype, 5, 0.1),
                "s": draw((rows, cols), dtype, 6, 2.0)}
    t = inputs()
    _, mean, rstd = api.layernorm(t["s"], w)
    want = api.dropout_add_layernorm_backward(t["dy"], t["ds"], t["s"], w, mean, rstd, 0.3, rng)
    ws = torch.empty(_lib.lm_layernorm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    for dx_at, dr_at in itertools.product(("dy", "ds", "s", None), repeat=2):
        if dx_at == dr_at:
            continue
        t = inputs()
        dx = torch.empty_like(t["s"]) if dx_at is None else t[dx_at]
        dr = torch.empty_like(t["s"]) if dr_at is None else t[dr_at]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        _lib.lm_dropout_add_layernorm_bwd(t["dy"], t["ds"], t["s"], w, mean, rstd, 0.3, rng, dx, dr,
                                          dw, db, ws)
        for got, one in zip((dx, dr, dw, db), want):
            assert torch.equal(got, one), (dx_at, dr_at)


@pytest.mark.parametrize("rows,cols,dtype", SHAPES, ids=IDS)
def test_outputs_laid_out_unlike_the_inputs(rows, cols, dtype):
    """Row strides and first elements of their own; what is between stays."""
    from fp8_gemms_b200 import api
    x, dy = draw((rows, cols), dtype, 1), draw((rows, cols), dtype, 2, pad=8)
    w, b, rng = vector(cols, dtype, 3, 0.3, 1.0), vector(cols, dtype, 4), api.dropout_rng(5)
    y, mean, rstd = api.layernorm(x, w, b)
    back = api.layernorm_backward(dy, x, w, mean, rstd)
    drop = api.dropout_add(x, 0.3, rng, residual=dy)

    for pad, shift in ((8, 8), (3, 0), (16, 5)):
        ld = cols + pad
        buf = torch.full((shift + rows * ld + 64,), float("nan"), dtype=dtype, device="cuda")
        out = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
        # scalar accesses sum a row in another order than wide ones
        got = api.layernorm(x, w, b, out=out)
        args = (f64(x), f64(w), f64(b), 1e-5)
        for a, one, bound in zip(got, ref.norm(*args), ref.norm_bounds(*args, dtype)):
            close(f64(a), one, bound, "forward")
        args = (f64(dy), f64(x), f64(w), f64(mean), f64(rstd))
        got = api.layernorm_backward(dy, x, w, mean, rstd, out=out)
        for a, one, bound in zip(got, ref.norm_grads(*args),
                                 ref.norm_grad_bounds(*args, dtype, dtype)):
            close(f64(a), one, bound, "backward")
        api.dropout_add(x, 0.3, rng, residual=dy, out=out)
        assert torch.equal(out, drop)
        out.fill_(float("nan"))
        assert torch.isnan(buf).all()
    assert torch.isfinite(y).all() and torch.isfinite(back[0]).all()


@pytest.mark.parametrize("rows,cols,dtype", SHAPES, ids=IDS)
def test_amax_goes_on_from_what_it_holds(rows, cols, dtype):
    """The largest of it and |y|; infinite and NaN values of y are above all."""
    from fp8_gemms_b200 import api
    x, r, rng = draw((rows, cols), dtype, 1), draw((rows, cols), dtype, 2), api.dropout_rng(5)
    w, b = vector(cols, dtype, 3, 0.3, 1.0), vector(cols, dtype, 4)
    calls = [lambda b, amax: api.layernorm(x, w, b, amax_out=amax)[0],
             lambda b, amax: api.dropout_add_layernorm(x, r, w, b, 0.3, rng, amax_out=amax)[1]]
    for call in calls:
        top = call(b, None).float().abs().max().item()
        for held in (0.0, top / 2, top * 2):
            amax = torch.full((1,), held, device="cuda")
            call(b, amax)
            assert amax.item() == max(held, top)
        bad = b.clone()
        bad[cols // 2] = float("-inf")
        amax = torch.zeros(1, device="cuda")
        call(bad, amax)
        assert amax.item() == float("inf")
        bad[cols - 1] = float("nan")
        call(bad, amax)
        assert torch.isnan(amax).all()


@pytest.mark.parametrize("rows,cols,dtype", SHAPES, ids=IDS)
def test_fused_without_weights_and_into_accumulators(rows, cols, dtype):
    from fp8_gemms_b200 import api
    x, r = draw((rows, cols), dtype, 1), draw((rows, cols), dtype, 2)
    dy, ds, rng = draw((rows, cols), dtype, 3), draw((rows, cols), dtype, 4), api.dropout_rng(5)
    w, b = vector(cols, dtype, 6, 0.3, 1.0), vector(cols, dtype, 7)
    for wi, bi in ((None, b), (w, None), (None, None)):
        s, y, mean, rstd = api.dropout_add_layernorm(x, r, wi, bi, 0.3, rng)
        args = (f64(s), None if wi is None else f64(wi), None if bi is None else f64(bi), 1e-5)
        for got, one, bound in zip((y, mean, rstd), ref.norm(*args), ref.norm_bounds(*args, dtype)):
            close(f64(got), one, bound, "forward")
    args = (f64(dy), f64(s), None, f64(mean), f64(rstd))
    grads, bounds = ref.norm_grads(*args), ref.norm_grad_bounds(*args, F32, F32)
    acc = [vector(cols, F32, 8), vector(cols, F32, 9)]
    before = [f64(a) for a in acc]
    dx, dr, dw, db = api.dropout_add_layernorm_backward(dy, ds, s, None, mean, rstd, 0.3, rng,
                                                        dweight=acc[0], dbias=acc[1],
                                                        accumulate=True)
    assert dw is acc[0] and db is acc[1]
    total = grads[0] + f64(ds)
    inner = bounds[0] + 2 * ref.U * np.abs(total)
    close(f64(dr), total, inner + ref.HALF[dtype] * (np.abs(total) + inner), "dresidual")
    for a, was, g, bound in zip(acc, before, grads[1:], bounds[1:]):
        close(f64(a), was + g, bound + ref.U * (np.abs(was) + np.abs(g)), "accumulator")


def test_state_as_unsigned_integers():
    from fp8_gemms_b200 import api
    x, rng = draw((9, 80), BF, 1), api.dropout_rng(1 << 63, 7)
    assert torch.equal(api.dropout_add(x, 0.5, rng.view(torch.uint64), 2), api.dropout_add(x, 0.5, rng, 2))


@pytest.mark.parametrize("il", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,heads,d,rot", [(1, 5000, 64, 64), (3, 3001, 20, 12), (2, 4097, 8, 6),
                                                (5, 3, 512, 512), (5, 3, 512, 508), (5, 3, 512, 510),
                                                (1500, 2, 512, 510), (2, 65536, 2, 2)])
def test_many_heads_and_wide_ones(tokens, heads, d, rot, dtype, il):
    from fp8_gemms_b200 import api
    gen = torch.Generator().manual_seed(1)
    x, k = (torch.randn(1, tokens, h, d, generator=gen).to(dtype).cuda() for h in (heads, 1))
    freq, mag = api.rope_frequencies(rot)
    pos = np.arange(tokens)[None] + 9
    # out: heads before tokens, with elements between the heads
    out = [torch.zeros(1, t.shape[2], tokens, d + 3, dtype=dtype, device="cuda")[..., 1:d + 1].transpose(1, 2)
           for t in (x, k)]
    for got in (api.rope([x, k], freq, start=9, interleaved=il),
                api.rope([x, k], freq, start=9, interleaved=il, out=out)):
        for t, y in zip((x, k), got):
            f = f64(freq)
            close(f64(y), ref.rope(f64(t), f, pos, il, mag),
                  ref.rope_bound(f64(t), f, pos, il, mag, dtype), "rope")
            assert torch.equal(y[..., rot:], t[..., rot:])
    for y in out:
        assert not y._base[..., 0].any() and not y._base[..., d + 1:].any()
