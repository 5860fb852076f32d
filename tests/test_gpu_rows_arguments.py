"""What the row operators' and rotary calls take for a stream and for whole numbers."""
import numpy as np
import pytest
import torch

from rows_ref import draw, vector

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def calls(stream):
    from fp8_gemms_b200 import api
    x, r, w = draw((40, 264), BF, 1), draw((40, 264), BF, 2), vector(264, BF, 3)
    q = draw((6, 64), BF, 4).view(1, 3, 2, 64)
    freq, _ = api.rope_frequencies(64)
    rng = api.dropout_rng(5)
    y, mean, rstd = api.layernorm(x, w, w)
    torch.cuda.synchronize()
    out = [*api.layernorm(x, w, w, stream=stream),
           *api.layernorm_backward(r, x, w, mean, rstd, stream=stream),
           api.dropout_add(x, 0.2, rng, residual=r, stream=stream),
           api.dropout_add_backward(x, 0.2, rng, stream=stream),
           *api.dropout_add_layernorm(x, r, w, w, 0.2, rng, stream=stream),
           *api.dropout_add_layernorm_backward(r, r, x, w, mean, rstd, 0.2, rng, stream=stream),
           *api.rope([q], freq, stream=stream), *api.rope_backward((q,), freq, stream=stream)]
    torch.cuda.synchronize()
    return out


def test_a_raw_stream_handle():
    """As every other call takes one: a torch stream, the integer handle of one, and 0 for
    the default stream."""
    want = calls(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        for got, ref in zip(calls(stream), want):
            assert torch.equal(got, ref), stream


def test_a_stream_and_a_generator_of_tensors():
    from fp8_gemms_b200 import api
    q = draw((6, 64), BF, 4).view(1, 3, 2, 64)
    freq, _ = api.rope_frequencies(64)
    want = api.rope([q], freq)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = api.rope((t for t in [q]), freq, stream=side.cuda_stream)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for call in (lambda: api.rope([], freq, stream=side), lambda: api.layernorm(None, stream=side),
                 lambda: api.rope([q.cpu()], freq, stream=0)):
        with pytest.raises(api.LmError) as e:
            call()
        assert e.value.status == 1


def test_work_on_a_raw_handle_is_on_that_stream():
    """Captured: a graph of a stream holds what was put on it by its handle."""
    from fp8_gemms_b200 import api
    x, w = draw((40, 264), BF, 1), vector(264, BF, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = api.layernorm(x, w, stream=side.cuda_stream)[0]
    x.mul_(-2.0)
    g.replay()
    want = api.layernorm(x, w)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients_side_by_side_in_one_buffer(accumulate):
    """One behind the other they are as elsewhere; with elements in common, refused."""
    from fp8_gemms_b200 import api
    dy, x, w = draw((40, 264), BF, 1), draw((40, 264), BF, 2), vector(264, BF, 3)
    _, mean, rstd = api.layernorm(x, w)
    buf = torch.ones(2 * 264 + 8, dtype=torch.float32 if accumulate else BF, device="cuda")

    def back(dw, db):
        return api.layernorm_backward(dy, x, w, mean, rstd, dweight=dw, dbias=db,
                                      accumulate=accumulate)
    want = [t.clone() for t in back(buf[:264].clone(), buf[264:528].clone())]
    got = back(buf[:264], buf[264:528])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (buf[528:] == 1).all()
    before = buf.clone()
    for dw, db in ((0, 0), (8, 0), (0, 263), (264, 1)):
        with pytest.raises(api.LmError) as e:
            back(buf[dw:dw + 264], buf[db:db + 264])
        assert e.value.status == 1
    assert torch.equal(buf, before)


@pytest.mark.parametrize("kind", [np.int64, np.uint64, torch.tensor])
def test_offsets_of_any_integer_type(kind):
    from fp8_gemms_b200 import api
    x, rng = draw((9, 80), BF, 1), api.dropout_rng(5)
    assert torch.equal(api.dropout_add(x, 0.5, rng, offset=kind(3)), api.dropout_add(x, 0.5, rng, offset=3))
    for bad in (3.0, "3", -1, 1 << 64, None):
        with pytest.raises(api.LmError) as e:
            api.dropout_add(x, 0.5, rng, offset=bad)
        assert e.value.status == 1
