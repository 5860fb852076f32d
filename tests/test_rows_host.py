"""Host side of the row operators (layer norm, dropout, rotary positions): the
reference generator's published vectors, the frequency helper against its
formulas, and the refusals of the C entry points and of the Python calls.  No
GPU: every refused call fails a host check before any launch."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import rows_ref as ref

FAKE = 0x10000   # never dereferenced
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    from fp8_gemms_b200 import _lib
    return _lib


def test_philox_known_answers():
    """The published known answers of Philox4x32-10."""
    def words(counter, key):
        return [int(w) for w in ref.philox4x32_10(counter, key)]
    assert words([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ff = 0xFFFFFFFF
    assert words([ff] * 4, [ff] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_rate_and_independence_of_offsets():
    keep, scale = ref.keep_mask(512, 1000, 0.3, 1234567890123, 7)
    n = keep.size
    q = 1.0 - round(0.3 * 65536) / 65536
    assert abs(keep.mean() - q) <= 6 * math.sqrt(q * (1 - q) / n)
    assert scale == np.float32(1 / q)
    other, _ = ref.keep_mask(512, 1000, 0.3, 1234567890123, 8)
    both = (keep & other).mean()
    assert abs(both - q * q) <= 6 * math.sqrt(q * q * (1 - q * q) / n)


def test_rope_frequencies(L):
    rot, theta = 64, 10000.0
    base = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    f, m = L.lm_rope_inv_freq(rot, theta)
    assert m == 1.0 and np.allclose(f, base, rtol=1e-14, atol=0)
    f, m = L.lm_rope_inv_freq(rot, theta, L.ROPE_LINEAR, 4.0)
    assert m == 1.0 and np.allclose(f, [b / 4 for b in base], rtol=1e-14, atol=0)
    f, m = L.lm_rope_inv_freq(rot, theta, L.ROPE_NTK, 4.0)
    t = theta * 4.0 ** (rot / (rot - 2))
    assert m == 1.0 and np.allclose(f, [t ** (-2 * i / rot) for i in range(rot // 2)], rtol=1e-13,
                                    atol=0)
    # NTK: the slowest pair is that of the interpolated positions
    assert math.isclose(f[-1], base[-1] / 4, rel_tol=1e-12)
    f, m = L.lm_rope_inv_freq(rot, theta, L.ROPE_BY_PARTS, 8.0, 2048.0, 1.0, 32.0)
    assert math.isclose(m, 0.1 * math.log(8.0) + 1.0, rel_tol=1e-7)
    for got, b in zip(f, base):
        turns = 2048.0 * b / (2 * math.pi)
        if turns >= 32:
            assert math.isclose(got, b, rel_tol=1e-14)
        elif turns <= 1:
            assert math.isclose(got, b / 8, rel_tol=1e-14)
        else:
            assert b / 8 < got < b
    assert L.lm_rope_inv_freq(0) == ([], 1.0)


def test_rope_frequency_refusals(L):
    for args in [(63,), (-2,), (64, 0.0), (64, float("nan")), (64, 1e4, L.ROPE_LINEAR, 0.5),
                 (64, 1e4, L.ROPE_LINEAR, float("inf")), (2, 1e4, L.ROPE_NTK, 2.0),
                 (64, 1e4, L.ROPE_BY_PARTS, 2.0, 0.0), (64, 1e4, L.ROPE_BY_PARTS, 2.0, 9.0, 3.0, 3.0)]:
        with pytest.raises(L.LmError) as e:
            L.lm_rope_inv_freq(*args)
        assert e.value.status == 1
    with pytest.raises(L.LmError) as e:
        L.lm_rope_inv_freq(64, 1e4, 9, 2.0)
    assert e.value.status == 4


def test_layernorm_fwd_refusals(L):
    def call(x=FAKE, ldx=64, w=FAKE, b=FAKE, rows=4, cols=64, eps=1e-5, dt=BF16, y=FAKE, ldy=64,
             mean=FAKE, rstd=FAKE, amax=None):
        return L.lib.lm_layernorm_fwd(x, ldx, w, b, rows, cols, eps, dt, y, ldy, mean, rstd, amax,
                                      None)
    assert call(rows=0) == 0 and call(rows=0, x=None, y=None) == 0
    assert call(dt=7) == 4
    for bad in [dict(x=None), dict(y=None), dict(rows=-1), dict(cols=0), dict(cols=-8),
                dict(eps=-1.0), dict(eps=float("nan")), dict(ldx=63), dict(ldy=0), dict(ldy=-64),
                dict(ldy=72)]:   # y over x with another stride
        assert call(**bad) == 1, bad
    for bad in [dict(x=FAKE + 1), dict(y=FAKE + 1), dict(w=FAKE + 1), dict(mean=FAKE + 2),
                dict(rstd=FAKE + 1), dict(amax=FAKE + 2), dict(x=FAKE + 2, dt=F32)]:
        assert call(**bad) == 2, bad
    for bad in [dict(rows=1 << 31), dict(cols=1 << 31, ldx=1 << 31, ldy=1 << 31),
                dict(ldx=1 << 31)]:
        assert call(**bad) == 3, bad


def test_layernorm_bwd_refusals(L):
    n = L.lm_layernorm_workspace_size(4, 64)
    assert n >= 4 * 2 * 64 * 4
    assert L.lm_layernorm_workspace_size(-1, 64) == 0 == L.lm_layernorm_workspace_size(4, 0)
    # bounded in the rows: partial sums, not a copy of the tensor
    assert L.lm_layernorm_workspace_size(1 << 20, 64) == L.lm_layernorm_workspace_size(1 << 24, 64)

    def call(dy=FAKE, lddy=64, x=FAKE, ldx=64, w=FAKE, mean=FAKE, rstd=FAKE, rows=4, cols=64,
             dt=BF16, dx=FAKE, lddx=64, dw=FAKE, db=FAKE, ws=FAKE, nb=n, flags=0):
        return L.lib.lm_layernorm_bwd(dy, lddy, x, ldx, w, mean, rstd, rows, cols, dt, dx, lddx, dw,
                                      db, ws, nb, flags, None)
    assert call(dt=-1) == 4
    for bad in [dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None),
                dict(flags=2), dict(ws=None), dict(nb=n - 1), dict(rows=-1), dict(cols=0),
                dict(lddx=32), dict(lddy=32)]:
        assert call(**bad) == 1, bad
    for bad in [dict(ws=FAKE + 8), dict(dw=FAKE + 1), dict(dw=FAKE + 2, flags=1),
                dict(db=FAKE + 2, dt=F32), dict(mean=FAKE + 1), dict(dx=FAKE + 1)]:
        assert call(**bad) == 2, bad
    # nothing to write: no rows and no weight gradients
    assert call(rows=0, dw=None, db=None, ws=None, nb=0) == 0
    # an accumulator gets nothing from no rows
    assert call(rows=0, flags=1) == 0


def test_dropout_refusals(L):
    def call(x=FAKE, ldx=64, r=FAKE, ldr=64, rows=4, cols=64, dt=BF16, p=0.1, rng=FAKE, off=0,
             y=FAKE, ldy=64):
        return L.lib.lm_dropout_add_fwd(x, ldx, r, ldr, rows, cols, dt, p, rng, off, y, ldy, None)
    assert call(rows=0) == 0
    assert call(dt=2) == 4
    for bad in [dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(rng=None), dict(x=None),
                dict(y=None), dict(rows=-1), dict(cols=0), dict(ldr=0), dict(ldx=1), dict(ldy=80)]:
        assert call(**bad) == 1, bad
    for bad in [dict(rng=FAKE + 4), dict(x=FAKE + 1), dict(r=FAKE + 1), dict(y=FAKE + 2, dt=F32)]:
        assert call(**bad) == 2, bad
    bwd = L.lib.lm_dropout_add_bwd
    assert bwd(FAKE, 64, 0, 64, BF16, 0.1, FAKE, 0, FAKE, 64, None) == 0
    assert bwd(FAKE, 64, 4, 64, BF16, 0.1, None, 0, FAKE, 64, None) == 1
    assert bwd(None, 64, 4, 64, BF16, 0.1, FAKE, 0, FAKE, 64, None) == 1


def test_dropout_layernorm_refusals(L):
    def fwd(x=FAKE, r=FAKE, s=FAKE, y=FAKE + 0x10000, p=0.1, rng=FAKE, lds=64, rows=4):
        return L.lib.lm_dropout_add_layernorm_fwd(x, 64, r, 64, FAKE, FAKE, rows, 64, 1e-5, BF16, p,
                                                  rng, 0, s, lds, y, 64, FAKE, FAKE, None, None)
    assert fwd(rows=0) == 0
    for bad in [dict(x=None), dict(r=None), dict(s=None), dict(y=None), dict(p=2.0), dict(rng=None),
                dict(lds=8)]:
        assert fwd(**bad) == 1, bad
    assert fwd(s=FAKE + 1) == 2
    assert fwd(y=FAKE) == 1                       # y where s is
    n = L.lm_layernorm_workspace_size(4, 64)

    def bwd(dy=FAKE, ds=FAKE, s=FAKE, dx=FAKE, dr=FAKE + 0x10000, p=0.1, rng=FAKE, ws=FAKE, nb=n):
        return L.lib.lm_dropout_add_layernorm_bwd(dy, 64, ds, 64, s, 64, FAKE, FAKE, FAKE, 4, 64,
                                                  BF16, p, rng, 0, dx, 64, dr, 64, FAKE, FAKE, ws,
                                                  nb, 0, None)
    for bad in [dict(dy=None), dict(s=None), dict(dx=None), dict(dr=None), dict(p=-1.0),
                dict(rng=None), dict(ws=None), dict(nb=n - 1), dict(dr=FAKE)]:
        assert bwd(**bad) == 1, bad
    assert bwd(ds=FAKE + 1) == 2 and bwd(rng=FAKE + 4) == 2


def test_rope_refusals(L):
    def tensor(x=FAKE, y=FAKE + 0x100000, heads=4, xs=(2048, 256, 64), ys=(2048, 256, 64)):
        return L.RopeTensor(x, y, heads, *xs, *ys)

    def call(ts=None, count=None, batch=2, seq=8, dim=64, rot=64, dt=BF16, freq=FAKE, pos=None,
             start=0, mag=1.0, flags=0):
        ts = [tensor()] if ts is None else ts
        arr = (L.RopeTensor * max(1, len(ts)))(*ts)
        return L.lib.lm_rope(arr, len(ts) if count is None else count, batch, seq, dim, rot, dt,
                             freq, pos, start, mag, flags, None)
    assert call(batch=0) == 0 and call(seq=0) == 0 and call(ts=[tensor(heads=0)]) == 0
    assert call(dt=5) == 4
    for bad in [dict(count=0), dict(count=3), dict(batch=-1), dict(seq=-1), dict(dim=0),
                dict(rot=63), dict(rot=66), dict(rot=-2), dict(flags=4), dict(freq=None),
                dict(mag=float("nan")), dict(mag=float("inf")), dict(ts=[tensor(x=None)]),
                dict(ts=[tensor(y=None)]), dict(ts=[tensor(heads=-1)]),
                dict(ts=[tensor(xs=(2048, -256, 64))]),
                # outputs that overlap: heads 32 apart, one row for all tokens, batches folded
                dict(ts=[tensor(ys=(2048, 256, 32))]), dict(ts=[tensor(ys=(2048, 0, 64))]),
                dict(ts=[tensor(ys=(1024, 256, 64))]), dict(ts=[tensor(ys=(2048, 256, -64))]),
                # one output for both, an output over the other's input
                dict(ts=[tensor(), tensor(x=FAKE + 0x300000)]),
                dict(ts=[tensor(), tensor(x=FAKE + 0x300000, y=FAKE)]),
                dict(ts=[tensor(), tensor(x=FAKE + 0x100000, y=FAKE + 0x300000)]),
                dict(start=(1 << 63) - 5),
                # in place with other strides
                dict(ts=[tensor(y=FAKE, xs=(2048, 64, 512))])]:
        assert call(**bad) == 1, bad
    for bad in [dict(ts=[tensor(x=FAKE + 1)]), dict(ts=[tensor(y=FAKE + 1)]), dict(freq=FAKE + 4),
                dict(pos=FAKE + 4), dict(ts=[tensor(x=FAKE + 2)], dt=F32)]:
        assert call(**bad) == 2, bad
    for bad in [dict(batch=1 << 31), dict(batch=1 << 20, seq=1 << 20), dict(dim=1 << 17, rot=64),
                dict(ts=[tensor(heads=1 << 30)])]:
        assert call(**bad) == 3, bad


def test_python_calls_refuse_what_they_cannot_run(L):
    """The Python calls refuse host tensors, other types and other ranks by name
    (shapes and strides that need a CUDA tensor are tested with the kernels)."""
    from fp8_gemms_b200 import api
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    rng = torch.zeros(2, dtype=torch.int64)
    freq = torch.ones(8, dtype=torch.float64)
    for call in [lambda: api.layernorm(x), lambda: api.layernorm(x[0]),
                 lambda: api.layernorm_backward(x, x, None, x[:, 0].float(), x[:, 0].float()),
                 lambda: api.layernorm_backward(x[0], x[0], None, x[0].float(), x[0].float()),
                 lambda: api.layernorm(x[0, 0]),
                 lambda: api.dropout_add(x, 0.1, rng), lambda: api.dropout_add_backward(x, 0.1, rng),
                 lambda: api.dropout_add_layernorm(x, x, None, None, 0.1, rng),
                 lambda: api.dropout_add_layernorm_backward(x, None, x, None, x[:, 0].float(),
                                                            x[:, 0].float(), 0.1, rng),
                 lambda: api.rope([x[None, None]], freq), lambda: api.rope_backward([x], freq)]:
        with pytest.raises(L.LmError) as e:
            call()
        assert e.value.status == 1


def test_gradient_formulas_against_differences():
    """The reference gradients that the GPU tests compare with, against central
    differences of the reference forward in fp64: the error of a central difference at
    step e is e^2 times third derivatives (below 1e-7 here) plus 2^-52 / e of the loss."""
    r = np.random.default_rng(5)
    x, w, b = r.normal(size=(3, 11)), r.normal(size=11) + 1, r.normal(size=11)
    dy, e = r.normal(size=(3, 11)), 1e-5

    def loss(x, w, b):
        return float((ref.norm(x, w, b, 1e-3)[0] * dy).sum())
    _, mean, rstd = ref.norm(x, w, b, 1e-3)
    for got, arg in zip(ref.norm_grads(dy, x, w, mean, rstd), (x, w, b)):
        num = np.zeros_like(arg)
        for i in np.ndindex(arg.shape):
            keep = arg[i]
            arg[i] = keep + e
            up = loss(x, w, b)
            arg[i] = keep - e
            num[i] = (up - loss(x, w, b)) / (2 * e)
            arg[i] = keep
        assert np.abs(num - got).max() <= 1e-7
    # the rotation is linear: <rope(x), dy> = <x, rope'(dy)>
    x, dy = r.normal(size=(2, 3, 4, 10)), r.normal(size=(2, 3, 4, 10))
    pos = r.integers(0, 1000, size=(2, 3))
    f = np.array([1.0, 0.1, 0.01])
    for il in (False, True):
        a = (ref.rope(x, f, pos, il, 1.2) * dy).sum()
        assert math.isclose(a, (x * ref.rope(dy, f, pos, il, 1.2, inverse=True)).sum(), rel_tol=1e-12)


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace
    from fp8_gemms_b200 import api
    stream = SimpleNamespace(device=torch.device("cuda", 1))
    q = torch.zeros(1, 2, 1, 8)
    for call in (lambda: api.layernorm(q[0, :, 0], stream=stream),
                 lambda: api.rope([q], torch.ones(4, dtype=torch.float64), stream=stream)):
        with pytest.raises(api.LmError) as e:
            call()
        assert e.value.status == 1


def test_arguments_that_are_no_tensors_are_refused():
    from fp8_gemms_b200 import api
    for call in (lambda: api.layernorm([1.0]), lambda: api.dropout_add(None, 0.1, None),
                 lambda: api.rope([], None), lambda: api.rope([None], None),
                 lambda: api.rope([torch.zeros(1, 1, 1, 2)] * 3, None)):
        with pytest.raises(api.LmError) as e:
            call()
        assert e.value.status == 1
    with pytest.raises(TypeError):
        api.rope(3, None)
