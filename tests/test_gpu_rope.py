"""Rotary positions on the GPU against the 64-bit form of rows_ref: pairings, partial heads,
layouts and strides, far positions, in place, and the backward pass."""
import numpy as np
import pytest
import torch

import rows_ref as ref
from rows_ref import close, f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# batch, seq, Q heads, K heads, head_dim, rot_dim, type, layout
SHAPES = [(1, 1, 1, 1, 2, 2, F32, "bshd"), (2, 3, 5, 1, 6, 4, BF, "bshd"),
          (2, 9, 24, 8, 128, 128, BF, "bshd"), (64, 1, 24, 8, 128, 128, BF, "bshd"),
          (2, 17, 6, 2, 64, 64, BF, "qkv"), (3, 33, 4, 4, 80, 32, F32, "bhsd"),
          (1, 70, 3, 1, 96, 48, BF, "bhsd"), (2, 11, 7, 7, 100, 50, BF, "qkv"),
          (1, 300, 2, 1, 256, 256, BF, "bshd"), (2, 5, 2, 2, 192, 64, F32, "qkv"),
          (1, 13, 3, 2, 40, 0, BF, "bshd"), (1, 7, 3, 3, 72, 16, BF, "odd"),
          (2, 19, 64, 1, 32, 32, F32, "bshd"), (1, 5, 1, 1, 333, 332, BF, "bshd"),
          (1, 2100, 1, 1, 16, 16, BF, "bshd"), (2, 6, 100, 4, 64, 32, BF, "bhsd")]
# the copied rest with few tokens and with many, at each width of access
SHAPES += [(3, 700, 3, 2, 40, 16, BF, "bshd"), (3, 701, 3, 2, 40, 20, BF, "bhsd"), (1, 1301, 2, 1, 23, 6, BF, "odd"),
           (3, 701, 3, 2, 40, 20, F32, "bshd"), (2, 650, 17, 2, 24, 16, F32, "bhsd"), (1185, 1, 2, 2, 12, 4, BF, "qkv"),
           (7, 1, 33, 5, 48, 16, BF, "qkv"), (5, 3, 2, 2, 512, 320, BF, "bshd")]
IDS = ["-".join(str(v).replace("torch.", "") for v in s) for s in SHAPES]


def tensors(b, s, hq, hk, d, dtype, layout, seed):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).to(dtype).cuda()
    if layout == "qkv":
        qkv = normal(b, s, hq + 2 * hk, d)
        return qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    if layout == "bhsd":
        return normal(b, hq, s, d).transpose(1, 2), normal(b, hk, s, d).transpose(1, 2)
    if layout == "odd":       # odd strides, an odd first element
        q, k = normal(b, s, hq, d + 3), normal(b, s, hk, d + 5)
        return q[..., 1:d + 1], k[..., 3:d + 3]
    return normal(b, s, hq, d), normal(b, s, hk, d)


def check(xs, got, freq, pos, il, mag, inverse=False):
    f = f64(freq)
    for x, y in zip(xs, got):
        assert y.dtype == x.dtype and y.shape == x.shape
        want = ref.rope(f64(x), f, pos, il, mag, inverse)
        close(f64(y), want, ref.rope_bound(f64(x), f, pos, il, mag, x.dtype, inverse), "rope")
        assert torch.equal(y[..., 2 * len(f):], x[..., 2 * len(f):])


@pytest.mark.parametrize("il", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("b,s,hq,hk,d,rot,dtype,layout", SHAPES, ids=IDS)
def test_forward_and_backward(b, s, hq, hk, d, rot, dtype, layout, il):
    from fp8_gemms_b200 import api
    q, k = tensors(b, s, hq, hk, d, dtype, layout, 1)
    freq, mag = api.rope_frequencies(rot, scaling=api.ROPE_BY_PARTS, factor=4.0, context=2048.0)
    assert freq.shape == (rot // 2,)
    gen = torch.Generator().manual_seed(2)
    positions = torch.randint(0, 100000, (b, s), generator=gen).cuda()
    pos = positions.cpu().numpy()
    kw = dict(positions=positions, interleaved=il, magnitude=mag)
    check((q, k), api.rope([q, k], freq, **kw), freq, pos, il, mag)
    check((q, k), api.rope_backward([q, k], freq, **kw), freq, pos, il, mag, inverse=True)
    # one tensor; positions counted from `start`
    one = api.rope([k], freq, start=77, interleaved=il, magnitude=mag)
    count = np.broadcast_to(77 + np.arange(s), (b, s))
    check((k,), one, freq, count, il, mag)


@pytest.mark.parametrize("start", [0, -5, 1 << 20, (1 << 31) + 7, 1 << 40])
def test_far_positions(start):
    """The angle is right where fp32 would not hold the position, let alone its product."""
    from fp8_gemms_b200 import api
    q, _ = tensors(1, 40, 2, 1, 64, F32, "bshd", 3)
    freq, _ = api.rope_frequencies(64)
    pos = start + np.arange(40)[None]
    check((q,), api.rope([q], freq, start=start), freq, pos, False, 1.0)
    positions = torch.from_numpy(pos.copy()).cuda()
    assert torch.equal(api.rope([q], freq, positions=positions)[0],
                       api.rope([q], freq, start=start)[0])


@pytest.mark.parametrize("il", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("layout,d,rot", [("bshd", 128, 128), ("qkv", 64, 32), ("bhsd", 80, 32),
                                          ("odd", 72, 16), ("bshd", 50, 50)])
def test_in_place_leaves_the_rest_alone(layout, d, rot, il):
    from fp8_gemms_b200 import api
    freq, _ = api.rope_frequencies(rot)
    q, k = tensors(2, 21, 6, 2, d, BF, layout, 4)
    want = api.rope([q, k], freq, start=9, interleaved=il)
    base = q._base if q._base is not None else q
    before = base.clone()
    got = api.rope([q, k], freq, start=9, interleaved=il, out=[q, k])
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    if layout == "qkv":       # V, behind Q and K in the same buffer
        assert torch.equal(base[:, :, 8:], before[:, :, 8:])
    if layout == "odd":       # the elements around each head
        assert torch.equal(base[..., :1], before[..., :1])
        assert torch.equal(base[..., d + 1:], before[..., d + 1:])


def test_shared_heads_as_an_expanded_view():
    """One K head seen as four by a zero stride is read as such; an output cannot be."""
    from fp8_gemms_b200 import _lib, api
    freq, _ = api.rope_frequencies(64)
    k = torch.randn(2, 5, 1, 64, device="cuda").to(BF)
    many = k.expand(2, 5, 4, 64)
    got = api.rope([many], freq, out=[torch.empty(2, 5, 4, 64, dtype=BF, device="cuda")])[0]
    one = api.rope([k], freq)[0]
    for h in range(4):
        assert torch.equal(got[:, :, h], one[:, :, 0])
    with pytest.raises(_lib.LmError):
        api.rope([many], freq, out=[many])


def test_inverse_undoes_the_rotation():
    """R^-1 R x = x up to two passes' bounds (the second's input is off by the first's)."""
    from fp8_gemms_b200 import api
    x, _ = tensors(2, 50, 3, 1, 96, F32, "bshd", 5)
    freq, _ = api.rope_frequencies(96)
    y = api.rope_backward(api.rope([x], freq, start=5), freq, start=5)[0]
    pos = np.broadcast_to(5 + np.arange(50), (2, 50))
    one = ref.rope_bound(f64(x), f64(freq), pos, False, 1.0, F32)
    # a rotation of an error of size e in both elements is at most sqrt(2) e in each
    close(f64(y), f64(x), one + 1.5 * (one + np.roll(one, 48, -1)), "inverse")


def test_empty_shapes():
    from fp8_gemms_b200 import api
    freq, _ = api.rope_frequencies(64)
    for shape in [(0, 5, 2, 64), (2, 0, 2, 64), (2, 5, 0, 64)]:
        x = torch.empty(shape, dtype=BF, device="cuda")
        assert api.rope([x], freq)[0].shape == shape
    # no K heads beside Q heads, and the other way round
    q = torch.randn(2, 5, 3, 64, device="cuda").to(BF)
    none = torch.empty(2, 5, 0, 64, dtype=BF, device="cuda")
    want = api.rope([q], freq)[0]
    assert torch.equal(api.rope([q, none], freq)[0], want)
    assert torch.equal(api.rope([none, q], freq)[1], want)


def test_streams_and_graphs():
    from fp8_gemms_b200 import api
    q, k = tensors(2, 33, 6, 2, 128, BF, "qkv", 6)
    freq, _ = api.rope_frequencies(128)
    positions = torch.arange(33, device="cuda").repeat(2, 1)
    want = api.rope([q, k], freq, positions=positions)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = api.rope([q, k], freq, positions=positions, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        outs = api.rope([q, k], freq, positions=positions)
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, outs):
        assert torch.equal(a, b) and torch.equal(a, c)
    positions += 1000
    g.replay()
    want = api.rope([q, k], freq, positions=positions)
    torch.cuda.synchronize()
    for a, c in zip(want, outs):
        assert torch.equal(a, c)


def test_refusals():
    from fp8_gemms_b200 import _lib, api
    freq, _ = api.rope_frequencies(64)
    x = torch.zeros(2, 5, 3, 64, dtype=BF, device="cuda")
    pos = torch.zeros(2, 5, dtype=torch.int64, device="cuda")
    for call, status in [(lambda: api.rope([x[0]], freq), 1),
                         (lambda: api.rope([x, x, x], freq), 1),
                         (lambda: api.rope([x, x[:1]], freq), 1),
                         (lambda: api.rope([x, x.float()], freq), 1),
                         (lambda: api.rope([x.half()], freq), 4),
                         (lambda: api.rope([x[..., :32]], freq), 1),
                         (lambda: api.rope([x[..., ::2]], freq[:16]), 1),
                         (lambda: api.rope([x], freq.float()), 1),
                         (lambda: api.rope([x], freq.cpu()), 1),
                         (lambda: api.rope([x], freq, positions=pos.int()), 1),
                         (lambda: api.rope([x], freq, positions=pos[:1]), 1),
                         (lambda: api.rope([x], freq, start=1 << 63), 1),
                         (lambda: api.rope([x], freq, magnitude=float("nan")), 1),
                         (lambda: api.rope([x], freq, out=[x[:1]]), 1)]:
        with pytest.raises(_lib.LmError) as err:
            call()
        assert err.value.status == status


def test_elements_past_two_to_the_31():
    from fp8_gemms_b200 import api
    b, s, h, d = 2, 65552, 128, 128
    x = torch.zeros(b, s, h, d, dtype=BF, device="cuda")
    x[-1, -3:] = torch.randn(3, h, d, device="cuda").to(BF)
    freq, _ = api.rope_frequencies(d)
    tail = x[-1:, -3:].clone()
    api.rope([x], freq, out=[x])
    pos = (s - 3 + np.arange(3))[None]
    check((tail,), (x[-1:, -3:],), freq, pos, False, 1.0)
