"""Plain 64-bit forms of the row operators (layer norm, dropout, rotary
positions) and the error bounds their tests use.  numpy only; shares no code
with the library.

Bounds count roundings.  U = 2^-24 is half a step of fp32 relative to the value,
HALF[dtype] that of an output's type.  A sum of n fp32 values in any order that
adds at most `depth` values one after the other along any path is off by at most
depth U sum|x|."""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(shape, dtype, seed, sigma=1.0, mean=0.0, pad=0, shift=0):
    """A seeded [rows x cols] CUDA tensor whose rows are `cols + pad` apart and
    which starts `shift` elements into its buffer; the buffer is NaN elsewhere."""
    rows, cols = shape
    ld = cols + pad
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((shift + max(rows, 1) * ld + 64,), float("nan"), dtype=dtype)
    view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen) * sigma + mean)
    dev = buf.cuda()
    return dev[shift:shift + rows * ld].view(rows, ld)[:, :cols]


def vector(n, dtype, seed, sigma=1.0, mean=0.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=gen) * sigma + mean).to(dtype).cuda()


def close(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), (f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound, "
                               f"worst |d| {np.abs(got - ref).max():.3e}, by {over.max():.3e}")


# ------------------------------------------------------------------ layer norm
def row_depth(cols):
    """Additions on a path of a row's sum: a thread's own columns one after the
    other (at least 32 lanes share a row; a wide row has 256 threads), five
    shuffles, and at most 32 warps."""
    return max(64, -(-cols // 256) + 8) + 5 + 32


def norm(x, w, b, eps):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    h = c * rstd[:, None]
    return h * (1.0 if w is None else w) + (0.0 if b is None else b), mean, rstd


def norm_bounds(x, w, b, eps, dtype):
    """(y, mean, rstd) bounds.  The mean is off by depth U mean|x| =: m.  A centred value
    is off by m + U|c|, their mean square by m^2 + (depth + 4) U var (the terms
    linear in m cancel in the sum up to U), rstd relatively by half of that over
    var + eps, plus 3 roundings."""
    y, mean, rstd = norm(x, w, b, eps)
    d = row_depth(x.shape[1])
    m = (d + 1) * U * np.abs(x).mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    # |m| mean|c| bounds what is left of the linear terms after the centring
    dr = 0.5 * (m * m + (d + 4) * U * var + 2 * U * m * np.abs(c).mean(1)) / (var + eps) + 3 * U
    h, wa = c * rstd[:, None], np.abs(1.0 if w is None else w)
    dh = rstd[:, None] * (m[:, None] + U * np.abs(c)) + np.abs(h) * (dr[:, None] + U)
    return (HALF[dtype] * np.abs(y) + (1 + HALF[dtype]) * (wa * dh + 2 * U * (np.abs(h) * wa + np.abs(
        0.0 if b is None else b))) + 1e-38, m + U * np.abs(mean) + 1e-38, rstd * dr)


def norm_grads(dy, x, w, mean, rstd):
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def norm_grad_bounds(dy, x, w, mean, rstd, dtype, wgrad_dtype):
    """(dx, dw, db) bounds: g and h are off by U and 2 U of themselves, their means by the
    sums' depth, and dx adds four roundings; a column's sum is at most `rows` deep."""
    dx, dw, db = norm_grads(dy, x, w, mean, rstd)
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    k = (row_depth(x.shape[1]) + 16) * U
    inner = np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(h) * np.abs(g * h).mean(
        1, keepdims=True)
    kr = (x.shape[0] + 16) * U
    hw = HALF[wgrad_dtype]
    return (HALF[dtype] * np.abs(dx) + 1.01 * np.abs(rstd)[:, None] * k * inner + 1e-38,
            hw * np.abs(dw) + 1.01 * kr * np.abs(dy * h).sum(0) + 1e-38,
            hw * np.abs(db) + 1.01 * kr * np.abs(dy).sum(0) + 1e-38)


# --------------------------------------------------------------------- dropout
def philox4x32_10(counter, key):
    """Four uint32 words (Salmon et al., 2011); counter: four, key: two arrays or
    numbers."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [np.uint64(v) for v in key]
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ k[0], b & low, (a >> sh) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return [v.astype(np.uint32) for v in c]


def keep_mask(rows, cols, p, seed, offset, first_row=0):
    """(keep [rows x cols], scale as fp32): the documented mask."""
    groups = -(-cols // 8)
    offset &= (1 << 64) - 1
    shape = (rows, groups)
    c0 = np.broadcast_to(np.arange(groups, dtype=np.uint64)[None], shape)
    c1 = np.broadcast_to(np.arange(first_row, first_row + rows, dtype=np.uint64)[:, None], shape)
    w = philox4x32_10([c0, c1, np.full(shape, offset & 0xFFFFFFFF, np.uint64),
                       np.full(shape, offset >> 32, np.uint64)],
                      [seed & 0xFFFFFFFF, seed >> 32])
    half = np.stack([h for v in w for h in (v & np.uint32(0xFFFF), v >> np.uint32(16))], -1)
    drop = int(np.rint(p * 65536.0))
    scale = np.float32(65536.0 / (65536.0 - drop)) if drop < 65536 else np.float32(0)
    return half.reshape(rows, -1)[:, :cols] >= drop, scale


def dropped(x, keep, scale):
    """The documented fp32 product, as fp32."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(keep, x.astype(np.float32) * scale, np.float32(0))


# ---------------------------------------------------------------------- rotary
def rope(x, inv_freq, positions, interleaved, magnitude, inverse=False):
    """x: [batch, seq, heads, dim] fp64; positions: [batch, seq] integers."""
    rot = 2 * len(inv_freq)
    turn = positions.astype(np.longdouble)[:, :, None] * np.asarray(inv_freq, np.longdouble)
    c = (np.cos(turn) * magnitude).astype(np.float64)[:, :, None]
    s = (np.sin(turn) * magnitude).astype(np.float64)[:, :, None]
    if inverse:
        s = -s
    y = x.copy()
    i1, i2 = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved
              else (np.arange(rot // 2), np.arange(rot // 2, rot)))
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def rope_bound(x, inv_freq, positions, interleaved, magnitude, dtype, inverse=False):
    """The angle: the fp64 product position * (f / 2 pi) carries three roundings of
    2^-53 of itself in turns, 2 pi of that in radians; fp32 keeps the reduced half-turn
    to U of at most 1, pi U radians.  sincospif is good to 2 ulp (4 U); the products
    with the magnitude, with x and the sum add 4 U.  The last rounding is half a step of
    the output itself, which the inverse turns the other way: of that one."""
    rot = 2 * len(inv_freq)
    turns = np.abs(positions.astype(np.float64))[:, :, None] * inv_freq / (2 * np.pi)
    angle = 2 * np.pi * 3 * 2.0 ** -53 * turns + np.pi * U
    i1, i2 = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved
              else (np.arange(rot // 2), np.arange(rot // 2, rot)))
    size = (np.abs(x[..., i1]) + np.abs(x[..., i2])) * magnitude
    bound = np.zeros_like(x)
    for i in (i1, i2):
        bound[..., i] = size * (angle[:, :, None] + 8 * U) + 1e-38
    y = rope(x, inv_freq, positions, interleaved, magnitude, inverse)
    bound[..., :rot] += HALF[dtype] * (np.abs(y[..., :rot]) + bound[..., :rot])
    return bound
