"""Plain definitions of the FP4, gated-norm and rotary operators, in float64
numpy, for the parity tests. The scales of the FP4 formats are defined by
single-precision steps, taken here in numpy float32; everything else is 64 bits."""
import math

import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
F32 = np.float32


def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, (b & 7) / 8.0
    v = np.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e.astype(np.float64) - 7))
    v = np.where((b & 0x7f) == 0x7f, np.nan, v)
    return np.where(b & 0x80, -v, v)


E4M3 = e4m3_table()


def e4m3_code(x):
    """Byte of the E4M3 value nearest to x >= 0 (ties to even, at most 448)."""
    grid = E4M3[:127]
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    hi = np.clip(np.searchsorted(grid, x), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def e2m1_code(y):
    """Code of the E2M1 value nearest to y (ties to the even code, at most 6)."""
    a = np.minimum(np.abs(np.asarray(y, np.float64)), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c | (np.signbit(y) << 3)).astype(np.uint8)


def tensor_scale(x):
    a = np.abs(np.asarray(x, F32))
    a = a[np.isfinite(a)]
    m = a.max() if a.size else F32(0)
    return max(F32(m / F32(2688)), F32(2.0 ** -149)) if m > 0 else F32(1)


def quantize(fmt, x, g=None):
    """x fp32 [rows, k] -> codes [rows, k] and scale bytes [rows, blocks]. A block
    with a NaN or an infinity has the NaN byte (its codes are not compared)."""
    x = np.asarray(x, F32)
    rows, k = x.shape
    bs = BLOCK[fmt]
    b = x.reshape(rows, k // bs, bs)
    with np.errstate(all="ignore"):
        amax = np.abs(b).max(-1)
        bad = ~np.isfinite(amax)
        if fmt == MX:
            e = np.frexp(np.where(bad | (amax == 0), 1, amax).astype(np.float64))[1] - 1
            byte = np.where(amax > 0, np.maximum(e - 2 + 127, 0), 0)
            y = b.astype(np.float64) * 2.0 ** (127.0 - byte)[..., None]
            byte = np.where(bad, 255, byte)
        else:
            g = F32(1 if g is None else g)
            r6 = F32(1) / F32(F32(6) * g)
            want = np.where(amax > 0, (amax * r6).astype(F32), F32(0))
            byte = e4m3_code(np.where(bad, 0, want))
            d = (E4M3[byte].astype(F32) * g).astype(F32)
            inv = np.where(d >= F32(2.0 ** -126), F32(1) / d, F32(0)).astype(F32)
            y = (b * inv[..., None]).astype(F32)
            byte = np.where(bad | ~(g > 0) | ~np.isfinite(g), 127, byte)
        codes = e2m1_code(np.where(bad[..., None], 0, y))
    return codes.reshape(rows, k), byte.astype(np.uint8)


def scale_values(fmt, byte):
    if fmt == MX:
        return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return E4M3[byte]


def values(fmt, codes, byte, g=None):
    """float64 values of codes [rows, k] under scale bytes [rows, blocks]."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = scale_values(fmt, byte) * (1.0 if g is None else float(g))
    return v * np.repeat(s, BLOCK[fmt], 1)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def sf_index(rows, blocks):
    r, s = np.arange(rows)[:, None], np.arange(blocks)[None]
    return ((r // 128) * (-(-blocks // 4)) + s // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + s % 4


def sf_bytes(fmt, rows, k):
    return -(-rows // 128) * (-(-k // (4 * BLOCK[fmt]))) * 512


def sf_layout(byte, fill=0):
    """Scale bytes [rows, blocks] in the array a kernel reads."""
    rows, blocks = byte.shape
    out = np.full(-(-rows // 128) * (-(-blocks // 4)) * 512, fill, np.uint8)
    out[sf_index(rows, blocks)] = byte
    return out


def gelu(x):
    return 0.5 * x * np.vectorize(math.erfc, otypes=[np.float64])(-x / math.sqrt(2))


def rms(x, eps=1e-6):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def gated_norm(x, branch=None, gate=None, shift=None, scale=None, per=0, post_norm=False,
               post_weight=None, pre_weight=None, r=1.0, eps=1e-6):
    x = np.asarray(x, np.float64)
    n = x.shape[0]
    grp = np.arange(n) // per if per else np.zeros(n, int)
    mod = lambda t, none: none if t is None else np.atleast_2d(np.asarray(t, np.float64))[grp]  # noqa: E731
    xo = r * x
    if branch is not None:
        y = np.asarray(branch, np.float64)
        if post_norm:
            y = rms(y, eps) * (1.0 if post_weight is None else post_weight)
        xo = xo + mod(gate, 1.0) * y
    v = rms(xo, eps) * (1.0 if pre_weight is None else pre_weight)
    return xo, v * (1.0 + mod(scale, 0.0)) + mod(shift, 0.0)


def rope(h, pos, sections, theta, interleaved, weight=None, norm=False, inverse=False, eps=1e-6):
    """h [n, heads, dh] float64; returns what the operator does to it, and
    |a| + |b| of each element's pair (for error bounds)."""
    h = np.array(h, np.float64)
    if norm:
        h = rms(h, eps) * (1.0 if weight is None else weight)
    out, size, col = h.copy(), np.abs(h), 0
    for axis, s in enumerate(sections):
        j = np.arange(s)
        ang = np.asarray(pos, np.float64)[:, axis, None] * np.float64(theta) ** (-j / max(s, 1))
        if inverse:
            ang = -ang
        c, sn = np.cos(ang)[:, None], np.sin(ang)[:, None]
        i0 = col + 2 * j if interleaved else col + j
        i1 = i0 + 1 if interleaved else i0 + s
        a, b = h[..., i0], h[..., i1]
        out[..., i0], out[..., i1] = a * c - b * sn, b * c + a * sn
        size[..., i0] = size[..., i1] = np.abs(a) + np.abs(b)
        col += 2 * s
    return out, size
