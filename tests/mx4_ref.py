"""4-bit microscaled values from their definition (OCP Microscaling Formats 1.0), in
numpy and 64 bits; shares nothing with the library."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """Codes [rows, cols] (0..15) and scale bytes [rows, cols/32] of finite or
    non-finite x [rows, cols] (any float type)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    a = np.abs(b).max(axis=2)
    bad = ~np.isfinite(a)
    with np.errstate(divide="ignore"):
        _, ex = np.frexp(np.where(bad, 1.0, a))              # a = m * 2^ex, m in [0.5, 1)
    e = np.where(a == 0, -127, np.maximum(ex - 1 - 2, -127))
    v = np.abs(np.where(bad[..., None], 0.0, b)) * np.ldexp(1.0, -e)[..., None]
    # nearest magnitude; of two equally near the one whose code is even
    d = np.abs(v[..., None] - MAGNITUDES)
    near = d == d.min(axis=-1, keepdims=True)
    order = np.where(near, np.arange(8) % 2, 9)
    codes = order.argmin(axis=-1).astype(np.uint8)
    codes |= (np.signbit(b) & ~bad[..., None]).astype(np.uint8) << 3
    return codes.reshape(rows, cols), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed):
    c = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = packed & 15, packed >> 4
    return c


def tiles(scales, fill=0):
    """[ceil(rows/128), blocks/4, 32, 4, 4] from [rows, blocks], element by element."""
    rows, blocks = scales.shape
    t = np.full((-(-rows // 128), blocks // 4, 32, 4, 4), fill, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    t[r // 128, b // 4, r % 32, r // 32 % 4, b % 4] = scales
    return t


def untile(t, rows):
    r, b = np.meshgrid(np.arange(rows), np.arange(4 * t.shape[1]), indexing="ij")
    return t[r // 128, b // 4, r % 32, r // 32 % 4, b % 4]


def values(codes, scales):
    """fp64 values of codes [rows, cols] and scale bytes [rows, cols/32] (255: NaN)."""
    v = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)
