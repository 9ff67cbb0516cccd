"""The microscaled 4-bit format in numpy and 64 bits: what the tests of ob_mx4
compare with.  Shares no code with the library."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDDLES = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
U64 = (1 << 64) - 1
U32 = 0xFFFFFFFF


def widths(cols):
    """Bytes of a row of codes and of a row of scales."""
    return 64 * -(-cols // 128), 16 * -(-cols // 512)


def keys(seed):
    z = (seed * 0x6A09E667F3BCC909) & U64
    for mul in (0x3C6EF372FE94F82B, 0x6A09E667F3BCC909):
        z = ((z ^ (z >> 31)) * mul) & U64
    z ^= z >> 32
    return z & U32, z >> 32


def noise(rows, cols, seed, first_row=0):
    """16 random bits for every element of the padded matrix (from a row on)."""
    k0, k1 = keys(seed)
    quad = np.arange(rows * widths(cols)[0] // 2, dtype=np.uint64)
    quad += np.uint64(first_row * widths(cols)[0] // 2)
    h = ((quad & U32) ^ np.uint64(k0)) ^ ((quad >> np.uint64(32)) * np.uint64(0x9E3779B9) & U32)
    h = (h ^ (h >> np.uint64(16))) * np.uint64(0x3C6EF373) & U32
    h = (h ^ (h >> np.uint64(15))) * np.uint64(0xBB67AE85) & U32
    a = h ^ (h >> np.uint64(16))
    h = ((a ^ np.uint64(k1)) * np.uint64(0x9E3779B9) + np.uint64(1)) & U32
    b = h ^ (h >> np.uint64(15))
    four = np.stack([a & 0xFFFF, a >> np.uint64(16), b & 0xFFFF, b >> np.uint64(16)], 1)
    return four.astype(np.float64).reshape(rows, -1)


def quantize(c, seed=None, first_row=0):
    """(codes, scales) of a matrix of fp32 values, as the library lays them out, or
    of the rows from first_row on of a larger one."""
    c = np.asarray(c, dtype=np.float32)
    rows, cols = c.shape
    cb, sb = widths(cols)
    wide = np.zeros((rows, 2 * cb), dtype=np.float64)
    sign = np.zeros((rows, 2 * cb), dtype=bool)
    with np.errstate(invalid="ignore"):
        wide[:, :cols] = np.abs(c.astype(np.float64))
    sign[:, :cols] = np.signbit(c)
    index = np.zeros(wide.shape, dtype=np.uint8)
    scales = np.zeros((rows, sb), dtype=np.uint8)
    u = None if seed is None else noise(rows, cols, seed, first_row)
    for b in range(cb // 16):
        part = slice(32 * b, 32 * b + 32)
        v = wide[:, part]
        good = np.isfinite(v).all(1)
        top = np.where(good, np.where(np.isfinite(v), v, 0).max(1), 0.0)
        k = np.full(rows, -127.0)
        # the least k that takes the largest value
        for _ in range(300):
            over = top >= 7 * 2.0 ** k if seed is None else top > 6 * 2.0 ** k
            if not over.any():
                break
            k[over] += 1
        scales[:, b] = np.where(good, k + 127, 255)
        y = np.where(good[:, None], v, 0.0) / (2.0 ** k)[:, None]
        if seed is None:
            i = np.searchsorted(MIDDLES, y, side="left")  # below or at the middle above
            tie = np.isin(y, MIDDLES) & (i % 2 == 1)
            i = i + tie
        else:
            g = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
            i = np.searchsorted(MAGNITUDES, np.floor(y / g + u[:, part] / 65536) * g)
        index[:, part] = np.where(good[:, None], i + 8 * sign[:, part], 0)
    return index[:, ::2] | (index[:, 1::2] << 4), scales


def values(codes, scales, cols):
    """float64 values of a quantised matrix."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    index = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    v = MAGNITUDES[index & 7] * np.where(index > 7, -1.0, 1.0)
    e = scales[:, :codes.shape[1] // 16].astype(np.float64)
    factor = np.where(e == 255, np.nan, 2.0 ** (e - 127))
    return (v * np.repeat(factor, 32, 1))[:, :cols]


def quantized(c, seed=None):
    c = np.asarray(c)
    return values(*quantize(c, seed), c.shape[1])


def spread(rows, cols, seed, scale=1.0):
    """Normal values whose blocks differ in size by powers of ten."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * 10.0 ** r.uniform(-3, 3, (rows, -(-cols // 32))).repeat(
        32, 1)[:, :cols]
    return (x * scale).astype(np.float32)
