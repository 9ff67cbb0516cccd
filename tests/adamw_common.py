"""Plain numpy forms of AdamW's step over many tensors: one in fp32 that
rounds once per operation in the stated order (the kernels have to equal it
bit for bit), one in 64 bits from the formulas, and the 8-bit codes.

Bounds of the fp32 form against the 64-bit one, with u = 2^-24 (half a step,
relative), for g' exact and first-order in u:
  m: two products and a sum: 2u(|b1 m| + |ob1 g'|) <= 3u(...) with the next orders
  v: g'*g' and the factor round before the sum: 3u on every term <= 4u v
  den: sqrt(v) 2u + u, times rbc2 (itself rounded) 2u, plus eps u: <= 6u den,
       so m/den carries |dm|/den + 7u|m|/den, and the rate (rounded) and the
       product 2u more: 9u |up| + rate |dm|/den
  x: decay rounded, product, difference: 3u|x| + u|up| on top

Beside 8-bit states the kernels take the square root and the reciprocal from
instructions of one ulp (2u) each.  From the same m and v, then: sqrt 2u, the
factor u, eps's sum u, the reciprocal 2u, the product u, the rate u, against u
for each of the five operations in the form below: 8u + 5u of the update, and
the final difference rounds u|x| on either side, so 2u|x| + 13u|up|; 14u covers
the higher orders.  The rounding to bfloat16 is monotone, so a parameter lies
between the roundings of the two ends.
"""
import math

import numpy as np

U = 2.0 ** -24
F = np.float32
B1, B2, EPS = F(0.9), F(0.999), F(1e-8)
OB1, OB2 = F(1) - B1, F(1) - B2
M32 = np.uint64(0xFFFFFFFF)


# ------------------------------------------------------------ random bits --
def keys_of(seed, t):
    m64 = (1 << 64) - 1
    z = (seed * 0x6A09E667F3BCC909 + t * 0xBB67AE8584CAA73B) & m64
    z = ((z ^ (z >> 31)) * 0x3C6EF372FE94F82B) & m64
    z = ((z ^ (z >> 31)) * 0x6A09E667F3BCC909) & m64
    z ^= z >> 32
    return z & 0xFFFFFFFF, z >> 32


def random16(first, n, seed, t, word):
    """16-bit integers of elements [first, first + n) (first a multiple of 4)
    from words `word` and `word + 1`."""
    k0, k1 = (np.uint64(k) for k in keys_of(seed, t))
    q = np.uint64(first // 4) + np.arange(-(-n // 4), dtype=np.uint64)
    h = (q & M32) ^ k0 ^ (((q >> np.uint64(32)) * np.uint64(0x9E3779B9)) & M32)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x3C6EF373)) & M32
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0xBB67AE85)) & M32
    w = [h ^ (h >> np.uint64(16))]
    for i in range(1, word + 2):
        h = ((w[-1] ^ k1) * np.uint64(0x9E3779B9) + np.uint64(i)) & M32
        w.append(h ^ (h >> np.uint64(15)))
    a, b = w[word], w[word + 1]
    lo = np.uint64(0xFFFF)
    return np.stack([a & lo, a >> np.uint64(16), b & lo, b >> np.uint64(16)], 1).ravel()[:n].astype(
        np.int64)


# ------------------------------------------------------------- bfloat16 ----
def bf16_nearest(x):
    """fp32 -> the fp32 value of its bfloat16 (nearest even); NaN stays NaN."""
    x = np.asarray(x, F)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + np.uint64(0x7FFF) + ((b >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)
         << np.uint64(16)).astype(np.uint32).view(F)
    return np.where(np.isnan(x), x, r).astype(F)


def bf16_stochastic(x, r16):
    x = np.asarray(x, F)
    b = x.view(np.uint32).astype(np.int64)
    r = ((b + r16) & 0xFFFF0000).astype(np.uint32).view(F)
    return np.where(np.isfinite(x), r, x).astype(F)


# ------------------------------------------------------------ 8-bit codes --
def _e4m3_table():
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out[c] = math.nan if c & 127 == 127 else (-v if c & 128 else v)
    return out


E4M3 = _e4m3_table()


def _blocks(a, fill=0.0):
    n = -(-a.size // 256) * 256
    out = np.full(n, fill, a.dtype)
    out[:a.size] = a
    return out.reshape(-1, 256)


def encode_m(m):
    """(codes, exponent bytes) of one tensor's first moments."""
    m = np.asarray(m, F)
    b = _blocks(m)
    top = np.where(np.isfinite(b), np.abs(b), F(0)).astype(F).max(1).view(np.uint32) >> 23
    e = np.maximum(top, 8).astype(np.int64)
    y = b.astype(np.float64) * 2.0 ** (134.0 - e)[:, None]  # exact
    # nearest even on the e4m3 grid: steps of 2^-9 below 2^-6, of 1/8 binade above
    with np.errstate(all="ignore"):
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
        v = np.rint(y / step) * step
    mag = E4M3[:127]
    code = np.searchsorted(mag, np.abs(np.where(np.isfinite(v), v, 0.0)))
    assert np.array_equal(mag[code], np.abs(np.where(np.isfinite(v), v, 0.0)))
    code = np.where(np.isfinite(v), code, 127) | np.where(np.signbit(b), 128, 0)
    return code.ravel()[:m.size].astype(np.uint8), e.astype(np.uint8)


def decode_m(code, e):
    return (E4M3[code].astype(F) * np.repeat(F(2) ** (e.astype(F) - F(134)), 256)[:code.size]
            ).astype(F)


def encode_v(v, noise):
    """(codes, exponent bytes); noise: integers below 2^20, one per element."""
    v = np.asarray(v, F)
    b = _blocks(v)
    ok = np.isfinite(b)
    q = (np.where(ok, b, F(0)).astype(F).view(np.uint32).astype(np.int64)
         + _blocks(np.broadcast_to(noise, v.shape).astype(np.int64), 0)) >> 20
    q = np.minimum(q, 2039)
    top = np.where(ok, q, 0).max(1)
    e = np.maximum(top >> 3, 32)
    code = np.clip(q - ((e - 31) * 8 + 1)[:, None], 1, 254)
    code = np.where(b == 0, 0, code)
    code = np.where(ok, code, 255)
    return code.ravel()[:v.size].astype(np.uint8), e.astype(np.uint8)


def decode_v(code, e):
    c = code.astype(np.int64)
    low = np.repeat((e.astype(np.int64) - 31) * 8 + 1, 256)[:code.size]
    v = (((c + low) << 20).astype(np.uint32)).view(F)
    v = np.where(c == 0, F(0), v)
    return np.where(c == 255, F(np.nan), v).astype(F)


# ------------------------------------------------------------------ steps --
def scalars(t, lr, wd, gs=1.0):
    """(gs, decay, rate, rbc2) of step t as the kernels hold them."""
    p1 = p2 = 1.0
    for _ in range(t):
        p1, p2 = p1 * float(B1), p2 * float(B2)
    lr, wd = float(F(lr)), float(F(wd))
    return F(gs), F(1.0 - lr * wd), F(lr / (1.0 - p1)), F(1.0 / math.sqrt(1.0 - p2))


def step32(x, m, v, g, t, lr, wd, gs=1.0, eps=EPS):
    """fp32, one rounding per operation: new x, m, v."""
    x, m, v, g = (np.asarray(a, F) for a in (x, m, v, g))
    gs, decay, rate, rbc2 = scalars(t, lr, wd, gs)
    with np.errstate(all="ignore"):
        g = g * gs
        m = (B1 * m) + (OB1 * g)
        v = (B2 * v) + (OB2 * (g * g))
        x = (x * decay) - (rate * (m / ((np.sqrt(v) * rbc2) + eps)))
    return x, m, v


def step64(x, m, v, g, t, lr, wd, gs=1.0):
    """The formulas in 64 bits, and bounds on the fp32 form's errors: (x, m, v),
    (dx, dm, dv)."""
    x, m, v, g = (np.asarray(a, np.float64) for a in (x, m, v, g))
    b1, b2, eps = float(B1), float(B2), float(EPS)
    lr, wd = float(F(lr)), float(F(wd))
    g = g * gs
    dm = 3 * U * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = np.sqrt(v / (1 - b2 ** t)) + eps
    rate = lr / (1 - b1 ** t)
    up = rate * m / den
    dx = 3 * U * np.abs(x) + 10 * U * np.abs(up) + rate * dm / den
    return (x * (1 - lr * wd) - up, m, v), (dx, dm, 4 * U * v)


class Reference:
    """The fp32 form over a list of tensors, as the library's plan runs it."""

    def __init__(self, params, offsets, bits=32, param="f32", master=False, stochastic=False,
                 groups=None, seed=0, steps=0, eps=EPS):
        self.eps = F(eps)
        self.x = [np.asarray(p, F).copy() for p in params]
        self.offsets, self.bits, self.param = offsets, bits, param
        self.stochastic, self.seed, self.t = stochastic, seed, steps
        self.groups = groups or [0] * len(params)
        self.master = [p.copy() for p in self.x] if master else None
        z = [np.zeros(p.size, F) for p in self.x]
        self.m, self.v = z, [a.copy() for a in z]
        # what the last step rounded to the parameter, and how far it moved it
        self.exact, self.up = [None] * len(params), [None] * len(params)
        if bits == 8:
            self.m = [encode_m(a) for a in z]
            self.v = [encode_v(a, 0) for a in z]

    def bounds(self, i):
        """The least and the greatest value that tensor i may have."""
        # below 2^-30 the library keeps the correctly rounded forms
        if self.bits == 32 or self.up[i] is None or self.eps < 2.0 ** -30:
            x = self.x[i] if self.master is None else self.master[i]
            return x, x
        with np.errstate(all="ignore"):
            x = self.exact[i].astype(np.float64)
            d = U * (2 * np.abs(x) + 14 * np.abs(self.up[i].astype(np.float64)))
            ends = []
            for side in (-1, 1):
                y = np.nextafter((x + side * d).astype(F), F(side * np.inf))  # outwards
                y = np.where(np.isfinite(x), y, self.exact[i])
                ends.append(y if self.master is not None else self.rounded(i, y))
        return ends

    def rounded(self, i, x):
        if self.param == "f32":
            return x
        if self.stochastic:
            return bf16_stochastic(x, random16(self.offsets[i], x.size, self.seed, self.t, 2))
        return bf16_nearest(x)

    def norm(self, grads, scale=1.0):
        s = sum(float(np.dot(g.astype(np.float64), g.astype(np.float64))) for g in grads
                if g is not None and g.size)
        return math.sqrt(s) * scale

    def step(self, grads, lr, wd, max_norm=0.0, scale=1.0, norm=None):
        self.t += 1
        coef = 1.0
        if max_norm:
            n = self.norm(grads, float(F(scale))) if norm is None else norm
            mx = float(F(max_norm))
            coef = 1.0 if n <= mx else mx / n
        gs = F(float(F(scale)) * coef)
        for i, g in enumerate(grads):
            if g is None or g.size == 0:
                continue
            a, b = (q if np.isscalar(q) else q[self.groups[i]] for q in (lr, wd))
            m, v = self.m[i], self.v[i]
            if self.bits == 8:
                m, v = decode_m(*m), decode_v(*v)
            old = self.master[i] if self.master is not None else self.x[i]
            x, m, v = step32(old, m, v, g, self.t, a, b, gs, self.eps)
            off = self.offsets[i]
            if self.bits == 8:
                r = random16(off, x.size, self.seed, self.t, 0)
                m, v = encode_m(m), encode_v(v, r * 16 + 8)
            self.m[i], self.v[i] = m, v
            with np.errstate(all="ignore"):
                self.exact[i], self.up[i] = x, x - old * (F(1) - F(float(F(a)) * float(F(b))))
            if self.master is not None:
                self.master[i] = x
            self.x[i] = self.rounded(i, x)


def same(a, b):
    """Equal values: NaN equals NaN, and zeros of either sign are equal."""
    a, b = np.asarray(a), np.asarray(b)
    return a.shape == b.shape and bool(np.all((a == b) | ((a != a) & (b != b))))
