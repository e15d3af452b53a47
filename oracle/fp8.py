"""8-bit floating point (e4m3) in blocks of 128, the norm and SwiGLU before
it and the product of such operands, in plain loops and fp64.

e4m3 (OCP 8-bit floating point): a sign, 4 exponent bits of bias 7, 3 mantissa
bits; no infinities; the codes 0x7F and 0xFF are NaN, the largest value is 448."""
import numpy as np

BLOCK = 128


def decode(codes):
    """The values (fp64) of e4m3 codes (uint8)."""
    table = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = np.nan
        table[c] = -v if c & 128 else v
    return table[np.asarray(codes, np.uint8)]


def encode(v):
    """The e4m3 codes nearest to v (|v| <= 464 or NaN), ties to the even code."""
    v = np.asarray(v, np.float64)
    grid = decode(np.arange(127))  # 0 .. 448, ascending
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, np.where(np.isnan(a), 0.0, a)), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(v), 127, code)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def step(top):
    """(s, i) of blocks whose largest absolute values are top (fp32, IEEE)."""
    top = np.asarray(top, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.maximum(top / np.float32(448), np.float32(2.0 ** -126))
    s = np.where(np.isfinite(top), s, np.float32(np.nan)).astype(np.float32)
    return s, (np.float32(1) / s).astype(np.float32)


def _codes(x, i):
    with np.errstate(invalid="ignore"):
        return encode((np.asarray(x, np.float32) * i).astype(np.float32))


def quantize(x):
    """(codes uint8 [rows][cols], s fp32 [cols/128][rows]) of fp32 rows."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    q, s = np.empty((rows, cols), np.uint8), np.empty((cols // BLOCK, rows), np.float32)
    for b in range(cols // BLOCK):
        part = x[:, BLOCK * b:BLOCK * (b + 1)]
        s[b], i = step(np.abs(part).max(1))
        q[:, BLOCK * b:BLOCK * (b + 1)] = _codes(part, i[:, None])
    return q, s


def quantize_weight(w):
    """(codes [n][k], scale [ceil(n/128)][k/128]) of fp32 weights."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    codes, scale = np.empty((n, k), np.uint8), np.empty((-(-n // BLOCK), k // BLOCK), np.float32)
    for a in range(scale.shape[0]):
        for b in range(scale.shape[1]):
            at = (slice(BLOCK * a, BLOCK * (a + 1)), slice(BLOCK * b, BLOCK * (b + 1)))
            scale[a, b], i = step(np.abs(w[at]).max())
            codes[at] = _codes(w[at], i)
    return codes, scale


def rms_norm(x, weight, eps, residual=None):
    """(v, h) in fp64: h = x + residual, v = h / sqrt(mean h^2 + eps) * weight."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    return h / np.sqrt((h * h).sum(1, keepdims=True) / h.shape[1] + eps) * np.asarray(weight, np.float64), h


def swiglu(x):
    """g / (1 + exp(-g)) * u in fp64 of [rows][2 n]."""
    x = np.asarray(x, np.float64)
    n = x.shape[1] // 2
    with np.errstate(over="ignore"):
        return x[:, :n] / (1.0 + np.exp(-x[:, :n])) * x[:, n:]


def product(x, s_x, codes, scale, cut=True):
    """[m][n] in fp64: y; the sum of the terms' absolute values; and the sum over
    every eight consecutive k of the largest power of two that is no larger than
    a product of two binades there, 2^(ex + ew) of nonzero codes (what a matrix
    instruction that aligns eight products cuts them against; zeros without cut)."""
    xv, wv = decode(x), decode(codes)
    y = np.zeros((xv.shape[0], wv.shape[0]))
    size, top = np.zeros_like(y), np.zeros_like(y)
    rows = np.arange(wv.shape[0]) // BLOCK
    with np.errstate(divide="ignore"):
        xe, we = (np.where(v == 0, 0.0, 2.0 ** np.floor(np.log2(np.abs(v)))) for v in (xv, wv))
    for b in range(xv.shape[1] // BLOCK):
        at = slice(BLOCK * b, BLOCK * (b + 1))
        c = np.asarray(s_x[b], np.float64)[:, None] * np.asarray(scale, np.float64)[rows, b][None, :]
        y += c * (xv[:, at] @ wv[:, at].T)
        size += np.abs(c) * (np.abs(xv[:, at]) @ np.abs(wv[:, at]).T)
        for j in range(BLOCK * b, BLOCK * (b + 1), 8) if cut else ():
            big = np.zeros_like(y)
            for i in range(j, j + 8):
                np.maximum(big, xe[:, i, None] * we[None, :, i], out=big)
            top += np.abs(c) * big
    return y, size, top
