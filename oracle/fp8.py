"""Block-scaled FP8 linear layer, dense and by expert, in float64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Per row and 128 elements along K (the last block may be shorter):
    amax = largest finite |x|,  s = 2^e, e the smallest integer >= -127 with
    amax <= 448 * 2^e (e = -127 for a block of zeros),
    code = nearest e4m3 of x / s, ties to even; NaN for an infinity or NaN.
q(x) is the value the code and the scale stand for.
    Y = epilogue(q(X) q(W) + b)
"""
import numpy as np

BLOCK = 128
MAX = 448.0


def _blocks(x):
    x = np.asarray(x, dtype=np.float64)
    k = x.shape[-1]
    pad = np.zeros(x.shape[:-1] + (-k % BLOCK,))
    return np.concatenate([x, pad], -1).reshape(x.shape[:-1] + (-1, BLOCK))


def quantize(x):
    """x [..., K] -> (values under the scale [..., KS, 128], NaN where x is not finite; exponents [..., KS])."""
    b = _blocks(x)
    fin = np.where(np.isfinite(b), np.abs(b), 0.0)
    amax = fin.max(-1)
    e = np.full(amax.shape, -127, dtype=np.int64)
    # by definition, not by logarithm: raise e until 448 * 2^e covers amax
    while True:
        low = MAX * np.exp2(e.astype(np.float64)) < amax
        if not low.any():
            break
        e = np.where(low, e + 1, e)
    u = np.where(np.isfinite(b), b, 0.0) / np.exp2(e.astype(np.float64))[..., None]
    return np.where(np.isfinite(b), e4m3_round(u), np.nan), e


def e4m3_round(u):
    """Nearest e4m3 value of |u| <= 448, ties to even: the steps are 2^(p-3) between 2^p and 2^(p+1), 2^-9
    below 2^-6."""
    _, e2 = np.frexp(np.abs(u))
    step = np.exp2(np.maximum(e2 - 1.0, -6.0) - 3.0)
    return np.copysign(np.rint(np.abs(u) / step) * step, u)


def encode(v):
    """e4m3 bit patterns of exact e4m3 values (0x7F for NaN)."""
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    _, e2 = np.frexp(a)
    e = e2 - 1
    sub = a < 2.0 ** -6
    code = np.where(sub, a * 512.0, (e + 7) * 8 + (a / np.exp2(e.astype(np.float64)) - 1.0) * 8.0)
    code = np.where(a == 0.0, 0.0, code).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 7)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def decode(code):
    c = np.asarray(code, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    a = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    a = np.where((c & 127) == 127, np.nan, a)
    return np.where(c & 128, -a, a)


def value(x):
    """q(x), [..., K]."""
    v, e = quantize(x)
    y = v * np.exp2(e.astype(np.float64))[..., None]
    return y.reshape(y.shape[:-2] + (-1,))[..., :np.asarray(x).shape[-1]]


def gelu(y, kind):
    if kind == 1:
        from math import erfc, sqrt
        return 0.5 * y * np.vectorize(lambda t: erfc(-t / sqrt(2.0)) if t == t else t)(y)
    if kind == 2:
        z = np.sqrt(2.0 / np.pi) * (y + 0.044715 * y ** 3)
        return 0.5 * y * (1.0 + np.tanh(z))
    return y


def linear(x, w, b=None, epilogue=0, gelu_col_begin=0):
    """x [M, K], w [K, N], b [N] -> (Y [M, N] float64 before any rounding, sum of the terms' magnitudes)."""
    qx, qw = value(x), value(np.asarray(w).T).T
    y, mag = qx @ qw, np.abs(qx) @ np.abs(qw)
    if b is not None:
        y, mag = y + b, mag + np.abs(b)
    out = y.copy()
    if epilogue:
        out[:, gelu_col_begin:] = gelu(y[:, gelu_col_begin:], epilogue)
    return out, mag


def experts(x, w, offsets, b=None, epilogue=0, gelu_col_begin=0):
    """Rows offsets[e]..offsets[e+1]-1 of x meet w[e], b[e]; NaN in the rows of no expert."""
    out = np.full((x.shape[0], w.shape[2]), np.nan)
    mag = np.zeros(out.shape)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        if s.stop > s.start:
            out[s], mag[s] = linear(x[s], w[e], None if b is None else b[e], epilogue, gelu_col_begin)
    return out, mag
