"""float64 oracle of the microscaled 4-bit (MXFP4) operators: the definitions, in numpy.

A block is 32 consecutive values of a row.  Its scale is 2^(floor(log2 max|x|) - 2), clamped to
[2^-127, 2^127]; a code is the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, larger
magnitudes to 6) with a sign.  A block holding an infinity or a NaN is byte 255 and zero codes.
"""
import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BORDER = (GRID[1:] + GRID[:-1]) / 2


def pitches(K):
    b = -(-K // BLOCK)
    return 16 * b, -(-b // 4) * 4


def _blocks(x):
    x = np.asarray(x, np.float64)
    K = x.shape[-1]
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (-K % BLOCK,))], -1)
    return x.reshape(x.shape[:-1] + (-1, BLOCK))


def exponents(top):
    """floor(log2(top)) - 2 clamped, -127 for zero; exact (frexp: top = m 2^ex, 0.5 <= m < 1)."""
    _, ex = np.frexp(top)
    return np.where(top > 0, np.clip(ex - 3, -127, 127), -127)


def quantize(x):
    """(codes, scales) bytes of the rows of x."""
    v = _blocks(x)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    e = exponents(np.abs(v).max(-1))
    m = np.abs(np.ldexp(v, -e[..., None]))
    up = np.searchsorted(BORDER, m, side="left")      # a value on a border: the lower code ...
    on = np.searchsorted(BORDER, m, side="right")     # ... or the upper one,
    code = np.where((on != up) & (up % 2 == 1), on, up)  # whichever is even
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(v))
    code = code.reshape(code.shape[:-2] + (-1,)).astype(np.uint8)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    pad = pitches(np.shape(x)[-1])[1] - scales.shape[-1]
    return codes, np.concatenate([scales, np.zeros(scales.shape[:-1] + (pad,), np.uint8)], -1)


def values(codes, scales, K=None):
    """The values the blocks stand for, rows cut to K."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(n & 8, -1.0, 1.0) * GRID[n & 7]
    b = n.shape[-1] // BLOCK
    s = scales[..., :b].astype(np.float64)
    p = np.where(s == 255, np.nan, np.exp2(s - 127))
    return (v * np.repeat(p, BLOCK, -1))[..., :K]


def fake(x):
    return values(*quantize(x), K=np.shape(x)[-1])


def silu_mul(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def quantize_slack(a, rel):
    """How far fake(a') may be from fake(a), element by element, for any a' within a (1 +- rel):
    the distance to a neighbouring code where a border is that near, and where the block's scale
    may change, the larger of the two scales' errors on both sides."""
    v = _blocks(a)
    top = np.abs(v).max(-1)
    e = exponents(top)
    m = np.abs(np.ldexp(v, -e[..., None]))
    slack = np.zeros_like(m)
    for lo, hi, b in zip(GRID[:-1], GRID[1:], BORDER):
        slack = np.where(np.abs(m - b) <= rel * b, hi - lo, slack)
    # values near zero: a code of 0 either way
    slack = slack * np.exp2(e)[..., None]
    change = (exponents(top * (1 + rel)) != e) | (exponents(top * (1 - rel)) != e)
    # under one scale or its double every value is off by at most a step of the coarser grid
    coarse = np.maximum(2.0, np.where(m > 4, 4.0, 0.0)) * 2 * np.exp2(e)[..., None]
    slack = np.where(change[..., None], coarse, slack)
    return slack.reshape(slack.shape[:-2] + (-1,))[..., : np.shape(a)[-1]]
