"""float64 oracle of the microscaled 8-bit (MXFP8, e4m3) operators: the definitions, in numpy.

A block is 32 consecutive values of a row.  Its scale is the least power of two, in [2^-127, 2^127],
that leaves max|x| at most 448; a code is the nearest e4m3 number (ties to the even code) with a sign.
A block holding an infinity or a NaN is byte 255 and zero codes.
"""
import numpy as np

BLOCK = 32
# code x m: 2^(x - 7) (1 + m / 8), or 2^-6 m / 8 for x = 0; code 0x7F is NaN
_X, _M = np.divmod(np.arange(127), 8)
GRID = np.where(_X > 0, np.exp2(_X - 7.0) * (1 + _M / 8), 2.0 ** -6 * _M / 8)
BORDER = (GRID[1:] + GRID[:-1]) / 2


def pitches(K):
    b = -(-K // BLOCK)
    return 32 * b, -(-b // 4) * 4


def _blocks(x):
    x = np.asarray(x, np.float64)
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (-x.shape[-1] % BLOCK,))], -1)
    return x.reshape(x.shape[:-1] + (-1, BLOCK))


def exponents(top):
    """The least e with top 2^-e <= 448 = 0.875 2^9, clamped; -127 for zero (frexp: top = m 2^ex)."""
    m, ex = np.frexp(top)
    return np.where(top > 0, np.clip(ex - 9 + (m > 0.875), -127, 127), -127)


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
    code = np.where(bad[..., None], 0, code + 128 * np.signbit(v))
    codes = code.reshape(code.shape[:-2] + (-1,)).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    pad = pitches(np.shape(x)[-1])[1] - scales.shape[-1]
    return codes, np.concatenate([scales, np.zeros(scales.shape[:-1] + (pad,), np.uint8)], -1)


def values(codes, scales, K=None):
    """The values the blocks stand for, rows cut to K."""
    table = np.append(GRID, np.nan)
    v = np.where(codes & 128, -1.0, 1.0) * table[codes & 127]
    b = codes.shape[-1] // BLOCK
    s = scales[..., :b].astype(np.float64)
    p = np.where(s == 255, np.nan, np.exp2(s - 127))
    return (v * np.repeat(p, BLOCK, -1))[..., :K]


def fake(x):
    return values(*quantize(x), K=np.shape(x)[-1])


def quantize_slack(a, rel):
    """How far fake(a') may be from fake(a), element by element, for any a' within a (1 +- rel): the
    distance to a neighbouring code where a border is that near; where the block's scale may change,
    half a step of either grid, together at most a step of the coarser one."""
    v = _blocks(a)
    top = np.abs(v).max(-1)
    e = exponents(top)
    m = np.abs(np.ldexp(v, -e[..., None]))
    lo = np.clip(np.searchsorted(GRID, m, side="right") - 1, 0, len(GRID) - 2)
    slack = np.where(np.abs(m - BORDER[lo]) <= rel * BORDER[lo], GRID[lo + 1] - GRID[lo], 0.0)
    change = (exponents(top * (1 + rel)) != e) | (exponents(top * (1 - rel)) != e)
    coarse = np.maximum(np.exp2(np.floor(np.log2(np.maximum(m, 2.0 ** -20))) - 3), 2.0 ** -8)
    coarse = coarse * (1 + 2 * rel) + 2 * rel * m
    slack = np.where(change[..., None], coarse, slack) * np.exp2(e)[..., None]
    return slack.reshape(slack.shape[:-2] + (-1,))[..., : np.shape(a)[-1]]
