"""The block-scaled FP8 operators' definition in 64 bits (numpy), for the
tests: blocks of 128 along a row, bias = floor(log2(max / amax)), codes to
nearest even, values code * 2^-bias. Written from the formulas."""
import numpy as np

from oracle import E4M3, E5M2, encode
from oracle.formats import decode_table

BLOCK = 128
FMT = {"e4m3": E4M3, "e5m2": E5M2}
TOP = {"e4m3": (448.0, 8), "e5m2": (57344.0, 15)}
BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}          # mantissa bits, least normal exponent
BF16_HALF = 2.0 ** -8                               # half a bf16 step, relative
MFMA = 1e-4                                         # sums of the FP8 matrix instructions, relative to the sum of |a b|


def bias_of(amax: float, fmt: str) -> int:
    top, e_top = TOP[fmt]
    if amax == 0 or not np.isfinite(amax):
        return 0
    m, e = np.frexp(amax)
    b = e_top - (int(e) - 1)
    if np.ldexp(amax, b) > top:
        b -= 1
    return max(-126, min(126, b))


def blocks(x, fmt, biases=None):
    """codes [r, c rounded up to 128] (uint8) and biases [r, blocks] of x (float64); biases: taken as given."""
    x = np.asarray(x, dtype=np.float64)
    r, c = x.shape
    nb = -(-c // BLOCK)
    p = np.zeros((r, nb, BLOCK))
    p.reshape(r, -1)[:, :c] = x
    if biases is None:
        with np.errstate(invalid="ignore"):
            amax = np.max(np.abs(p), axis=2) if p.size else np.zeros((r, nb))
        biases = np.array([bias_of(float(a), fmt) for a in amax.ravel()], dtype=np.int32).reshape(r, nb)
    codes = np.zeros((r, nb, BLOCK), dtype=np.uint8)
    for i in range(r):
        for j in range(nb):
            codes[i, j] = encode(p[i, j] * 2.0 ** biases[i, j], FMT[fmt])
    return codes.reshape(r, nb * BLOCK), biases


def held(x, fmt="e4m3", slack=0.0):
    """The values of x's stored form; with slack > 0 also, for each element,
    how far its value may be off if x is off by slack relative: the distance
    to the values of its neighbours at x (1 - slack) and x (1 + slack), under
    either's scales; 0 where no rounding border and no border of the scale
    rule is that near."""
    x = np.asarray(x, dtype=np.float64)

    def value(x, biases=None):
        codes, biases = blocks(x, fmt, biases)
        per = np.repeat(biases, BLOCK, axis=1).astype(np.float64)
        return (decode_table(FMT[fmt])[codes] * 2.0 ** -per)[:, :x.shape[1]], biases
    v, _ = value(x)
    if not slack:
        return v
    lo, hi = x * (1 - slack), x * (1 + slack)
    (vl, bl), (vh, bh) = value(lo), value(hi)
    unsure = np.maximum(np.abs(vl - v), np.abs(vh - v))
    if not np.array_equal(bl, bh):
        for w in (value(lo, bh)[0], value(hi, bl)[0]):
            unsure = np.maximum(unsure, np.abs(w - v))
    return v, unsure


def to_bf16(x):
    """Nearest bf16 (ties to even) of float64 values within its normal range."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256) / 256, e)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))
