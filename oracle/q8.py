"""8-bit layer operators in fp64 -- TEST INFRASTRUCTURE ONLY (plain numpy).

An 8-bit matrix is held here as (values of the codes fp64 [rows, 128 * nb],
scale bytes [groups, 4 * ceil(nb / 4)]); every operator is written from its
definition, one block at a time where that is plainest.
"""
import numpy as np
from scipy.special import erfc

BLOCK = 128

# The non-negative e4m3 numbers in code order: 0, seven subnormals, then
# (1 + f / 8) 2^(x - 7); code 127 is NaN, so the largest is 448.
E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def round_e4m3(v):
    """Nearest e4m3 number of each |v| <= 448, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(E4M3[code], v)


def exponent(amax):
    """Smallest integer e in [-117, 120] with amax <= 448 * 2^e."""
    e = -117
    while e < 120 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantize(x, block_rows=1):
    """(code values, scale bytes); a block with a non-finite element is NaN, byte 255."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb, groups = -(-cols // BLOCK), -(-rows // block_rows)
    codes = np.zeros((rows, nb * BLOCK))
    scales = np.full((groups, -(-nb // 4) * 4), 127, np.uint8)
    for g in range(groups):
        for b in range(nb):
            part = x[g * block_rows:(g + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK]
            at = codes[g * block_rows:(g + 1) * block_rows, b * BLOCK:b * BLOCK + part.shape[1]]
            if not np.isfinite(part).all():
                scales[g, b] = 255
                at[...] = np.nan
                continue
            e = exponent(np.abs(part).max())
            scales[g, b] = e + 127
            at[...] = round_e4m3(part * 2.0 ** -e)
            if e == 120:  # 256 * 2^120 is past fp32's range
                at[...] = np.clip(at, -240.0, 240.0)
    return codes, scales


def values(codes, scales, cols, block_rows=1):
    rows, width = codes.shape
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    s = np.repeat(np.repeat(s, block_rows, 0)[:rows], BLOCK, 1)[:, :width]
    return (codes * s)[:, :cols]


def held(x, block_rows=1):
    """x as its 8-bit form holds it."""
    return values(*quantize(x, block_rows), np.asarray(x).shape[1], block_rows)


def cdf(z):
    return 0.5 * erfc(-z / np.sqrt(2.0))


def gelu(z):
    return z * cdf(z)


def gelu_slope(z):
    return cdf(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)


def rms_norm(h, gamma, eps):
    """(y before the 8 bits, rstd)."""
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * gamma, rstd


def rms_norm_bwd(dy, h, rstd, gamma, dres=None):
    n, g = h * rstd[:, None], dy * gamma
    dh = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return dh if dres is None else dh + dres, (dy * n).sum(0)
