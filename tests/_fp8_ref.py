"""The 8-bit layer in 64 bits, plainly (numpy on the CPU; no library code).

E4M3 values by their definition: 1 sign, 4 exponent (bias 7), 3 mantissa
bits; 0x7F / 0xFF are NaN, 448 the largest value.  Scales are bytes b standing
for 2^(b - 127).  Every encoder takes fp64 values, so a tolerance can be given
to it as an interval of values (`between`)."""

import math

import numpy as np

BLOCK = 128


def _e4m3_table():
    out = np.empty(256)
    for c in range(256):
        s, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        out[c] = s * (m / 8.0 * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7))
    out[0x7F] = out[0xFF] = np.nan
    return out


E4M3 = _e4m3_table()
_POS = E4M3[:0x7F]                       # 0 ... 448, ascending; code = index
_MID = (_POS[1:] + _POS[:-1]) / 2.0      # borders between neighbours (exact)


def e4m3_encode(u):
    """fp64 -> codes, nearest, ties to the even code, saturating at 448."""
    a = np.abs(u)
    lo = np.searchsorted(_MID, a, side="left")    # a == _MID[i] -> i, the lower code
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.int64)
    return np.where(np.signbit(u), code + 128, code).astype(np.uint8)


def scale_byte(amax):
    """Smallest b >= 0 with amax <= 448 * 2^(b - 127)."""
    out = np.zeros(np.shape(amax), dtype=np.uint8)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            e = math.frexp(a / 448.0)[1] - 1
            while a > 448.0 * 2.0 ** e:
                e += 1
            while a <= 448.0 * 2.0 ** (e - 1):
                e -= 1
            out[i] = max(e, -127) + 127
    return out


def blocks(v):
    rows, K = v.shape
    n = -(-K // BLOCK)
    out = np.zeros((rows, n * BLOCK))
    out[:, :K] = v
    return out.reshape(rows, n, BLOCK)


def encode(v):
    """fp64 [rows][K] -> (codes uint8 [rows][K], scale bytes [rows][blocks])."""
    rows, K = v.shape
    b = blocks(v)
    s = scale_byte(np.abs(b).max(axis=2))
    codes = e4m3_encode(b * np.exp2(127.0 - s.astype(np.float64))[:, :, None])
    return codes.reshape(rows, -1)[:, :K], s


def tiles(s):
    """Scale bytes [rows][blocks] -> the tile layout, byte by byte."""
    rows, n = s.shape
    nt = -(-n // 4)
    out = np.zeros(-(-rows // 128) * nt * 512, dtype=np.uint8)
    for r in range(rows):
        for j in range(n):
            out[((r // 128) * nt + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4] = s[r, j]
    return out


def untile(flat, rows, K):
    """-> (scale bytes [rows][blocks], mask of the layout's other bytes)."""
    n = -(-K // BLOCK)
    nt = -(-n // 4)
    r, j = np.meshgrid(np.arange(rows), np.arange(n), indexing="ij")
    at = ((r // 128) * nt + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    rest = np.ones(flat.shape, dtype=bool)
    rest[at.reshape(-1)] = False
    return flat[at], rest


def decode(codes, s):
    """codes uint8 [rows][K], scale bytes [rows][blocks] -> fp64 values."""
    rows, K = codes.shape
    f = np.exp2(s.astype(np.float64) - 127.0)
    return E4M3[codes] * np.repeat(f, BLOCK, axis=1)[:, :K]


def assert_encodes(codes, flat_scales, v, err):
    """The codes and scales are an encoding of values within `err` (fp64, same
    shape as v) of v: each scale is one that an amax in the block's interval
    takes, and each code one that a value in [v - err, v + err] takes under
    the block's own scale.  Padding scales are 0."""
    rows, K = v.shape
    s, rest = untile(flat_scales, rows, K)
    assert not flat_scales[rest].any(), "padding scales are not 0"
    a, e = np.abs(blocks(v)), blocks(err)
    lo = scale_byte(np.maximum(a - e, 0.0).max(axis=2))
    hi = scale_byte((a + e).max(axis=2))
    bad = (s < lo) | (s > hi)
    assert not bad.any(), f"{bad.sum()} scales outside their interval, first at {np.argwhere(bad)[0]}"
    f = np.repeat(np.exp2(127.0 - s.astype(np.float64)), BLOCK, axis=1)[:, :K]
    got = E4M3[codes]
    low, high = E4M3[e4m3_encode((v - err) * f)], E4M3[e4m3_encode((v + err) * f)]
    bad = ~((got >= low) & (got <= high))
    assert not bad.any(), (f"{bad.sum()} codes outside their interval, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} not in [{low[bad][0]}, {high[bad][0]}]")


def gelu(v):
    """x Phi(x) in fp64, without cancellation for negative x."""
    from scipy.special import ndtr
    return v * ndtr(v)


def bf16_round(v):
    """fp64 -> the nearest bf16 value (ties to even), as fp64.  Normal range."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(np.ldexp(m, 8)), e - 8)
