"""The 8-bit cache in float64: codes with one power-of-two scale per block of
64 positions, and attention over them with capped, biased and masked scores.

Written from the definitions, one block, one query row at a time."""
import math

import numpy as np

BLOCK = 64
E_MIN = -100
QMAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values():
    """Value of each of the 256 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F is NaN)."""
    out = np.zeros(256)
    for c in range(256):
        s, x, m = c >> 7, c >> 3 & 15, c & 7
        v = m / 8 * 2.0 ** -6 if x == 0 else (1 + m / 8) * 2.0 ** (x - 7)
        if x == 15 and m == 7:
            v = math.nan
        out[c] = -v if s else v
    return out


def _e4m3_tables():
    v = e4m3_values()[:127]           # 0 .. 448, ascending
    return v, (v[1:] + v[:-1]) / 2    # midpoints, exact in float64


def to_grid(y, code):
    """y (already scaled) on the code's grid, ties to the even code; NaN to 0, past the range to the largest."""
    y = np.where(np.isnan(y), 0.0, np.asarray(y, dtype=np.float64))
    q = QMAX[code]
    if code == "int8":
        return np.clip(np.rint(np.clip(y, -2 * q, 2 * q)), -q, q)
    v, mid = _e4m3_tables()
    a = np.minimum(np.abs(y), q)
    lo = np.searchsorted(mid, a, side="left")        # codes whose upper midpoint lies below a
    tie = (lo < len(mid)) & (a == mid[np.minimum(lo, len(mid) - 1)])
    lo = np.where(tie & (lo % 2 == 1), lo + 1, lo)   # a tie between lo and lo + 1: the even one
    return np.copysign(v[lo], y)


def exponent(a, code):
    """The least integer e >= E_MIN with a <= QMAX 2^e."""
    e = E_MIN
    while a > QMAX[code] * 2.0 ** e:
        e += 1
    return e


def append(values, exps, rows, start, capacity, code):
    """Rows [n, 128] to positions start .. of one (layer, sequence, head) and kind.

    values [T, 64, 128]: what the codes stand for without their scale; exps [T].
    Both are changed in place."""
    rows = np.asarray(rows, dtype=np.float64)
    n = max(0, min(len(rows), capacity - start))
    for t in range(start // BLOCK, (start + n - 1) // BLOCK + 1 if n else 0):
        lo, hi = max(start, t * BLOCK), min(start + n, (t + 1) * BLOCK)
        new = rows[lo - start:hi - start]
        mag = np.abs(new)
        e = exponent(mag[np.isfinite(mag)].max(initial=0.0), code)
        if lo > t * BLOCK:
            if e > exps[t]:
                values[t] = to_grid(values[t] * 2.0 ** float(exps[t] - e), code)
            e = max(e, int(exps[t]))
        exps[t] = e
        values[t, lo - t * BLOCK:hi - t * BLOCK] = to_grid(new * 2.0 ** float(-e), code)


def visible(length, n_q, i, window=0, prefix=0, doc_start=0):
    """Truth values [length]: what query i of n_q sees."""
    t = np.arange(length)
    p = length - n_q + i
    lo = max(doc_start, 0)
    if window > 0:
        lo = max(lo, p - window + 1)
    return ((t >= lo) & (t <= p)) | (t < min(max(prefix, 0), length))


def attention_row(q, k, v, see, pos, scale=1 / math.sqrt(128), softcap=0.0, slope=0.0):
    """One query row [128] against k, v [len, 128]: (output [128], sum p |v| [128], S) with S a bound of the row's
    score magnitudes: max over the visible t of scale sum |q| |k_t|, and of the bias."""
    if not see.any():
        return np.zeros(128), np.zeros(128), 0.0
    k, v, t = k[see], v[see], np.arange(len(see))[see]
    x = k @ q * scale
    s = (np.abs(k) @ np.abs(q)).max() * scale
    if softcap > 0:
        x = softcap * np.tanh(x / softcap)
    x = x - slope * (pos - t)
    w = np.exp(x - x.max())
    w /= w.sum()
    return w @ v, w @ np.abs(v), s
