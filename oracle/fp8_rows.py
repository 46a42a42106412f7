"""Plain definition of the 8-bit cache's rows (numpy, float64; test
infrastructure).

A row of d values x is codes c (e4m3) and an exponent s: s is the smallest
integer with max|x| <= 448 * 2^s over the finite values, held within [-56, 40];
c is the e4m3 value nearest to x * 2^-s, ties to the even code, saturating.
"""
import numpy as np

S_MIN, S_MAX = -56, 40


def code_values() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    exponent 0 is subnormal and the all-ones code is NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = float("nan") if (e, m) == (15, 7) else v
        if c >= 128:
            out[c] = -out[c]
    return out


_VALUES = code_values()
_POSITIVE = _VALUES[:127]  # ascending, 0 .. 448


def exponent(x: np.ndarray) -> np.ndarray:
    """s of rows x [..., d]."""
    a = np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1)
    s = np.full(a.shape, S_MIN, dtype=np.int64)
    for e in range(S_MIN, S_MAX):  # raise s while the row does not fit
        s = np.where((s == e) & (a > 448.0 * 2.0 ** e), e + 1, s)
    return s


def encode(x: np.ndarray):
    """Rows x [..., d] (float64) -> (codes uint8 [..., d], scale bytes uint8 [...])."""
    s = exponent(x)
    y = np.abs(x) * 2.0 ** -s[..., None].astype(np.float64)
    y = np.minimum(y, 448.0)  # NaN stays
    hi = np.clip(np.searchsorted(_POSITIVE, np.nan_to_num(y), side="left"), 1, 126)
    lo = hi - 1
    dlo, dhi = y - _POSITIVE[lo], _POSITIVE[hi] - y
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(y), 127, code)
    code = code + np.where(np.signbit(x) & ~np.isnan(y), 128, 0)
    return code.astype(np.uint8), (s + 127).astype(np.uint8)


def decode(codes: np.ndarray, scale_bytes: np.ndarray) -> np.ndarray:
    """Codes [..., d] and bytes [...] -> float64 values."""
    return _VALUES[codes] * 2.0 ** (scale_bytes.astype(np.float64) - 127)[..., None]
