"""Bit-level CPU oracle of the microscaled context cache: e4m3 values, one power-of-two scale per 32
elements.

TEST INFRASTRUCTURE ONLY (same rule as ``oracle.oracle``).

Definition: for each block of 32 elements, amax is the largest finite magnitude, e the least integer
>= -127 with amax <= 448 * 2^e (e = -127 for a block without a non-zero finite element); the scale byte
is e + 127 and each element is the e4m3 number nearest to x * 2^-e, ties to the even mantissa, an
infinity saturating to 448 and NaN staying NaN.  The list of all e4m3 numbers is written out from the
format (4 exponent bits, bias 7, 3 mantissa bits, S.1111.111 is NaN) and the nearest is searched in it.
"""
from __future__ import annotations

import numpy as np

__all__ = ["E4M3", "quantise", "values", "kv_append_mx", "kv_read_mx"]


def _e4m3_table():
    t = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = np.nan
        t[code] = -x if code & 128 else x
    return t


E4M3 = _e4m3_table()
_POS = E4M3[:127]          # 0 .. 448, ascending: the code is the index


def quantise(x):
    """x [..., D] float64 -> (codes uint8 [..., D], scale bytes uint8 [..., D / 32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    mag = np.where(np.isfinite(b), np.abs(b), 0.0)
    amax = mag.max(axis=-1)
    e = np.full(amax.shape, -127)
    some = amax > 0
    guess = np.floor(np.log2(np.where(some, amax, 1.0))).astype(int) - 9
    for _ in range(3):
        guess = np.where(amax > 448.0 * np.exp2(guess.astype(float)), guess + 1, guess)
    e[some] = np.maximum(guess[some], -127)
    with np.errstate(invalid="ignore", over="ignore"):
        y = b / np.exp2(e.astype(float))[..., None]
    a = np.where(np.isnan(y), 0.0, np.minimum(np.abs(y), 448.0))
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _POS[lo], _POS[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == _POS[hi], hi, code)
    code = np.where(np.isnan(y), 127, code)
    code = code | np.where(np.signbit(y), 128, 0)
    return code.reshape(x.shape).astype(np.uint8), (e + 127).astype(np.uint8)


def values(codes, scales):
    """What codes [..., D] and scale bytes [..., D / 32] stand for, in float64."""
    e = scales.astype(np.float64) - 127
    return E4M3[codes] * np.repeat(np.exp2(e), 32, axis=-1)


def kv_append_mx(new, codes, scales, ctx_lens, counts, advance=True):
    """One of K and V: new [B, T, Hkv, D] float64 into slabs codes [B, Hkv, cap, D] and scales, copied.
    Returns (codes', scales', lens', bad)."""
    codes, scales = codes.copy(), scales.copy()
    lens = np.array(ctx_lens, dtype=np.int64)
    B, T = new.shape[:2]
    bad = np.zeros(B, dtype=bool)
    for n in range(B):
        L, c = int(ctx_lens[n]), int(counts[n])
        if L < 0 or c < 0 or c > T or L + c > codes.shape[2]:
            bad[n] = True
            continue
        q, s = quantise(new[n, :c])
        codes[n, :, L:L + c] = q.transpose(1, 0, 2)
        scales[n, :, L:L + c] = s.transpose(1, 0, 2)
        if advance:
            lens[n] = L + c
    return codes, scales, lens, bad


def kv_read_mx(codes, scales, ctx_lens, starts, out):
    """Rows back into out [B, Hkv, T, D] (copied): out[n, :, t] = position starts[n] + t below ctx_lens[n]."""
    out = out.copy()
    for n in range(out.shape[0]):
        a = int(starts[n])
        b = min(a + out.shape[2], int(ctx_lens[n]))
        if b > a:
            out[n, :, :b - a] = values(codes[n, :, a:b], scales[n, :, a:b])
    return out
