"""Plain statement of the 8-bit pool (test infrastructure only).

A K (or V) row of one token and kv head is held as e4m3 codes and one scale byte
s: value = code * 2^(s - 127). With a the row's largest magnitude, e is the least
integer >= -117 with a <= 448 * 2^e, s = e + 127, and each code is the e4m3 number
nearest to x * 2^-e, ties to the even code, or 240 where that is 256 and e is 120
(2^128 is no bf16). A row with an infinity or a NaN is held as NaN: codes 0, scale
255. The pages name no such cache: the definition
is the library's own.
"""

from __future__ import annotations

import numpy as np

from .paged_oracle import bf16_bits_to_f64


def _magnitudes():
    """The values of the codes 0 .. 126: eeee mmm is mmm * 2^-9 for exponent 0,
    else 1.mmm * 2^(eeee - 7)."""
    out = np.zeros(127)
    for c in range(127):
        e, m = c >> 3, c & 7
        out[c] = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return out


MAGNITUDES = _magnitudes()


def e4m3_values(codes):
    """fp64 values of e4m3 codes (uint8); 0x7f and 0xff are NaN."""
    codes = np.asarray(codes, dtype=np.uint8)
    mag = codes & 0x7F
    out = np.where(mag == 0x7F, np.nan, MAGNITUDES[np.minimum(mag, 126)])
    return np.where(codes & 0x80, -out, out)


def quantise_rows(bits):
    """(codes uint8 [..., D], scales uint8 [...]) of bf16 rows (bit patterns [..., D])."""
    x = bf16_bits_to_f64(bits)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    top = np.abs(x).max(axis=-1)
    e = np.full(top.shape, -117, dtype=np.int64)
    while True:
        short = 448.0 * np.exp2(e.astype(np.float64)) < top
        if not short.any():
            break
        e += short
    y = np.abs(x) / np.exp2(e.astype(np.float64))[..., None]
    hi = np.searchsorted(MAGNITUDES, y).clip(1, 126)  # MAGNITUDES[hi - 1] <= y <= MAGNITUDES[hi]
    lo = hi - 1
    up, down = MAGNITUDES[hi] - y, y - MAGNITUDES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where((e == 120)[..., None], np.minimum(code, 0x77), code)  # 0x77: 240
    code = code | np.where(np.signbit(x), 0x80, 0)
    code = np.where(bad[..., None], 0, code)
    return code.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def quant_values(codes, scales):
    """fp64 values of codes [..., D] under scale bytes [...]."""
    s = np.asarray(scales, dtype=np.float64)
    return e4m3_values(codes) * np.where(s == 255, np.nan, np.exp2(s - 127.0))[..., None]


def quant_pool_bits(codes, scales):
    """The same as bf16 bit patterns, which every value is exactly."""
    x = quant_values(codes, scales).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    back = bf16_bits_to_f64(bits)
    assert ((back == quant_values(codes, scales)) | np.isnan(back)).all()
    return bits


def quant_write(codes, scales, key, value, slots):
    """(codes, scales) of a pool [NB, 2, B, Hkv, D] after the bf16 rows key, value
    [T, Hkv, D] were written at their slots (negative ones are skipped)."""
    codes, scales = codes.copy(), scales.copy()
    B = codes.shape[2]
    for t, s in enumerate(np.asarray(slots)):
        if s < 0:
            continue
        for i, x in enumerate((key, value)):
            codes[s // B, i, s % B], scales[s // B, i, s % B] = quantise_rows(x[t])
    return codes, scales


def quant_read(key, value, codes, scales, slots):
    """(key, value) bf16 bit patterns with the pool's rows at the slots; rows of
    negative slots as they were."""
    key, value = key.copy(), value.copy()
    B = codes.shape[2]
    for t, s in enumerate(np.asarray(slots)):
        if s < 0:
            continue
        for i, x in enumerate((key, value)):
            x[t] = quant_pool_bits(codes[s // B, i, s % B], scales[s // B, i, s % B])
    return key, value
