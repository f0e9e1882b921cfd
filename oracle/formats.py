"""Block-scaled 8- and 4-bit formats by their definition.  TEST INFRASTRUCTURE.

OCP e4m3 and e2m1 values with one power-of-two scale per 32 values (bytes: exponent plus
127, 255 is NaN), the scale the smallest 2^e, e >= -127, that clips nothing (moonep.h).
Rounding is by search over the type's finite values, ties to the even code.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def _e4m3_values():
    """Values of codes 0..126 (127 is NaN)."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = _e4m3_values()
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def codes(v, table, sign_bit):
    """Codes of v (no magnitude above the table's largest), to nearest, ties to even."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.searchsorted(table, a, side="left").clip(0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(table[hi] == a, hi, pick)
    return (pick | np.where(np.signbit(v), sign_bit, 0)).astype(np.uint8)


def values(code, table, sign_bit):
    code = np.asarray(code).astype(int)
    v = table[code & (sign_bit - 1)]
    return np.where(code & sign_bit, -v, v)


def scale_bytes(blocks, top):
    """Scale byte of every block [..., n]."""
    amax = np.abs(np.asarray(blocks, dtype=np.float64)).max(-1)
    out = np.zeros(amax.shape, dtype=np.uint8)
    for at in np.ndindex(amax.shape):
        a = amax[at]
        if not np.isfinite(a):
            out[at] = 255
            continue
        e = -127
        while a > top * 2.0 ** e:
            e += 1
        out[at] = e + 127
    return out


def quantise(x, table, top, sign_bit):
    """(codes [rows, width], scale bytes [rows, ceil(width/32)]) of float64 x [rows, width];
    the codes of a NaN block are 0."""
    rows, width = x.shape
    nb = -(-width // BLOCK)
    pad = np.zeros((rows, nb * BLOCK))
    pad[:, :width] = x
    blocks = pad.reshape(rows, nb, BLOCK)
    s = scale_bytes(blocks, top)
    bad = (s == 255)[..., None]
    q = codes(np.where(bad, 0.0, blocks) / 2.0 ** (np.where(bad, 127, s[..., None]) - 127.0), table,
              sign_bit)
    return np.where(bad, 0, q).reshape(rows, -1)[:, :width].astype(np.uint8), s


def dequantise(q, s, table, sign_bit):
    rows, width = q.shape
    scale = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return values(q, table, sign_bit) * np.repeat(scale, BLOCK, axis=1)[:, :width]


def checkpoint(x):
    """Finite magnitudes above 240 * 2^120 become that value: rounded up they would be 2^128,
    which float32 does not hold."""
    x = np.asarray(x, dtype=np.float64)
    top = 240.0 * 2.0 ** 120
    return quantise(np.where(np.isfinite(x), np.clip(x, -top, top), x), E4M3, 448.0, 128)


def checkpoint_values(q, s):
    return dequantise(q, s, E4M3, 128)


def mx(x):
    """Codes (one per value) and scale bytes of 4-bit rows."""
    return quantise(np.asarray(x, dtype=np.float64), E2M1, 6.0, 8)


def mx_values(q, s):
    return dequantise(q, s, E2M1, 8)


def mx_pack_rows(q, s):
    """Token-row layout of codes [rows, width] and scales [rows, width/32]."""
    rows, width = q.shape
    T, C = -(-width // 128), -(-width // 512)
    out, sc = np.zeros((rows, 64 * T), np.uint8), np.zeros((rows, 16 * C), np.uint8)
    for k in range(width):
        out[:, k // 2] |= q[:, k] << (4 * (k % 2))
    for b in range(s.shape[1]):
        sc[:, 16 * (b // 16) + 4 * (b % 4) + (b // 4) % 4] = s[:, b]
    return out, sc


def mx_pack_weight(q, s):
    """Weight layout of one expert: codes [Hp, H] and scales [Hp, H/32] (rows are columns n)."""
    Hp, H = q.shape
    T, C = -(-H // 128), -(-H // 512)
    out, sc = np.zeros((Hp // 16, T, 64, 16), np.uint8), np.zeros((Hp // 16, C, 64, 4), np.uint8)
    n = np.arange(Hp)
    for k in range(H):
        lane = 16 * ((k // 32) % 4) + n % 16
        out[n // 16, k // 128, lane, (k % 32) // 2] |= q[:, k] << (4 * (k % 2))
        if k % 32 == 0:
            sc[n // 16, k // 512, lane, (k // 128) % 4] = s[:, k // 32]
    return out, sc
