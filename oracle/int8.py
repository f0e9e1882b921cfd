"""8-bit integers with a scale per row by their definition, and the products and gradients on
them, in float64.  TEST INFRASTRUCTURE.

A row's scale is max(amax / 127, 2^-126) rounded to float32; a value is held as the whole
number nearest to value / scale, ties to even (moonep.h). Products of whole numbers are exact.
"""
from __future__ import annotations

import numpy as np

from . import ffn as FF

LEAST = 2.0 ** -126


def rows(x):
    """(whole values [rows, width] as float64, scales [rows]) of float64 rows x."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    x = np.where(bad[:, None], 0.0, x)
    scale = np.maximum(np.abs(x).max(axis=1, initial=0.0) / 127.0, LEAST).astype(np.float32)
    scale = scale.astype(np.float64)
    # x and scale have 24 bits: a quotient that is not half-way between whole numbers is
    # further from that than a float64 rounding
    q = np.rint(x / scale[:, None])
    return q, np.where(bad, np.nan, scale)


def values(q, scale):
    return q * scale[:, None]


def weight(w):
    """(whole values [H, Hp], scales [Hp]) of one expert's weight [H, Hp]."""
    q, s = rows(np.asarray(w, dtype=np.float64).T)
    return q.T, s


def pack_rows(q):
    """Token-row layout int8 [rows, 128*ceil(width/128)]."""
    n, width = q.shape
    out = np.zeros((n, 128 * -(-width // 128)), np.int8)
    out[:, :width] = q
    return out


def pack_weight(q):
    """Weight layout of one expert's whole values [H, Hp]."""
    H, Hp = q.shape
    out = np.zeros((-(-Hp // 16), 2 * -(-H // 128), 64, 16), np.int8)
    for k in range(H):
        n = np.arange(Hp)
        out[n // 16, k // 64, 16 * ((k // 16) % 4) + n % 16, k % 16] = q[k]
    return out


def pack_scales(s):
    """Column scales padded with zeros to a multiple of 16."""
    out = np.zeros(16 * -(-len(s) // 16), np.float32)
    out[:len(s)] = s
    return out


def product(qx, sx, qw, sw):
    """float64 rows of (qx @ qw) scaled by rows and columns."""
    return (qx @ qw) * sx[:, None] * sw[None, :]


def swiglu(h):
    """act of h (interleaved gate/up columns), unrounded."""
    gate, up = FF.gate_up_columns(h.shape[1] // 2)
    return FF.silu(h[:, gate]) * h[:, up]


def grad_rows(dc, sw, gates=None):
    """(whole values, scales) of upstream rows dc times the columns' scales sw [rows, width],
    which product is held in float32; the gate multiplies the scale."""
    g = (np.asarray(dc, dtype=np.float64) * np.asarray(sw, dtype=np.float64)).astype(np.float32)
    q, s = rows(g)
    return q, s if gates is None else s * gates
