"""Pins of the block-scaled formats' oracle against torch's e4m3 and the stated bounds."""
import numpy as np
import torch

from oracle import formats as F


def test_e4m3_values_and_rounding_match_torch():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, F.E4M3)
    v = np.random.default_rng(0).uniform(-448, 448, 20000).astype(np.float32)
    v = np.concatenate([v, v * 2.0 ** -12, (F.E4M3[1:] + F.E4M3[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.codes(v, F.E4M3, 128), want)


def test_e2m1_ties_go_to_the_even_code():
    mids = (F.E2M1[1:] + F.E2M1[:-1]) / 2
    assert F.values(F.codes(mids, F.E2M1, 8), F.E2M1, 8).tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]


def test_scales_clip_nothing_and_are_the_smallest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 64)) * 2.0 ** rng.integers(-20, 20, (50, 1))
    for top, f in ((448.0, F.checkpoint), (6.0, F.mx)):
        s = f(x)[1].astype(int) - 127
        amax = np.abs(x).reshape(50, 2, 32).max(-1)
        assert (amax <= top * 2.0 ** s).all() and (amax > top * 2.0 ** (s - 1.0)).all()
    assert F.scale_bytes(np.zeros((1, 32)), 6.0)[0] == 0
    assert F.scale_bytes(np.array([[1.0, np.nan]]), 6.0)[0] == 255


def test_errors_stay_within_half_a_step():
    x = np.random.default_rng(2).standard_normal((40, 96))
    for f, val, rel, low in ((F.checkpoint, F.checkpoint_values, 2.0 ** -4, 2.0 ** -10),
                             (F.mx, F.mx_values, 2.0 ** -2, 2.0 ** -2)):
        q, s = f(x)
        scale = np.repeat(2.0 ** (s.astype(float) - 127), 32, 1)
        assert (np.abs(val(q, s) - x) <= np.maximum(rel * np.abs(x), low * scale)).all()


def test_checkpoints_of_the_largest_values_stay_finite():
    """What rounds up to 256 * 2^120 = 2^128 is kept as 240 * 2^120, still within 2^-4."""
    big = np.float32([np.finfo(np.float32).max, 248.0 * 2.0 ** 120, 247.99 * 2.0 ** 120, 240.0 * 2.0 ** 120])
    x = np.concatenate([big, -big, np.ones(24, np.float32)])[None].astype(np.float64)
    v = F.checkpoint_values(*F.checkpoint(x))
    assert (np.abs(v[0, :8]) == 240.0 * 2.0 ** 120).all() and np.isfinite(v.astype(np.float32)).all()
    assert (np.abs(v - x)[0, :8] <= 2.0 ** -4 * np.abs(x)[0, :8]).all()
    assert F.checkpoint(np.array([[np.inf] * 32]))[1][0, 0] == 255
