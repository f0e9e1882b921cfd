"""The stated bound of the bfloat16 activation of the 8-bit integer products (moonep.h), which
takes the exponential and the reciprocal from instructions that are off by up to a unit in the
last place (2^-23 of the value): its steps in float32 with every combination of such errors."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


def _stated():
    """(a, b) of (a |gate| + b) * 2^-24 in the header."""
    text = open(os.path.join(ROOT, "include", "moonep.h")).read()
    found = re.search(r"\(([\d.]* ?)\|gate\| \+ (\d+)\) \* 2\^-24", text)
    return float(found[1] or 1), float(found[2])


def _constant():
    text = open(os.path.join(ROOT, "redundant_expert_balancing_amd", "csrc", "int8.hip")).read()
    return np.float32(float.fromhex(re.search(r"exp2f\(g \* (-0x[0-9a-f.]+p0)f\)", text)[1]))


def _moved(v, units):
    return v if units == 0 else np.nextafter(v, np.float32(np.inf if units > 0 else -np.inf))


def test_the_stated_bound_holds():
    a, b = _stated()
    log2e = _constant()
    rng = np.random.default_rng(0)
    # 1 + e^-gate below 2^126: beyond, the other bound holds
    g = np.concatenate([np.linspace(-87.3, 89, 400001), rng.uniform(-4, 4, 100000),
                        rng.uniform(-46, -44, 100000), [-44.371693, -44.696]]).astype(np.float32)
    g = g[g != 0]
    exact = g.astype(np.longdouble)
    exact = exact / (1 + np.exp(-exact))
    for exp_units in (-1, 0, 1):
        for rcp_units in (-1, 0, 1):
            e = np.exp2((g * log2e).astype(np.float64)).astype(np.float32)
            e = np.where(e < np.float32(2.0 ** -126), np.float32(0), _moved(e, exp_units))
            r = _moved((1.0 / (np.float32(1) + e).astype(np.float64)).astype(np.float32), rcp_units)
            off = np.abs((g * r).astype(np.longdouble) / exact - 1)
            # the product with up, one more rounding
            assert (off + U * (1 + off) <= (a * np.abs(g) + b) * U).all(), (exp_units, rcp_units)
