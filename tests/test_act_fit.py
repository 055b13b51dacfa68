"""The polynomial of the activations' normal share as its coefficients stand in the
source, evaluated in 64 bits against the complementary error function: off by no more
than the comment beside them says."""
import math
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "uniform_grid_fp4_amd", "csrc", "act_device.h")


def test_the_fit_is_as_close_as_stated():
    text = open(SRC).read()
    first = re.search(r"float p = (-?[\d.]+)f;", text)
    more = re.findall(r"p = __builtin_fmaf\(p, t, (-?[\d.]+)f\);", text)
    coefficients = [np.float64(np.float32(c)) for c in (first.group(1), *more)]
    assert len(coefficients) == 10
    stated = re.search(r"within ([\d.]+e-\d+) of log\(erfc", re.sub(r"\n// ", " ", text))
    t = np.linspace(0.155, 1.0, 200001)
    z = 2.0 / t - 2.0
    # erfc stays normal and exp(z^2) finite down to this t
    want = np.array([math.log(math.erfc(v)) for v in z]) + z * z - np.log(t)
    off = np.abs(np.polyval(coefficients, t) - want).max()
    assert off <= float(stated.group(1)), off
    assert off >= 0.9 * float(stated.group(1)), off
