"""The selection's exponential: its polynomial, as it stands in the source, against
2^f over the whole interval.  The header promises each exponential to 1e-10 of
itself, the code's own comment 5e-11; the check in extended precision is of the
polynomial alone, the 64-bit roundings of its steps (eight of 2^-53) come on
top and are below 1e-15."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gram_memory_layer_amd", "csrc",
                   "beam.hip")


def test_polynomial_is_within_its_bound():
    body = re.search(r"double exp2_near\(.*?\{(.*?)return", open(SRC).read(), re.S).group(1)
    coef = [re.search(r"double p = ([-0-9.e]+);", body).group(1)]
    coef += re.findall(r"p = __builtin_fma\(p, f, ([-0-9.e]+)\);", body)
    assert len(coef) == 8 and float(coef[-1]) == 1.0
    f = np.linspace(-0.5, 0.5, 200001).astype(np.longdouble)
    p = np.full_like(f, float(coef[0]))
    for c in coef[1:]:
        p = p * f + np.longdouble(float(c))
    exact = np.exp2(f)
    worst = float(np.abs((p - exact) / exact).max())
    assert worst < 5e-11, worst


def test_sampling_weights_polynomial_is_within_its_bound():
    """The header promises each weight to 2e-12 of itself, the code's comment 1.1e-12 for the polynomial;
    what its argument's roundings add is below 1000 * 2^-52."""
    src = open(os.path.join(os.path.dirname(SRC), "sample.hip")).read()
    body = re.search(r"double weight\(double d.*?\{(.*?)return", src, re.S).group(1)
    coef = [re.search(r"double p = ([-0-9.e]+);", body).group(1)]
    coef += re.findall(r"p = __builtin_fma\(p, f, ([-0-9.e]+)\);", body)
    assert len(coef) == 9 and float(coef[-1]) == 1.0
    f = np.linspace(-0.5, 0.5, 200001).astype(np.longdouble)
    p = np.full_like(f, float(coef[0]))
    for c in coef[1:]:
        p = p * f + np.longdouble(float(c))
    worst = float(np.abs((p - np.exp2(f)) / np.exp2(f)).max())
    assert worst < 1.1e-12, worst
