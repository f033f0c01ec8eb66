"""The polynomial of the exact GELU's kernel code, read from its source, against
exp(a^2) erfc(a) in fp64 (no GPU)."""
import math
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_decode_amd", "csrc",
                      "ffn_kernels.h")


def scaled_erfc(a):
    """exp(a^2) erfc(a): directly while that is accurate, then its asymptotic series."""
    if a < 6.0:
        return math.exp(a * a) * math.erfc(a)
    term = total = 1.0
    for n in range(1, 20):
        term *= -(2 * n - 1) / (2 * a * a)
        total += term
    return total / (a * math.sqrt(math.pi))


def fit_error(low, high):
    with open(SOURCE) as f:
        text = f.read()
    body = text[text.index("float normal_cdf(float z)"):]
    c = [float(np.float32(v)) for v in re.search(r"c\[9\] = \{([^}]*)\}", body).group(1).replace("f", "").split(",")]
    assert len(c) == 9
    worst = 0.0
    for a in np.linspace(low, high, 4001):
        t = 1.0 / (1.0 + 0.4 * a)
        p = 0.0
        for v in reversed(c):
            p = p * t + v
        worst = max(worst, abs(p * t / scaled_erfc(a) - 1.0))
    return worst


def test_fit_is_as_good_as_its_comment_says():
    assert fit_error(0.0, 4.0) < 3.2e-8
    assert fit_error(4.0, 6.0) < 1e-7
    assert fit_error(6.0, 9.5) < 1.2e-5
