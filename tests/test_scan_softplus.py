"""The polynomial of the selective scan's softplus (csrc/scan.hip): the written coefficients, rounded to f32 as the compiler takes
them, against log1p(e) = 2 atanh(s) over the whole of its interval, in 80 bits."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_softplus_polynomial():
    text = open(os.path.join(ROOT, "fp8_w8a8_linear_amd", "csrc", "scan.hip")).read()
    body = text[text.index("float softplus_poly(float x)"):]
    body = body[:body.index("\n}\n")]
    first = re.search(r"float p = fmaf\(q, 2 \* ([\d.]+)f, 2 \* ([\d.]+)f\);", body)
    rest = re.findall(r"p = fmaf\(q, p, (2 \* )?([\d.]+)f\);", body)
    assert first and len(rest) == 3
    c = [2 * np.float32(v) for v in first.groups()] + [(2 if two else 1) * np.float32(v) for two, v in rest]
    # s = e / (2 + e) of e = exp(-|x|) in (0, 1]
    s = np.linspace(0, np.longdouble(1) / 3, 400001, dtype=np.longdouble)[1:]
    p = np.zeros_like(s)
    for v in c:
        p = p * s * s + np.longdouble(float(v))
    error = np.abs(s * p / (2 * np.arctanh(s)) - 1).max()
    stated = float(re.search(r"within 2\^-([\d.]+) of the value", text).group(1))
    assert error <= 2.0 ** -stated, np.log2(float(error))
