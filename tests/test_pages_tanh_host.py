"""The polynomial that stands for tanh near 0 in capped scores: its error, from
the coefficients in the source, against the bound that stands beside them."""

import os
import re

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))


def test_error_of_the_polynomial():
    with open(os.path.join(HERE, "..", "shared_quantized_kv_gb300", "csrc", "pages.cuh")) as f:
        text = f.read()
    q = [float(np.float32(x)) for x in re.search(r"kTanh\[5\] = \{([^}]*)\}", text).group(1).replace("f", "").split(",")]
    upto, bound = (float(x) for x in re.search(r"\|z\| <= ([0-9.]+) within ([0-9.e-]+)\s+relative", text).groups())
    assert upto == 0.7 and len(q) == 5
    z = np.concatenate([np.linspace(1e-3, upto, 1 << 20), np.geomspace(1e-8, 1e-3, 1 << 12)])
    u = z * z
    p = z * (1 + u * (q[0] + u * (q[1] + u * (q[2] + u * (q[3] + u * q[4])))))
    worst = np.max(np.abs(p / np.tanh(z) - 1))
    assert bound / 2 < worst <= bound, worst
