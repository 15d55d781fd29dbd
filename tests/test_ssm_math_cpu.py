"""The logarithm's polynomial of the selective mixer's kernels (csrc/ssm.cuh),
its coefficients as the source has them, against its stated error bounds."""
from __future__ import annotations

import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_scans_gb300", "csrc",
                      "ssm.cuh")


def test_log1p_over_the_unit_interval():
    text = open(SOURCE).read()
    body = re.search(r"log1p_coef\(int i\)\s*\{.*?\{([^}]*)\}", text, re.S).group(1)
    coef = [np.float32(v.strip().rstrip("f")) for v in body.split(",")]
    assert len(coef) == 10
    stated = re.search(r"relative error ([\d.e-]+), with the evaluation's roundings ([\d.e-]+)\)", re.sub(r"\s*//\s*", " ", text))
    exact_bound, rounded_bound = (float(v) for v in stated.groups())
    e = np.concatenate([np.linspace(2.0 ** -24, 1, 400001), 2.0 ** np.linspace(-60, 0, 60001)]).astype(np.float32)
    true = np.log1p(e.astype(np.float64)) / e
    exact, rounded = np.zeros(e.shape), np.zeros(e.shape, np.float32)
    for c in reversed(coef):
        exact = exact * e + float(c)
        rounded = (rounded.astype(np.float64) * e + float(c)).astype(np.float32)   # a fused multiply-add
    rounded = rounded.astype(np.float64) * e
    worst = np.max(np.abs(exact / true - 1)), np.max(np.abs(rounded.astype(np.float32) / np.log1p(e.astype(np.float64)) - 1))
    assert worst[0] <= exact_bound and worst[1] <= rounded_bound, worst
