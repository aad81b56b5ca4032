"""The degree-5 exp2 of attn_fwd_sinks, emulated step by step in float32 on the CPU (same coefficients,
same range reduction, same exponent insertion), against exact 2^x.

Tolerance: the polynomial's own relative error (7.5e-8 by the fit), the rounding of its six
coefficients (2^-24 each, weighted by |f|^i <= 2^-i: under 2 * 2^-24) and one rounding of 2^-24 in each
of the five Horner steps, halved from step to step by |f| <= 1/2 (under 2 * 2^-24 again), the last at the
scale of the result (which is >= 1/sqrt(2): times sqrt(2))."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "scaled_dot_product_16_b200", "csrc", "fwd_bf16_sm100.cu")
TOL = 7.5e-8 + 4 * 2.0 ** -24 * 2 ** 0.5


def _emulate(x):
    body = open(SRC).read()
    body = body[body.index("void exp2_poly5"):]
    a = [np.float32(float(re.search(rf"a{i} = ([0-9.e+-]+)f", body).group(1))) for i in range(6)]
    x = np.maximum(x.astype(np.float32), np.float32(-126.0))
    shift = np.float32(12582912.0)
    t = (x + shift).astype(np.float32)
    f = (x - (t - shift)).astype(np.float32)
    q = a[5]
    for c in a[4::-1]:  # an fma: one rounding
        q = (q.astype(np.float64) * f.astype(np.float64) + np.float64(c)).astype(np.float32)
    return (q.view(np.uint32) + (t.view(np.uint32) << np.uint32(23))).astype(np.uint32).view(np.float32)


def test_relative_error():
    x = np.concatenate([np.linspace(-126.0, 8.0, 400001), np.linspace(-1.0, 1.0, 200001), -np.arange(127.0)])
    x = x.astype(np.float32)
    err = np.abs(_emulate(x).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1)
    assert err.max() <= TOL, err.max()


def test_masked_scores_become_nothing():
    p = _emulate(np.array([-np.inf, -1e30, -127.0, -500.0], np.float32))
    assert np.all(p >= 0) and np.all(p < 2.0 ** -125)
