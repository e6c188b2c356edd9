"""The capped scores' small-argument tanh (score_tile.cuh, kTanh1 .. kTanh7):
the header's constants are those the Remez exchange in
sparse_mask_transformer_gb300/csrc/tanh_poly.py derives, and their error
bound holds.  The kernels that use them are checked against 64-bit tanh in
tests/test_gpu_scored_attention.py."""
import os
import re
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mask_transformer_gb300", "csrc")


def _header_coefficients():
    src = open(os.path.join(CSRC, "score_tile.cuh")).read()
    found = dict(re.findall(r"kTanh([1357]) = (-?0x1\.[0-9a-f]+p-?\d+)f", src))
    return [float.fromhex(found[k]) for k in "1357"]


def test_header_constants_are_the_remez_coefficients():
    sys.path.insert(0, CSRC)
    try:
        import tanh_poly
    finally:
        sys.path.remove(CSRC)
    coef, level = tanh_poly.remez_tanh()
    # double precision throughout: the fp32 roundings of coefficients known to about 1e-12
    assert [np.float32(c) for c in coef] == [np.float32(c) for c in _header_coefficients()]
    err = tanh_poly.largest_error(coef)
    assert err <= 1.35e-7 and abs(err - level) < 0.1 * level  # levelled: the exchange converged


def test_polynomial_error_bound():
    c = _header_coefficients()
    y = np.linspace(-0.5, 0.5, 100001)
    t = y * y
    p = y * (c[0] + t * (c[1] + t * (c[2] + t * c[3])))
    assert np.max(np.abs(p - np.tanh(y))) <= 1.35e-7
    # a dropped term is far off
    assert np.max(np.abs(y * (c[0] + t * (c[1] + t * c[2])) - np.tanh(y))) > 1e-4
