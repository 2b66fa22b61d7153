"""The decay of the gated recurrence (csrc/block_common.cuh: decay2) on the host:
its polynomial is the one that csrc/fit_polys.py fits, and its sequence, emulated
in fp32 with fused multiply-adds, gives a = 2^x and 1 - a^2 to full relative
accuracy for every x <= 0, decays next to 1 included."""
import os
import re

import numpy as np

from test_polys_host import CSRC, _fit, _fma32


def _constants():
    text = open(os.path.join(CSRC, "block_common.cuh")).read()
    found = dict(re.findall(r"constexpr float kDecayQ(\d+) = ([-+0-9.e]+)f;", text))
    assert sorted(found) == [str(k) for k in range(6)]
    return np.array([np.float32(found[str(k)]) for k in range(6)], dtype=np.float32)


def test_constants_are_the_fitted_ones():
    np.testing.assert_array_equal(_constants(), _fit().fit_exp2(5))


def _decay(x):
    """(a, w) of decay2, w without the 1e-36 that keeps its inverse root finite."""
    f = np.float32
    x = np.maximum(x, f(-126.0))
    t = (x + f(12582912.0)).astype(f)
    j = (t - f(12582912.0)).astype(f)
    s = _fma32(j, f(-1.0), x)
    c = _constants()
    q = np.full_like(s, c[5])
    for k in range(4, -1, -1):
        q = _fma32(q, s, c[k])
    p = (q * s).astype(f)
    S = (((t.view(np.int32).astype(np.int64) << 23) + 0x3f800000) & 0xffffffff).astype(np.uint32).view(f)
    a = _fma32(S, p, S)
    m = _fma32(S, p, (S - f(1.0)).astype(f))
    return a, _fma32(m, _fma32(m, f(-1.0), f(-2.0)), f(0.0))


def test_sequence_in_fp32():
    x = -np.concatenate([np.linspace(0.0, 126.0, 400001), np.logspace(-30, 2.1, 200001)]).astype(np.float32)
    a, w = _decay(x)
    ref = np.maximum(x, np.float32(-126.0)).astype(np.float64) * np.log(2.0)
    # the fit's 2.2e-8 and a rounding of 2^-24 in each of the last few operations, below 2^-21 together
    assert np.max(np.abs(a / np.exp(ref) - 1.0)) < 2.0 ** -21
    on = x < 0
    assert np.max(np.abs(w[on] / -np.expm1(2.0 * ref[on]) - 1.0)) < 2.0 ** -21
    assert (w[~on] == 0).all() and (a[~on] == 1).all()
    # a decay is never 0: a product of them is 0 only where a sequence starts
    assert a.min() == np.float32(2.0 ** -126)
    assert _decay(np.array([-np.inf, -1e30, -126.5, -126.0], dtype=np.float32))[0].tolist() == [2.0 ** -126] * 4
