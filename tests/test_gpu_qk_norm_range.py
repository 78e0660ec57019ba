"""Gradients of the norm of queries and keys where rows are far from unit size: no power of the inverse root leaves fp32's
range before the result does.  Against the plain 64-bit form."""
import math

import pytest

from _selective_ref import close
from test_gpu_qk_norm import BF16, F32, bwd, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("s", [1e-15, 1e16])
@pytest.mark.parametrize("how", [dict(), dict(norm="l2", interleaved=True)])
@pytest.mark.parametrize("shape", [(2, 9, 4, 2, 64, 32), (1, 17, 5, 5, 128, 64), (1, 6, 2, 2, 100, 12), (1, 3, 2, 1, 255, 127)])
def test_gradients_of_small_and_large_rows(shape, how, s, t):
    k = make(*shape, t, far=5000)
    k["q"], k["k"] = (k["q"].float() * s).to(t), (k["k"].float() * s).to(t)
    got, want = bwd(k, t, dict(how, eps=0.0))
    for n in got:
        if n in ("dq", "dk"):  # to about unit size by a power of two, so without another rounding: `close` takes 1e-30 for none
            by = 2.0 ** round(math.log2(s))
            got[n], want[n] = got[n] * by, want[n] * by
        close(got[n], want[n], n)
