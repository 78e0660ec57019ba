"""Gates that empty the state, before and after others that make it grow: what was emptied does not come back."""
import math

import pytest
import torch

from _selective_ref import close
from test_gpu_delta import BF16, F16, F32, cuda, gpu, gpu_bwd, grads, make, plain, plain_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("empty", [-math.inf, -1000.0, -150.0])
@pytest.mark.parametrize("growth", [40.0, 80.0])
def test_growth_after_emptying(t, empty, growth):
    """Ten tokens that write nothing and grow the (empty) state by e^growth, ten more that shrink it again: sums of later gates
    up to 88, where exp leaves 32 bits."""
    if t == F16:
        growth = 6.0  # products q . k and u, as many times larger, stay below 65504
    k = make(1, 150, 2, 2, 128, 128, t, b32=True)
    k["g"] = torch.full_like(k["g"], -0.05)
    k["g"][:, 20], k["g"][:, 21:31], k["g"][:, 31:41] = empty, growth / 10, -growth / 10
    k["beta"][:, 20:41] = 0
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")
    dy, df = grads(k)
    if empty > -math.inf:  # differentiating the plain form multiplies infinity and zero there
        got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
        for n in got:
            close(got[n], want[n], n)


@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("order", ["after", "before"])
def test_growth_beyond_all_numbers(t, order):
    """Gates that sum to +210 beside one that empties the state: in a chunk a factor of e^210 is infinite, and some of the results
    are not finite; those that are, are right."""
    k = make(1, 150, 2, 2, 128, 128, t, b32=True)
    k["g"] = torch.full_like(k["g"], -0.05)
    k["g"][:, 20 if order == "after" else 31] = -1000.0
    k["g"][:, 21:31] = 21.0
    k["beta"][:, 20:32] = 0
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    dy, df = grads(k)
    got, want = gpu_bwd(cuda(k), dy.cuda(), df.cuda()), plain_bwd(k, dy, df)
    for n, a, b in [("y", y, ry), ("final", fin, rfin)] + [(n, got[n], want[n]) for n in got]:
        a = a.double().cpu()
        assert not torch.isfinite(a[b.abs() > 4e38]).any(), n
        on = torch.isfinite(a) & (b.abs() < 1e30)
        half = {F32: 0.0, F16: 2.0 ** -11, BF16: 2.0 ** -8}[(y if n == "y" else fin if n == "final" else got[n]).dtype]
        assert not on.any() or ((a - b).abs() <= half * b.abs() + 1e-4 * b[on].abs().max())[on].all(), n
