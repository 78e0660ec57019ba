"""NaN among the live inputs of the selective scan: it reaches what the formula
says it reaches, and nothing else."""
import math

import pytest
import torch

from test_gpu_selective import BF16, F16, F32, cuda, gpu_scan, gpu_scan_bwd, grads_like, make, ref_scan, ref_scan_bwd, ssd

pytestmark = pytest.mark.gpu

LIMITS = [(0.0, math.inf), (0.004, 0.05)]


def same_nans(got, want, what):
    assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want).cpu()), what


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("t", [F32, F16, BF16])
@pytest.mark.parametrize("L", [20, 400])  # a walk in one piece; a cut one
def test_scan_of_nan_steps(L, t, softplus, limit):
    k = make(2, L, 24, 16, 1, t)
    if not softplus:
        k["dt"], k["dt_bias"] = k["dt"].abs() * 0.3, None
    k["dt"][1, 7, 5] = math.nan
    y, fin = gpu_scan(cuda(k), softplus, limit)
    ry, rfin = ref_scan(k, softplus, limit)
    same_nans(y, ry, "y")
    same_nans(fin, rfin, "final state")
    assert torch.isnan(y[1, 7:, 5]).all() and torch.isnan(fin[1, 5]).all()


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("L", [20, 400])
def test_gradients_of_nan_steps(L, t, limit):
    k = make(2, L, 24, 16, 1, t)
    k["dt"][1, 7, 5] = math.nan
    dy, df = grads_like(k)
    got = gpu_scan_bwd(cuda(k), dy.cuda(), df.cuda(), True, limit)
    want = ref_scan_bwd(k, dy, df, True, limit)
    for n in ("dx", "dB", "dC", "dA", "dz", "dh0"):
        same_nans(got[n], want[n], n)


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("B", [3, 130])  # one sequence per lane, and four
def test_step_of_nan_steps(B, limit):
    D = 40 if B == 3 else 2048
    k = cuda(make(B, 1, D, 16, 1, BF16))
    k["dt"][1, 0, 5] = math.nan
    h = k["h0"].clone()
    y = ssd().selective_scan_step(k["x"][:, 0], k["dt"][:, 0], k["A"], k["B"][:, 0], k["C"][:, 0], h, True, D=k["D"],
                                  z=k["z"][:, 0], dt_bias=k["dt_bias"], dt_limit=limit)
    want = torch.zeros((B, D), dtype=torch.bool)
    want[1, 5] = True
    assert torch.equal(torch.isnan(y).cpu(), want)
    assert torch.equal(torch.isnan(h).all(-1).cpu(), want) and torch.isnan(h).sum() == 16
