"""Gradients of many chunks that a CTA takes one after another, in which some of a warp's lanes have nothing to store (short
rows, narrow heads): run after run the same, and right."""
import pytest
import torch

from _selective_ref import close
from test_gpu_delta import BF16, F16, cuda, gpu, gpu_bwd, grads, make, plain, plain_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("shape", [(5, 3, 128, 2, 8, 8), (4, 3, 128, 128, 64, 128), (6, 67, 128, 64, 40, 72), (6, 5, 100, 25, 120, 16)])
def test_many_units(shape, t):
    k = make(*shape, t)
    dy, df = grads(k)
    c, dyc, dfc = cuda(k), dy.cuda(), df.cuda()
    first, firsty = gpu_bwd(c, dyc, dfc), gpu(c)
    want = plain_bwd(k, dy, df)
    for n in first:
        close(first[n], want[n], n)
    for got, w in zip(firsty, plain(k)):
        close(got, w)
    for _ in range(10):
        again = gpu_bwd(c, dyc, dfc)
        assert all(torch.equal(again[n], first[n]) for n in first)
        assert all(torch.equal(a, b) for a, b in zip(gpu(c), firsty))
