"""The gated delta rule where a row is cut into segments walked side by side: few heads, many chunks.
Against the plain 64-bit form, in both 16-bit types, with ragged rows and states carried in."""
import pytest
import torch

from _selective_ref import close
from test_gpu_delta import BF16, F16, cuda, gpu, make, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("opts", [dict(), dict(h0=False), dict(ragged=True)])
@pytest.mark.parametrize("shape", [(2, 1300, 2, 1, 128, 128), (1, 2111, 1, 1, 64, 64), (3, 1100, 1, 1, 96, 200), (1, 1500, 3, 3, 24, 136)])
def test_cut_rows(shape, t, opts):
    k = make(*shape, t, **opts)
    if opts.get("ragged") and shape[0] > 2:
        k["lengths"][2] = 257  # ends inside an early segment: the later ones have nothing
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")


@pytest.mark.parametrize("t", [F16, BF16])
def test_cut_rows_of_slow_decay_and_alike_keys(t):
    """What a segment's transition keeps of a state, over ten segments."""
    k = make(1, 1500, 1, 1, 128, 128, t)
    k["g"] = torch.full_like(k["g"], -1e-3)
    k["beta"] = k["beta"] * 0.1
    y, fin = gpu(cuda(k))
    ry, rfin = plain(k)
    close(y, ry, "y")
    close(fin, rfin, "final state")


def test_padding_does_not_leak_into_segments():
    k = make(3, 1300, 1, 1, 128, 128, BF16, ragged=True)
    k["lengths"] = torch.tensor([1300, 0, 700], dtype=torch.int32)
    want = gpu(cuda(k))
    for n in ("q", "k", "v", "g", "beta"):
        for b, e in enumerate(k["lengths"].tolist()):
            k[n][b, e:] = float("nan")
    for a, b in zip(gpu(cuda(k)), want):
        assert torch.equal(a, b)
