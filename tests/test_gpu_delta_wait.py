"""The delta rule's waits in chunks give up instead of hanging, and what follows from a chunk whose preparation has given up is
NaN throughout.  No GPU fault is involved: the wait that runs out is on an mbarrier that nothing arrives on, for two
tries of a millisecond."""
import pytest
import torch

from test_gpu_delta import BF16, cuda, gpu, make, plain, ssd
from _selective_ref import close

pytestmark = pytest.mark.gpu


def test_gates_of_a_preparation_that_gives_up():
    out = torch.zeros(388, device="cuda")
    ssd().ssd_selftest_chunk_wait(out)
    torch.cuda.synchronize()
    assert torch.isnan(out).all(), torch.isnan(out).sum()
    ssd().ssd_selftest_chunk_wait(out, arrive=True)
    assert (out == 1).all()
    k = make(1, 70, 2, 1, 128, 128, BF16)  # the context is intact
    close(gpu(cuda(k))[0], plain(k)[0], "y")


def test_refusals():
    with pytest.raises(ssd().SsdError):
        ssd().ssd_selftest_chunk_wait(torch.zeros(387, device="cuda"))
    with pytest.raises(ValueError):
        ssd().ssd_selftest_chunk_wait(torch.zeros(388, device="cuda", dtype=torch.float64))
