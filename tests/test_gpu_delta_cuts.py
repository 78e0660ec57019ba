"""The sizes that stand for rows cut into segments are cut: into how many follows from the workspace, which holds a state and a
transition of every segment."""
import ctypes

import pytest
import torch

from test_gpu_delta import ssd

pytestmark = pytest.mark.gpu


def segments(B, L, H, G, N, P):
    def size(rows):
        a = ssd().SsdDeltaArgs()
        a.B, a.L, a.H, a.G, a.N, a.P = rows, L, H, G, N, P
        a.dtype, a.g_dtype, a.beta_dtype, a.scale = 2, 0, 2, 1.0
        n = ctypes.c_size_t(0)
        assert ssd().load_library().ssd_delta_rule_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    many = 2 * torch.cuda.get_device_properties(0).multi_processor_count  # rows that fill the GPU twice are walked whole
    rest = size(B) - size(many) * B // many
    each, trans = B * H * P * N * 4, B * H * N * N * 4
    # n states and n - 1 transitions, each part to 256 bytes
    n = (rest + trans) // (each + trans)
    assert rest == 0 or abs(rest - n * each - (n - 1) * trans) < 1024
    return n if rest else 1


# the sizes of test_gpu_delta_cut.py: three segments or more, so that a transition and the fold are reached
@pytest.mark.parametrize("shape", [(2, 1300, 2, 1, 128, 128), (1, 2111, 1, 1, 64, 64), (3, 1100, 1, 1, 96, 200), (1, 1500, 3, 3, 24, 136),
                                   (1, 1500, 1, 1, 128, 128), (3, 1300, 1, 1, 128, 128), (1, 2000, 1, 1, 128, 64), (1, 1300, 2, 1, 128, 128)])
def test_rows_are_cut(shape):
    assert segments(*shape) >= 3, segments(*shape)


def test_full_grids_are_not():
    assert segments(4, 4096, 64, 16, 128, 128) == 1
