"""Arguments of the block norm that would have no effect are refused, on the host."""
import pytest
import torch

import mamba_ssd_chunked_fwd_gb300 as ssd


def test_type_beside_a_block():
    """n has o's type; another one asked for is an error, not ignored."""
    o, r, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, 8), torch.ones(8)
    with pytest.raises(ValueError, match="dtype"):
        ssd.block_norm(o, r, w, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):  # o's own type: goes on to the next check
        ssd.block_norm(o, r, w, dtype=torch.bfloat16)


def test_stream_output_without_a_block():
    """Without o nothing is written to r_out, so it cannot be given."""
    r, w = torch.zeros(2, 8), torch.ones(8)
    with pytest.raises(ValueError, match="r_out"):
        ssd.block_norm(None, r, w, r_out=torch.zeros(2, 8))
