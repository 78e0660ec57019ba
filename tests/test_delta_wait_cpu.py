"""Host side of the self-test of the delta rule's bounded waits: what it refuses before anything is enqueued."""
import ctypes

import mamba_ssd_chunked_fwd_gb300 as ssd


def test_refusals():
    lib = ssd.load_library()
    memory = ctypes.c_void_p(1 << 20)
    assert lib.ssd_selftest_chunk_wait(None, 388, 0, None) == 1
    assert lib.ssd_selftest_chunk_wait(memory, 387, 0, None) == 1
    assert lib.ssd_selftest_chunk_wait(memory, 389, 1, None) == 1
    assert "388" in lib.ssd_last_error_detail().decode()
