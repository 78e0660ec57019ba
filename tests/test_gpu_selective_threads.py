"""The C entries called from several host threads at once."""
import ctypes
import threading

import pytest
import torch

import mamba_ssd_chunked_fwd_gb300 as ssd

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def together(calls, times):
    """Each (entry, arguments) in a thread of its own, over and over; the statuses that are not 0.
    ctypes drops the interpreter's lock within a call, so the entries run side by side."""
    lib = ssd.load_library()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    bad = [[] for _ in calls]
    start = threading.Barrier(len(calls))

    def run(i, name, args):
        fn, ref = getattr(lib, name), ctypes.byref(args)
        start.wait()
        for _ in range(times):
            st = fn(ref, stream)
            if st:
                bad[i].append((st, lib.ssd_last_error_detail()))

    threads = [threading.Thread(target=run, args=(i, *c)) for i, c in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_norms_of_two_widths():
    """One instantiation, two needs of shared memory."""
    calls, keep = [], []
    for D in (4096, 8192, 4096, 8192):
        o, r = torch.randn(2, D, device="cuda").to(BF16), torch.randn(2, D, device="cuda").to(BF16)
        w, n, out = torch.ones(D, device="cuda"), torch.empty(2, D, device="cuda", dtype=BF16), torch.empty(2, D, device="cuda", dtype=BF16)
        a = ssd.SsdBlockNormArgs()
        a.rows, a.D, a.rows_per_gate, a.eps, a.dtype, a.stream_dtype = 2, D, 1, 1e-5, 2, 2
        a.o, a.r, a.w_post, a.w_pre, a.n, a.r_out = (t.data_ptr() for t in (o, r, w, w, n, out))
        keep.append((o, r, w, n, out))
        calls.append(("ssd_block_norm", a))
    assert together(calls, 4000) == [[]] * len(calls)


def test_norm_gradients_of_two_widths():
    calls, keep = [], []
    for D in (4096, 8192, 4096, 8192):
        t = [torch.randn(2, D, device="cuda").to(BF16) for _ in range(6)]
        w = [torch.ones(D, device="cuda") for _ in range(4)]
        b = ssd.SsdBlockNormBwdArgs()
        a = b.fwd
        a.rows, a.D, a.rows_per_gate, a.eps, a.dtype, a.stream_dtype = 2, D, 1, 1e-5, 2, 2
        a.o, a.r_out, a.w_post, a.w_pre = t[0].data_ptr(), t[1].data_ptr(), w[0].data_ptr(), w[1].data_ptr()
        b.dn, b.d_o, b.dr, b.dw_post, b.dw_pre = t[2].data_ptr(), t[3].data_ptr(), t[4].data_ptr(), w[2].data_ptr(), w[3].data_ptr()
        size = ctypes.c_size_t()
        assert ssd.load_library().ssd_block_norm_bwd_workspace_size(ctypes.byref(b), ctypes.byref(size)) == 0
        ws = torch.empty(size.value, dtype=torch.uint8, device="cuda")
        b.workspace, b.workspace_bytes = ws.data_ptr(), size.value
        keep.append((t, w, ws))
        calls.append(("ssd_block_norm_bwd", b))
    assert together(calls, 4000) == [[]] * len(calls)


@pytest.mark.parametrize("backward", [False, True])
def test_scans_of_two_types_of_steps(backward):
    """Steps in fp32 beside 16-bit tensors need more shared memory than steps in 16 bits."""
    calls, keep = [], []
    B, L, D, N = 1, 8, 64, 16
    for dt_type in (BF16, torch.float32, BF16, torch.float32):
        x, B_, C = (torch.randn(s, device="cuda").to(BF16) for s in ((B, L, D), (B, L, 1, N), (B, L, 1, N)))
        dt, A = torch.rand(B, L, D, device="cuda").to(dt_type), -torch.rand(D, N, device="cuda")
        y = torch.empty_like(x)
        a = ssd.make_scan_args(x, dt, A, B_, C, y=y)
        name, size = "ssd_selective_scan", ctypes.c_size_t()
        if backward:
            outs = [torch.empty_like(t) for t in (x, dt, A, B_, C)]
            b = ssd.SsdScanBwdArgs()
            b.fwd, b.dy = a, x.data_ptr()
            b.dx, b.ddt, b.dA, b.dB, b.dC = (t.data_ptr() for t in outs)
            keep.append(outs)
            a, name = b, "ssd_selective_scan_bwd"
        assert getattr(ssd.load_library(), name + "_workspace_size")(ctypes.byref(a), ctypes.byref(size)) == 0
        ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), size.value
        keep.append((x, dt, A, B_, C, y, ws))
        calls.append((name, a))
    assert together(calls, 4000) == [[]] * len(calls)
