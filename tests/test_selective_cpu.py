"""Refusals of the selective scan, its convolution and the block norm, without
a GPU: every case fails the host's checks before anything is enqueued.  And the
plain 64-bit forms against closed forms."""
import ctypes
import os
import subprocess

import pytest
import torch

import _selective_ref as ref
import mamba_ssd_chunked_fwd_gb300 as ssd

FAKE = 1 << 20  # never dereferenced
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INF, NAN = float("inf"), float("nan")


def scan_args(**over):
    a = ssd.SsdScanArgs()
    a.B, a.L, a.D, a.N, a.G = 2, 64, 32, 16, 2
    for n in ("x", "dt", "A", "Bm", "Cm", "y"):
        setattr(a, n, FAKE)
    a.dt_max = INF
    for k, v in over.items():
        setattr(a, k, v)
    return a


def call(name, a):
    lib = ssd.load_library()
    st = getattr(lib, name)(ctypes.byref(a), None)
    assert st == 0 or lib.ssd_last_error_detail()
    return st


SCAN_BAD = [("B", 0, 1), ("L", -1, 1), ("D", 0, 1), ("N", 0, 1), ("G", 3, 1), ("N", 129, 2), ("B", 70000, 2), ("L", 1 << 31, 2),
            ("x_dtype", 9, 1), ("dt_dtype", 9, 1), ("dt_dtype", 2, 2), ("x", None, 1), ("dt", None, 1), ("A", None, 1),
            ("Bm", None, 1), ("Cm", None, 1), ("dt_min", NAN, 1), ("dt_max", -1.0, 1), ("x_stride", (-1, 32), 1)]


def put(a, field, value):
    if isinstance(value, tuple):
        getattr(a, field)[:] = value
    else:
        setattr(a, field, value)
    return a


@pytest.mark.parametrize("field,value,code", SCAN_BAD + [("y", None, 1)])
def test_scan_refuses(field, value, code):
    assert call("ssd_selective_scan", put(scan_args(), field, value)) == code


@pytest.mark.parametrize("field,value,code", SCAN_BAD)
def test_scan_bwd_refuses(field, value, code):
    b = ssd.SsdScanBwdArgs()
    b.fwd = put(scan_args(), field, value)
    for n in ("dy", "dx", "ddt", "dA", "dB", "dC"):
        setattr(b, n, FAKE)
    assert call("ssd_selective_scan_bwd", b) == code


def test_scan_bwd_needs_its_outputs():
    def bwd(**over):
        b = ssd.SsdScanBwdArgs()
        b.fwd = scan_args()
        for n in ("dy", "dx", "ddt", "dA", "dB", "dC"):
            setattr(b, n, FAKE)
        for k, v in over.items():
            setattr(b.fwd if k in ("Dskip", "z", "dt_bias") else b, k, v)
        return b
    for n in ("dy", "dx", "ddt", "dA", "dB", "dC"):
        assert call("ssd_selective_scan_bwd", bwd(**{n: None})) == 1
    for n in ("Dskip", "z", "dt_bias"):
        assert call("ssd_selective_scan_bwd", bwd(**{n: FAKE})) == 1
    assert call("ssd_selective_scan_bwd", bwd()) == 3  # no workspace
    b = bwd()
    b.workspace, b.workspace_bytes = 4096 + 8, 1 << 40
    assert call("ssd_selective_scan_bwd", b) == 3  # not aligned


def test_workspace_queries():
    lib, out = ssd.load_library(), ctypes.c_size_t(7)
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(scan_args()), ctypes.byref(out)) == 0
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(scan_args(N=200)), ctypes.byref(out)) == 2
    assert lib.ssd_selective_scan_workspace_size(None, ctypes.byref(out)) == 1
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(scan_args()), None) == 1
    b = ssd.SsdScanBwdArgs()
    b.fwd = scan_args()
    assert lib.ssd_selective_scan_bwd_workspace_size(ctypes.byref(b), ctypes.byref(out)) == 0
    assert out.value >= 2 * 8 * 32 * 16 * 4  # the state before every eighth token


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, 1), ("D", -2, 1), ("G", 3, 1), ("N", 129, 2), ("nslots", 1, 1), ("nslots", 0, 1), ("x_dtype", 4, 1), ("dt_dtype", 1, 2),
    ("state", None, 1), ("state_out", None, 1), ("y", None, 1), ("Cm", None, 1), ("x_row", -4, 1), ("dt_min", 2.0, 1), ("B", 65536, 2)])
def test_scan_step_refuses(field, value, code):
    a = ssd.SsdScanStepArgs()
    a.B, a.D, a.N, a.G, a.nslots = 2, 32, 16, 2, 1 << 20
    for n in ("x", "dt", "A", "Bm", "Cm", "state", "state_out", "y"):
        setattr(a, n, FAKE)
    a.dt_max = 1.0
    setattr(a, field, value)
    assert call("ssd_selective_scan_step", a) == code


def conv_args(**over):
    a = ssd.SsdConvArgs()
    a.B, a.L, a.C, a.W = 2, 64, 32, 4
    a.x = a.w = a.y = FAKE
    for k, v in over.items():
        put(a, k, v)
    return a


@pytest.mark.parametrize("field,value,code", [("B", 0, 1), ("L", 0, 1), ("C", -1, 1), ("W", 0, 1), ("W", 9, 2), ("L", 9_000_000, 2),
                                              ("dtype", 3, 1), ("x", None, 1), ("w", None, 1), ("y", None, 1), ("x_stride", (3, -1), 1)])
def test_conv_refuses(field, value, code):
    assert call("ssd_causal_conv_carry", conv_args(**{field: value})) == code
    b = ssd.SsdConvBwdArgs()
    b.fwd = conv_args(**{field: value})
    b.dy = b.dx = b.dw = FAKE
    assert call("ssd_causal_conv_bwd", b) == (code if field != "y" else 3)


def test_conv_bwd_needs_its_outputs():
    b = ssd.SsdConvBwdArgs()
    b.fwd = conv_args(bias=FAKE)
    b.dy = b.dx = b.dw = FAKE
    assert call("ssd_causal_conv_bwd", b) == 1  # dbias
    b.dbias = FAKE
    assert call("ssd_causal_conv_bwd", b) == 3  # workspace
    b.dw = None
    assert call("ssd_causal_conv_bwd", b) == 1


@pytest.mark.parametrize("field,value,code", [("B", 0, 1), ("C", 0, 1), ("W", 9, 2), ("nslots", 1, 1), ("dtype", 7, 1), ("x", None, 1),
                                              ("state", None, 1), ("state_out", None, 1), ("x_row", -1, 1), ("B", 65536, 2)])
def test_conv_step_refuses(field, value, code):
    a = ssd.SsdConvStepArgs()
    a.B, a.C, a.W, a.nslots = 2, 32, 4, 1 << 20
    for n in ("x", "w", "state", "state_out", "y"):
        setattr(a, n, FAKE)
    setattr(a, field, value)
    assert call("ssd_causal_conv_step", a) == code


def norm_args(**over):
    a = ssd.SsdBlockNormArgs()
    a.rows, a.D, a.rows_per_gate, a.eps = 6, 32, 3, 1e-5
    for n in ("o", "r", "w_pre", "n", "r_out"):
        setattr(a, n, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(rows=0), 1), (dict(D=0), 1), (dict(D=16385), 2), (dict(rows=1 << 31), 2), (dict(dtype=5), 1), (dict(stream_dtype=5), 1),
    (dict(dtype=2, stream_dtype=1), 2), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(w_pre=None), 1),
    (dict(gate=FAKE, rows_per_gate=4), 1), (dict(gate=FAKE, rows_per_gate=0), 1), (dict(o=None, gate=FAKE), 1),
    (dict(o=None, w_post=FAKE), 1), (dict(o=None, scale=FAKE), 1)])
def test_norm_refuses(over, code):
    assert call("ssd_block_norm", norm_args(**over)) == code
    b = ssd.SsdBlockNormBwdArgs()
    b.fwd = norm_args(**over)
    b.dn = b.dr = b.dw_pre = b.d_o = b.dgate = b.dw_post = b.dscale = FAKE
    assert call("ssd_block_norm_bwd", b) == code


@pytest.mark.parametrize("over", [dict(r=None), dict(n=None), dict(r_out=None)])
def test_norm_needs_its_tensors(over):
    assert call("ssd_block_norm", norm_args(**over)) == 1


@pytest.mark.parametrize("given,missing", [(None, "dn"), (None, "dr"), (None, "dw_pre"), (None, "d_o"), ("gate", "dgate"),
                                           ("w_post", "dw_post"), ("scale", "dscale"), (None, "workspace")])
def test_norm_bwd_needs_its_outputs(given, missing):
    b = ssd.SsdBlockNormBwdArgs()
    b.fwd = norm_args(**({given: FAKE} if given else {}))
    for n in ("dn", "dr", "dw_pre", "d_o", "dgate", "dw_post", "dscale"):
        setattr(b, n, FAKE)
    if missing != "workspace":
        setattr(b, missing, None)
    assert call("ssd_block_norm_bwd", b) == (3 if missing == "workspace" else 1)


def test_structures_match_the_header(tmp_path):
    """Sizes and last offsets of the binding's structures, from a C compiler."""
    pairs = [("ssd_scan_args", ssd.SsdScanArgs), ("ssd_scan_bwd_args", ssd.SsdScanBwdArgs), ("ssd_scan_step_args", ssd.SsdScanStepArgs),
             ("ssd_conv_args", ssd.SsdConvArgs), ("ssd_conv_bwd_args", ssd.SsdConvBwdArgs), ("ssd_conv_step_args", ssd.SsdConvStepArgs),
             ("ssd_block_norm_args", ssd.SsdBlockNormArgs), ("ssd_block_norm_bwd_args", ssd.SsdBlockNormBwdArgs)]
    lines = []
    for name, cls in pairs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "ssd.h"\nint main(void) {' + "".join(lines) + "return 0;}")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in pairs:
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, B, A = torch.zeros(1, 4, 8), torch.zeros(1, 4, 1, 16), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.causal_conv1d_carry(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.block_norm(x, x, torch.zeros(8))
    # the marshalling itself, which does not look at the device
    with pytest.raises(ValueError, match="dimensions"):
        ssd.make_scan_args(x[0], x, A, B, B)
    with pytest.raises(ValueError, match="B: shape|C: shape"):
        ssd.make_scan_args(x, x, A, B, B[:, :3])
    with pytest.raises(ValueError, match="dt"):
        ssd.make_scan_args(x, x.half(), A, B, B)
    with pytest.raises(ValueError, match="unsupported dtype"):
        ssd.make_scan_args(x.double(), x.double(), A, B, B)
    with pytest.raises(ValueError, match="contiguous"):
        ssd.make_scan_args(x, x.transpose(1, 2).contiguous().transpose(1, 2), A, B, B)
    with pytest.raises(ValueError, match="broadcast"):
        ssd.make_scan_args(x, x[:, :1].expand(1, 4, 8), A, B, B)
    with pytest.raises(ValueError, match="lengths"):
        ssd.make_scan_args(x, x, A, B, B, lengths=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="initial_state"):
        ssd.make_conv_args(x, torch.zeros(8, 4), initial_state=torch.zeros(1, 4, 8))
    a = ssd.make_scan_args(torch.zeros(2, 4, 20)[..., 3:11], torch.zeros(2, 4, 8), A, torch.zeros(2, 4, 1, 16), torch.zeros(2, 4, 1, 16))
    assert list(a.x_stride) == [80, 20] and list(a.dt_stride) == [0, 0]


def test_plain_scan_against_closed_forms():
    """No decay: a running sum; a constant step: a geometric sum; the quadratic form; two halves."""
    g = torch.Generator().manual_seed(0)
    x, B, C = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((1, 9, 2), (1, 9, 1, 3), (1, 9, 1, 3)))
    d = torch.rand((1, 9, 2), generator=g, dtype=torch.float64)
    A = torch.zeros((2, 3), dtype=torch.float64)
    y, h = ref.scan(x, d, A, B, C, softplus=False)
    run = torch.cumsum((d * x)[..., None] * B, 1)
    torch.testing.assert_close(y, (run * C).sum(-1))
    torch.testing.assert_close(h, run[:, -1])
    A = -torch.rand((2, 3), generator=g, dtype=torch.float64)
    y, h = ref.scan(x, d, A, B, C, softplus=False)
    for t in range(9):
        want = 0
        for s in range(t + 1):
            want = want + (torch.exp(A * d[0, s + 1:t + 1].sum(0)[:, None]) * (d * x)[0, s][:, None] * B[0, s] * C[0, t]).sum(-1)
        torch.testing.assert_close(y[0, t], want)
    _, mid = ref.scan(x[:, :4], d[:, :4], A, B[:, :4], C[:, :4], softplus=False)
    y2, end = ref.scan(x[:, 4:], d[:, 4:], A, B[:, 4:], C[:, 4:], h0=mid, softplus=False)
    torch.testing.assert_close(y2, y[:, 4:])
    torch.testing.assert_close(end, h)


def test_plain_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    k = {n: torch.randn(s, generator=g, dtype=torch.float64) for n, s in
         dict(x=(1, 5, 2), dt=(1, 5, 2), B=(1, 5, 1, 3), C=(1, 5, 1, 3), z=(1, 5, 2), D=(2,), dt_bias=(2,), h0=(1, 2, 3)).items()}
    k["A"] = -torch.rand((2, 3), generator=g, dtype=torch.float64)
    w = (torch.randn((1, 5, 2), generator=g, dtype=torch.float64), torch.randn((1, 2, 3), generator=g, dtype=torch.float64))

    def f(**a):
        return ref.scan(**a)
    grads = ref.gradients(f, k, w)
    for n in k:
        v = torch.randn(k[n].shape, generator=g, dtype=torch.float64)

        def value(s):
            return sum((o * u).sum() for o, u in zip(f(**{**k, n: k[n] + s * 1e-6 * v}), w))
        slope = (value(1) - value(-1)) / 2e-6
        torch.testing.assert_close((grads[n] * v).sum(), slope, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("x,x_stride,y,code", [(FAKE, (0, 0), FAKE, 1), (FAKE, (0, 0), FAKE + 2 * 64 * 32 * 4 - 4, 1),
                                               (FAKE, (128 * 64, 64), FAKE + (128 * 64 + 63 * 64 + 32) * 4 - 4, 1),
                                               (FAKE + 2 * 64 * 32 * 4 - 4, (0, 0), FAKE, 1)])
def test_conv_refuses_its_own_input_as_output(x, x_stride, y, code):
    assert call("ssd_causal_conv_carry", conv_args(x=x, x_stride=x_stride, y=y)) == code


@pytest.mark.parametrize("off", [0, 4, -4])
def test_carried_states_must_not_overlap(off):
    assert call("ssd_selective_scan", scan_args(initial_state=FAKE, final_state=FAKE + off)) == 1
    assert call("ssd_causal_conv_carry", conv_args(y=2 * FAKE, initial_state=FAKE, final_state=FAKE + off)) == 1
