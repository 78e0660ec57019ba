"""Outputs laid over inputs that other threads still read: each of these calls is
refused on the host, so nothing is enqueued and no address is looked at."""
import ctypes

import pytest

import mamba_ssd_chunked_fwd_gb300 as ssd

INF = float("inf")
MB = 1 << 20


def place(a, names, **over):
    """Every tensor on its own megabytes, then what the case moves."""
    for i, n in enumerate(names):
        setattr(a, n, (16 + 4 * i) * MB)
    for k, v in over.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def call(name, a):
    lib = ssd.load_library()
    st = getattr(lib, name)(ctypes.byref(a), None)
    return st, lib.ssd_last_error_detail().decode()


def refused(name, a, who):
    st, detail = call(name, a)
    assert st == 1 and "overlap" in detail and who in detail, (st, detail)


SCAN = ("x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "initial_state", "lengths", "y", "final_state")
AT = {n: (16 + 4 * i) * MB for i, n in enumerate(SCAN)}
Y = 2 * 64 * 32 * 2  # bytes of y; so are x's, z's and dt's


def scan_args(**over):
    a = ssd.SsdScanArgs()
    a.B, a.L, a.D, a.N, a.G = 2, 64, 32, 16, 2
    a.x_dtype = a.dt_dtype = 2
    a.dt_max = INF
    a.workspace, a.workspace_bytes = 512 * MB, 64 * MB
    return place(a, SCAN, **over)


@pytest.mark.parametrize("name", ["Bm", "Cm", "A", "Dskip", "dt_bias", "initial_state", "lengths", "final_state"])
def test_scan_output_over_what_every_channel_reads(name):
    refused("ssd_selective_scan", scan_args(y=AT[name]), "y")
    refused("ssd_selective_scan", scan_args(y=AT[name] + 4 - Y), "y")  # its last bytes


@pytest.mark.parametrize("name", ["x", "dt", "z"])
def test_scan_output_beside_its_own_place(name):
    """y may be x, dt or z itself, but not shifted against it, nor over a slice of something wider."""
    for off in (2, -2, 64, 16 - Y, Y - 16):
        refused("ssd_selective_scan", scan_args(y=AT[name] + off), "y")
    stride = {"x": "x_stride", "dt": "dt_stride", "z": "z_stride"}[name]
    for s in ((64 * 48, 48), (0, 32), (64 * 32, 0)):  # wider rows; one sequence, or one token, for all
        refused("ssd_selective_scan", scan_args(y=AT[name], **{stride: s}), "y")


def test_scan_output_over_wider_steps():
    refused("ssd_selective_scan", scan_args(y=AT["dt"], dt_dtype=0), "y")


@pytest.mark.parametrize("name", ["x", "dt", "z", "Bm", "Cm", "A", "Dskip", "dt_bias", "initial_state", "lengths"])
def test_scan_final_state_over_inputs(name):
    refused("ssd_selective_scan", scan_args(final_state=AT[name]), "final_state")


def test_scan_reads_through_strides():
    """The far end of a slice of a wider tensor counts."""
    far = AT["Bm"] + (64 * 100 + 63 * 100 + 32) * 2 - 2
    refused("ssd_selective_scan", scan_args(y=far, b_stride=(6400, 100)), "y")


CONV = ("x", "w", "bias", "initial_state", "lengths", "y", "final_state")
CONV_AT = {n: (16 + 4 * i) * MB for i, n in enumerate(CONV)}


def conv_args(**over):
    a = ssd.SsdConvArgs()
    a.B, a.L, a.C, a.W, a.dtype = 2, 64, 32, 4, 2
    return place(a, CONV, **over)


@pytest.mark.parametrize("name", ["x", "w", "bias", "initial_state", "lengths", "final_state"])
def test_conv_output_over_what_others_read(name):
    refused("ssd_causal_conv_carry", conv_args(y=CONV_AT[name]), "y")
    refused("ssd_causal_conv_carry", conv_args(y=CONV_AT[name] + 4 - Y), "y")


@pytest.mark.parametrize("name", ["x", "w", "bias", "initial_state", "lengths"])
def test_conv_final_state_over_inputs(name):
    refused("ssd_causal_conv_carry", conv_args(final_state=CONV_AT[name]), "final_state")


STEP = ("x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "state", "state_out", "slots", "y")
STEP_AT = {n: (16 + 4 * i) * MB for i, n in enumerate(STEP)}
ROWS, POOL = 4 * 32 * 2, 6 * 32 * 16 * 4  # bytes of y and of the states


def step_args(**over):
    a = ssd.SsdScanStepArgs()
    a.B, a.D, a.N, a.G, a.nslots = 4, 32, 16, 2, 6
    a.x_dtype = a.dt_dtype = 2
    a.dt_max = INF
    return place(a, STEP, **over)


@pytest.mark.parametrize("name", ["A", "Bm", "Cm", "Dskip", "dt_bias", "state", "state_out", "slots"])
def test_step_output_over_what_others_read(name):
    refused("ssd_selective_scan_step", step_args(y=STEP_AT[name]), "y")
    refused("ssd_selective_scan_step", step_args(y=STEP_AT[name] + 4 - ROWS), "y")


@pytest.mark.parametrize("name", ["x", "dt", "z"])
def test_step_output_beside_its_own_place(name):
    for off in (2, 64, 4 - ROWS):
        refused("ssd_selective_scan_step", step_args(y=STEP_AT[name] + off), "y")
    row = {"x": "x_row", "dt": "dt_row", "z": "z_row"}[name]
    refused("ssd_selective_scan_step", step_args(y=STEP_AT[name], **{row: 40}), "y")
    if name == "dt":
        refused("ssd_selective_scan_step", step_args(y=STEP_AT[name], dt_dtype=0), "y")


@pytest.mark.parametrize("name", ["x", "dt", "z", "A", "Bm", "Cm", "Dskip", "dt_bias", "slots"])
def test_step_states_over_inputs(name):
    refused("ssd_selective_scan_step", step_args(state_out=STEP_AT[name]), "state_out")
    refused("ssd_selective_scan_step", step_args(state=STEP_AT[name], state_out=STEP_AT[name]), "state_out")


@pytest.mark.parametrize("off", [4, 32 * 16 * 4, -32 * 16 * 4, POOL - 4])
def test_step_states_beside_their_own_place(off):
    """state_out is state or lies apart: a shifted pool holds other sequences' states."""
    refused("ssd_selective_scan_step", step_args(state_out=STEP_AT["state"] + off), "state_out")


CSTEP = ("x", "w", "bias", "state", "state_out", "slots", "y")
CSTEP_AT = {n: (16 + 4 * i) * MB for i, n in enumerate(CSTEP)}


def conv_step_args(**over):
    a = ssd.SsdConvStepArgs()
    a.B, a.C, a.W, a.nslots, a.dtype = 4, 32, 4, 6, 2
    return place(a, CSTEP, **over)


@pytest.mark.parametrize("name", ["w", "bias", "state", "state_out", "slots"])
def test_conv_step_output_over_what_others_read(name):
    refused("ssd_causal_conv_step", conv_step_args(y=CSTEP_AT[name]), "y")


def test_conv_step_output_beside_its_own_place():
    for off in (2, 64, 4 - ROWS):
        refused("ssd_causal_conv_step", conv_step_args(y=CSTEP_AT["x"] + off), "y")
    refused("ssd_causal_conv_step", conv_step_args(y=CSTEP_AT["x"], x_row=40), "y")


@pytest.mark.parametrize("name", ["x", "w", "bias", "slots"])
def test_conv_step_states_over_inputs(name):
    refused("ssd_causal_conv_step", conv_step_args(state_out=CSTEP_AT[name]), "state_out")


@pytest.mark.parametrize("off", [2, 3 * 32 * 2, -3 * 32 * 2])
def test_conv_step_states_beside_their_own_place(off):
    refused("ssd_causal_conv_step", conv_step_args(state_out=CSTEP_AT["state"] + off), "state_out")


NORM = ("o", "r", "gate", "w_post", "w_pre", "scale", "n", "r_out")
NORM_AT = {n: (16 + 4 * i) * MB for i, n in enumerate(NORM)}
NROWS = 6 * 32 * 2


def norm_args(**over):
    a = ssd.SsdBlockNormArgs()
    a.rows, a.D, a.rows_per_gate, a.eps, a.dtype, a.stream_dtype = 6, 32, 1, 1e-5, 2, 2
    return place(a, NORM, **over)


@pytest.mark.parametrize("out", ["n", "r_out"])
@pytest.mark.parametrize("name", ["w_post", "w_pre", "scale"])
def test_norm_output_over_weights(out, name):
    refused("ssd_block_norm", norm_args(**{out: NORM_AT[name]}), out)


def test_norm_outputs_over_each_other():
    refused("ssd_block_norm", norm_args(n=NORM_AT["r_out"]), "n")
    refused("ssd_block_norm", norm_args(n=NORM_AT["r_out"] + NROWS - 2), "n")
    refused("ssd_block_norm", norm_args(n=NORM_AT["r"], r_out=NORM_AT["r"]), "n")


@pytest.mark.parametrize("out", ["n", "r_out"])
@pytest.mark.parametrize("name", ["o", "r", "gate"])
def test_norm_output_beside_its_own_place(out, name):
    """An output may be o, r or a gate per token itself, in its own type, but not shifted against it."""
    for off in (2, 32 * 2, 2 - NROWS):
        refused("ssd_block_norm", norm_args(**{out: NORM_AT[name] + off}), out)


def test_norm_output_over_another_type_or_a_shared_gate():
    refused("ssd_block_norm", norm_args(n=NORM_AT["r"], stream_dtype=0), "n")
    refused("ssd_block_norm", norm_args(r_out=NORM_AT["o"], stream_dtype=0), "r_out")
    refused("ssd_block_norm", norm_args(r_out=NORM_AT["gate"], stream_dtype=0), "r_out")
    refused("ssd_block_norm", norm_args(n=NORM_AT["gate"], rows_per_gate=3), "n")
    refused("ssd_block_norm", norm_args(r_out=NORM_AT["gate"], rows_per_gate=3), "r_out")


def test_norm_of_the_stream_alone():
    a = norm_args(n=NORM_AT["r"] + 64)
    a.o = a.gate = a.w_post = a.scale = a.r_out = None
    refused("ssd_block_norm", a, "n")
