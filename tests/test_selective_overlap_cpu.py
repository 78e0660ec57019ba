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
