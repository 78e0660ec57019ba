"""Host side of the gated delta rule and of the norm of queries and keys: what the C entries
refuse before anything is enqueued, workspace sizes, structures, and the plain forms
against closed ones."""
import ctypes
import os
import subprocess

import pytest
import torch

import _delta_ref as ref
import mamba_ssd_chunked_fwd_gb300 as ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MB = 1 << 20
DELTA = ("q", "k", "v", "g", "beta", "initial_state", "lengths", "y", "final_state")
AT = {n: (16 + 4 * i) * MB for i, n in enumerate(DELTA)}


def call(name, a):
    lib = ssd.load_library()
    st = getattr(lib, name)(ctypes.byref(a), None)
    return st, lib.ssd_last_error_detail().decode()


def put(a, over):
    for k, v in over.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def delta_args(**over):
    a = ssd.SsdDeltaArgs()
    a.B, a.L, a.H, a.G, a.N, a.P = 2, 64, 4, 2, 32, 16
    a.dtype, a.g_dtype, a.beta_dtype, a.scale = 2, 0, 2, 0.1
    a.workspace, a.workspace_bytes = 512 * MB, 64 * MB
    return put(put(a, AT), over)


BAD = [(dict(B=0), 1), (dict(L=0), 1), (dict(H=-1), 1), (dict(G=3), 1), (dict(N=0), 1), (dict(P=0), 1), (dict(N=129), 2), (dict(P=1025), 2),
       (dict(L=1 << 31), 2), (dict(B=1 << 17), 2), (dict(B=65536, H=64), 2), (dict(dtype=3), 1), (dict(g_dtype=1), 2), (dict(beta_dtype=7), 1),
       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(v_stride=(-1, 4)), 1)]


@pytest.mark.parametrize("over,code", BAD + [(dict(q=None), 1), (dict(beta=None), 1), (dict(y=None), 1)])
def test_rule_refuses(over, code):
    assert call("ssd_delta_rule", delta_args(**over))[0] == code


def bwd_args(**over):
    b = ssd.SsdDeltaBwdArgs()
    b.fwd = delta_args(**{k: v for k, v in over.items() if k in dict(ssd.SsdDeltaArgs._fields_) and k not in ("workspace", "workspace_bytes")})
    for i, n in enumerate(("dy", "dq", "dk", "dv", "dg", "dbeta")):
        setattr(b, n, (600 + 4 * i) * MB)
    b.workspace, b.workspace_bytes = 512 * MB, 64 * MB
    return put(b, {k: v for k, v in over.items() if k in dict(ssd.SsdDeltaBwdArgs._fields_)})


@pytest.mark.parametrize("over,code", BAD + [({n: None}, 1) for n in ("dy", "dq", "dk", "dv", "dg", "dbeta")]
                         + [(dict(workspace=None), 3), (dict(workspace_bytes=100), 3), (dict(workspace=512 * MB + 16), 3)])
def test_gradients_refuse(over, code):
    assert call("ssd_delta_rule_bwd", bwd_args(**over))[0] == code


def test_workspace_queries():
    n = ctypes.c_size_t(0)
    lib = ssd.load_library()
    assert lib.ssd_delta_rule_workspace_size(ctypes.byref(delta_args()), ctypes.byref(n)) == 0
    assert lib.ssd_delta_rule_bwd_workspace_size(ctypes.byref(bwd_args()), ctypes.byref(n)) == 0
    assert n.value >= 2 * 2 * 4 * 32 * 16 * 4
    assert lib.ssd_delta_rule_bwd_workspace_size(ctypes.byref(bwd_args()), None) == 1
    assert lib.ssd_delta_rule_workspace_size(None, ctypes.byref(n)) == 1


Y, STATE = 2 * 64 * 4 * 16 * 2, 2 * 4 * 16 * 32 * 4


@pytest.mark.parametrize("name", [n for n in DELTA if n != "y"])
def test_output_over_inputs(name):
    for y in (AT[name], AT[name] + 4 - Y):
        st, detail = call("ssd_delta_rule", delta_args(y=y))
        assert st == 1 and "overlap" in detail and "y" in detail


@pytest.mark.parametrize("name", [n for n in DELTA if n not in ("y", "final_state")])
def test_final_state_over_inputs(name):
    for at in (AT[name], AT[name] + 4 - STATE):
        st, detail = call("ssd_delta_rule", delta_args(final_state=at))
        assert st == 1 and "overlap" in detail and "final_state" in detail


def test_output_in_the_gaps_of_a_strided_input():
    st, detail = call("ssd_delta_rule", delta_args(v_stride=(64 * 4096, 4096), y=AT["v"] + 2048))
    assert st == 1 and "overlap v" in detail


STEP = ("q", "k", "v", "g", "beta", "state", "slots", "y")
STEP_AT = {n: (16 + 4 * i) * MB for i, n in enumerate(STEP)}


def step_args(**over):
    a = ssd.SsdDeltaStepArgs()
    a.B, a.H, a.G, a.N, a.P, a.nslots = 2, 4, 2, 32, 16, 8
    a.dtype, a.g_dtype, a.beta_dtype, a.scale = 2, 0, 2, 0.1
    a = put(a, STEP_AT)
    a.state_out = a.state
    return put(a, over)


@pytest.mark.parametrize("over,code", [(dict(B=0), 1), (dict(G=3), 1), (dict(N=200), 2), (dict(nslots=0), 1), (dict(dtype=9), 1), (dict(g_dtype=1), 2),
                                       (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(state_out=None), 1), (dict(slots=None, nslots=1), 1),
                                       (dict(k_row=-4), 1)])
def test_step_refuses(over, code):
    assert call("ssd_delta_rule_step", step_args(**over))[0] == code


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "slots", "state"])
def test_step_outputs_over_inputs(name):
    st, detail = call("ssd_delta_rule_step", step_args(y=STEP_AT[name]))
    assert st == 1 and "overlap" in detail
    if name != "state":
        st, detail = call("ssd_delta_rule_step", step_args(state_out=STEP_AT[name]))
        assert st == 1 and "overlap" in detail
    st, detail = call("ssd_delta_rule_step", step_args(state_out=STEP_AT["state"] + 64))
    assert st == 1 and "overlap state" in detail


NORM = ("q", "k", "w_q", "w_k", "freqs", "positions", "q_out", "k_out")
NORM_AT = {n: (16 + 4 * i) * MB for i, n in enumerate(NORM)}


def norm_args(**over):
    a = ssd.SsdQkNormArgs()
    a.B, a.L, a.H, a.G, a.N, a.nfreq = 2, 64, 4, 2, 32, 8
    a.dtype, a.kind, a.eps = 2, ssd.SSD_NORM_RMS, 1e-6
    return put(put(a, NORM_AT), over)


BAD_NORM = [(dict(B=0), 1), (dict(G=0), 1), (dict(N=257), 2), (dict(N=0), 1), (dict(L=1 << 31), 2), (dict(dtype=5), 1), (dict(kind=2), 1),
            (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(nfreq=17), 1), (dict(nfreq=-1), 1),
            (dict(freqs=None), 1), (dict(q_stride=(-1, 1)), 1), (dict(q=None), 1), (dict(k=None), 1)]


@pytest.mark.parametrize("over,code", BAD_NORM + [(dict(q_out=None), 1), (dict(k_out=None), 1)])
def test_norm_refuses(over, code):
    assert call("ssd_qk_norm", norm_args(**over))[0] == code


def norm_bwd_args(**over):
    b = ssd.SsdQkNormBwdArgs()
    b.fwd = norm_args(**{k: v for k, v in over.items() if k in dict(ssd.SsdQkNormArgs._fields_)})
    for i, n in enumerate(("dq_out", "dk_out", "dq", "dk", "dw_q", "dw_k")):
        setattr(b, n, (600 + 4 * i) * MB)
    b.workspace, b.workspace_bytes = 512 * MB, 64 * MB
    return put(b, {k: v for k, v in over.items() if k in dict(ssd.SsdQkNormBwdArgs._fields_)})


@pytest.mark.parametrize("over,code", BAD_NORM + [({n: None}, 1) for n in ("dq_out", "dk_out", "dq", "dk", "dw_q", "dw_k")] + [(dict(workspace=None), 3)])
def test_norm_gradients_refuse(over, code):
    assert call("ssd_qk_norm_bwd", norm_bwd_args(**over))[0] == code


@pytest.mark.parametrize("out,own", [("q_out", "q"), ("k_out", "k")])
def test_norm_outputs_over_inputs(out, own):
    for n in NORM:
        if n in (out, own):
            continue
        st, detail = call("ssd_qk_norm", norm_args(**{out: NORM_AT[n]}))
        assert st == 1 and "overlap" in detail, n
    st, detail = call("ssd_qk_norm", norm_args(**{out: NORM_AT[own] + 64}))  # beside its own place
    assert st == 1 and "overlap" in detail
    st, detail = call("ssd_qk_norm", norm_args(**{out: NORM_AT[own], own + "_stride": (64 * 200, 200)}))  # over a slice of something wider
    assert st == 1 and "overlap" in detail


def test_structures_match_the_header(tmp_path):
    pairs = [("ssd_delta_args", ssd.SsdDeltaArgs), ("ssd_delta_bwd_args", ssd.SsdDeltaBwdArgs), ("ssd_delta_step_args", ssd.SsdDeltaStepArgs),
             ("ssd_qk_norm_args", ssd.SsdQkNormArgs), ("ssd_qk_norm_bwd_args", ssd.SsdQkNormBwdArgs)]
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


def test_binding_refuses_host_tensors_and_unknown_norms():
    q, v, g = torch.zeros(1, 4, 1, 8), torch.zeros(1, 4, 1, 8), torch.zeros(1, 4, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule(q, q, v, g, g)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule_bwd(q, q, v, g, g, v)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], torch.zeros(1, 1, 8, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.qk_norm(q, q)
    with pytest.raises(ValueError, match="norm"):
        ssd.qk_norm(q, q, norm="max")


def test_plain_rule_against_closed_forms():
    """Orthonormal keys and beta 1: a memory that gives back what was written last under a key; beta 0: decay alone."""
    gen = torch.Generator().manual_seed(1)
    eye = torch.eye(4, dtype=torch.float64)
    order = torch.tensor([0, 1, 0, 2, 3, 1])
    k = eye[order][None, :, None]
    v = torch.randn((1, 6, 1, 3), generator=gen, dtype=torch.float64)
    zero, one = torch.zeros((1, 6, 1), dtype=torch.float64), torch.ones((1, 6, 1), dtype=torch.float64)
    y, S = ref.delta(k, k, v, zero, one, scale=1.0)
    assert torch.allclose(y, v)
    for key, last in ((0, 2), (1, 5), (2, 3), (3, 4)):
        assert torch.allclose(S[0, 0] @ eye[key], v[0, last, 0])
    h0 = torch.randn((1, 1, 3, 4), generator=gen, dtype=torch.float64)
    _, S = ref.delta(k, k, v, zero - 0.5, zero, h0)
    assert torch.allclose(S, h0 * torch.exp(torch.tensor(-3.0, dtype=torch.float64)))


def test_plain_norm_keeps_lengths_and_relative_angles():
    gen = torch.Generator().manual_seed(2)
    q = torch.randn((1, 1, 1, 8), generator=gen, dtype=torch.float64).expand(1, 5, 1, 8)
    k = torch.randn((1, 1, 1, 8), generator=gen, dtype=torch.float64).expand(1, 5, 1, 8)
    f = torch.tensor([1.0, 0.3, 0.1, 0.01], dtype=torch.float64)
    for interleaved in (False, True):
        a, b = ref.qk_norm(q, k, norm="l2", freqs=f, eps=0.0, interleaved=interleaved)
        assert torch.allclose(a.norm(dim=-1), torch.ones((), dtype=torch.float64))
        far, near = ref.qk_norm(q, k, norm="l2", freqs=f, eps=0.0, positions=torch.arange(5)[None] + 1000, interleaved=interleaved)
        for i in range(5):
            for j in range(5):
                assert torch.allclose((a[0, i] * b[0, j]).sum(), (far[0, i] * near[0, j]).sum())
