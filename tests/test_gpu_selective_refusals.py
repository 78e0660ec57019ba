"""What the public calls refuse of CUDA tensors, before anything is enqueued."""
import pytest
import torch

import mamba_ssd_chunked_fwd_gb300 as ssd

pytestmark = pytest.mark.gpu

F32, F16, BF16, F64 = torch.float32, torch.float16, torch.bfloat16, torch.float64
B, L, D, N, G, W, S = 2, 5, 24, 16, 2, 4, 3


def t(*shape, dt=BF16):
    return torch.zeros(shape, device="cuda", dtype=dt)


def ints(*shape, dt=torch.int32):
    return torch.zeros(shape, device="cuda", dtype=dt)


def refused(fn, good, over, error, match):
    with pytest.raises(error, match=match):
        fn(**{**good, **over})


def scan_inputs():
    return dict(x=t(B, L, D), dt=t(B, L, D), A=t(D, N, dt=F32), B=t(B, L, G, N), C=t(B, L, G, N), D=t(D, dt=F32), z=t(B, L, D),
                dt_bias=t(D, dt=F32), initial_states=t(B, D, N, dt=F32), lengths=ints(B))


SCAN = [
    (dict(x=lambda: t(L, D)), "x: 2 dimensions"), (dict(B=lambda: t(B, L, N)), "B: 3 dimensions"), (dict(A=lambda: t(D, dt=F32)), "A: 1 dimensions"),
    (dict(x=lambda: t(B, L, D, dt=F64), dt=lambda: t(B, L, D, dt=F64)), "unsupported dtype"),
    (dict(dt=lambda: t(B, L, D, dt=F16)), "dt: dtype"), (dict(dt=lambda: t(B, L + 1, D)), "dt: shape"), (dict(dt=lambda: None), "dt is required"),
    (dict(A=lambda: t(D, N)), "A: dtype"), (dict(A=lambda: t(D, N + 1, dt=F32)), "A: shape"), (dict(A=lambda: t(N, D, dt=F32).t()), "A: must be contiguous"),
    (dict(C=lambda: t(B, L, G, N + 1)), "C: shape"), (dict(C=lambda: t(B, L, G, N, dt=F32)), "C: dtype"),
    (dict(C=lambda: t(B, L, N, G).transpose(2, 3)), "C: the values of a token"), (dict(z=lambda: t(B, L, D, dt=F32)), "z: dtype"),
    (dict(z=lambda: t(B, D, L).transpose(1, 2)), "z: the values of a token"), (dict(z=lambda: t(1, 1, D).expand(B, L, D)), "z: broadcast"),
    (dict(D=lambda: t(D + 1, dt=F32)), "D: shape"), (dict(D=lambda: "no"), "D: not a tensor"), (dict(dt_bias=lambda: t(D)), "dt_bias: dtype"),
    (dict(initial_states=lambda: t(B, N, D, dt=F32)), "initial_states: shape"), (dict(initial_states=lambda: t(B, D, N)), "initial_states: dtype"),
    (dict(lengths=lambda: ints(B, dt=torch.int64)), "lengths: dtype"), (dict(lengths=lambda: ints(B + 1)), "lengths: shape"),
    (dict(lengths=lambda: ints(B).cpu()), "lengths: on cpu"), (dict(z=lambda: t(B, L, D).cpu()), "z: on cpu"),
]


@pytest.mark.parametrize("over,match", SCAN)
def test_scan(over, match):
    over = {k: f() for k, f in over.items()}
    refused(ssd.selective_scan, scan_inputs(), over, ValueError, match)
    refused(ssd.selective_scan_bwd, {**scan_inputs(), "dy": t(B, L, D)}, over, ValueError, match)


@pytest.mark.parametrize("out,match", [(lambda: t(B, L, D + 1), "out: shape"), (lambda: t(B, L, D, dt=F32), "out: dtype"),
                                       (lambda: t(B, L, 2 * D)[..., :D], "out: must be contiguous"), (lambda: t(B, L, D).cpu(), "out: on cpu")])
def test_scan_output(out, match):
    refused(ssd.selective_scan, scan_inputs(), dict(out=out()), ValueError, match)


@pytest.mark.parametrize("over,match", [
    (dict(dy=lambda: t(B, L, D, dt=F32)), "dy: dtype"), (dict(dy=lambda: t(B, L, 2 * D)[..., :D]), "dy: must be contiguous"),
    (dict(dfinal=lambda: t(B, D, N)), "dfinal: dtype"), (dict(dfinal=lambda: t(B, D, N + 1, dt=F32)), "dfinal: shape")])
def test_scan_gradients(over, match):
    refused(ssd.selective_scan_bwd, {**scan_inputs(), "dy": t(B, L, D)}, {k: f() for k, f in over.items()}, ValueError, match)


def test_scan_errors_of_the_library():
    k = scan_inputs()
    odd = dict(B=t(B, L, 5, N), C=t(B, L, 5, N))
    wide = dict(A=t(D, 129, dt=F32), B=t(B, L, G, 129), C=t(B, L, G, 129), initial_states=None)
    none = dict(x=t(B, 0, D), dt=t(B, 0, D), z=None, B=t(B, 0, G, N), C=t(B, 0, G, N))
    for over, match in ((odd, "multiple of G"), (wide, "N must be"), (none, "every dim"), (dict(dt_limit=(2.0, 1.0)), "dt_limit"),
                        (dict(dt_limit=(float("nan"), 1.0)), "dt_limit"), (dict(out=k["B"].view(-1)[:1]), "out: shape")):
        refused(ssd.selective_scan, k, over, (ssd.SsdError, ValueError), match)
    buf = t(2 * B * L * D)
    refused(ssd.selective_scan, k, dict(x=buf[:B * L * D].view(B, L, D), out=buf[8:8 + B * L * D].view(B, L, D)), ssd.SsdError, "overlap")
    assert k["B"].numel() >= B * L * D
    refused(ssd.selective_scan, k, dict(out=k["B"].view(-1)[:B * L * D].view(B, L, D)), ssd.SsdError, "overlap")


def step_inputs():
    return dict(x=t(B, D), dt=t(B, D), A=t(D, N, dt=F32), B=t(B, G, N), C=t(B, G, N), state=t(S, D, N, dt=F32), slots=ints(B), D=t(D, dt=F32),
                z=t(B, D), dt_bias=t(D, dt=F32))


@pytest.mark.parametrize("over,match", [
    (dict(x=lambda: t(B, 1, D)), "x: 3 dimensions"), (dict(B=lambda: t(B, N)), "B: 2 dimensions"), (dict(state=lambda: t(S, D * N, dt=F32)), "state: 2 dimensions"),
    (dict(state=lambda: t(S, D, N)), "state: dtype"), (dict(state=lambda: t(S, N, D, dt=F32).transpose(1, 2)), "state: must be contiguous"),
    (dict(state=lambda: t(S, D + 1, N, dt=F32)), "state: shape"), (dict(state_out=lambda: t(S + 1, D, N, dt=F32)), "state_out: shape"),
    (dict(state_out=lambda: t(S, D, N)), "state_out: dtype"), (dict(slots=lambda: ints(B, dt=torch.int64)), "slots: dtype"),
    (dict(slots=lambda: ints(B + 1)), "slots: shape"), (dict(slots=lambda: ints(B).cpu()), "slots: on cpu"),
    (dict(x=lambda: t(1, D).expand(B, D)), "x: rows must be apart"), (dict(z=lambda: t(D, B).t()), "z: the values of a row"),
    (dict(dt=lambda: t(B, D, dt=F16)), "dt: dtype"), (dict(C=lambda: t(B, G, N + 1)), "C: shape"), (dict(out=lambda: t(B, 2 * D)[:, :D]), "out: must be contiguous")])
def test_step(over, match):
    refused(ssd.selective_scan_step, step_inputs(), {k: f() for k, f in over.items()}, ValueError, match)


def test_step_errors_of_the_library():
    k = step_inputs()
    refused(ssd.selective_scan_step, k, dict(state=t(1, D, N, dt=F32), slots=None), ssd.SsdError, "nslots")
    pool = t(S + 1, D, N, dt=F32)
    refused(ssd.selective_scan_step, k, dict(state=pool[:S], state_out=pool[1:]), ssd.SsdError, "overlap")


def conv_inputs():
    return dict(x=t(B, L, D), w=t(D, W, dt=F32), bias=t(D, dt=F32), initial_state=t(B, W - 1, D), lengths=ints(B))


@pytest.mark.parametrize("over,match", [
    (dict(x=lambda: t(L, D)), "x: 2 dimensions"), (dict(w=lambda: t(D, dt=F32)), "w: 1 dimensions"), (dict(w=lambda: t(D, W)), "w: dtype"),
    (dict(w=lambda: t(D + 1, W, dt=F32)), "w: shape"), (dict(w=lambda: t(W, D, dt=F32).t()), "w: must be contiguous"), (dict(bias=lambda: t(D)), "bias: dtype"),
    (dict(initial_state=lambda: t(B, W, D)), "initial_state: shape"), (dict(initial_state=lambda: t(B, W - 1, D, dt=F32)), "initial_state: dtype"),
    (dict(lengths=lambda: ints(B, dt=torch.int64)), "lengths: dtype"), (dict(x=lambda: t(B, D, L).transpose(1, 2)), "x: the values of a token"),
    (dict(x=lambda: t(1, 1, D).expand(B, L, D)), "x: broadcast"), (dict(w=lambda: t(D, W, dt=F32).cpu()), "w: on cpu")])
def test_conv(over, match):
    over = {k: f() for k, f in over.items()}
    refused(ssd.causal_conv1d_carry, conv_inputs(), over, ValueError, match)
    refused(ssd.causal_conv1d_bwd, {**conv_inputs(), "dy": t(B, L, D)}, over, ValueError, match)


def test_conv_errors_of_the_library():
    k = conv_inputs()
    refused(ssd.causal_conv1d_carry, k, dict(w=t(D, 9, dt=F32), initial_state=None), ssd.SsdError, "W must be")
    refused(ssd.causal_conv1d_carry, k, dict(out=k["x"]), ssd.SsdError, "overlap")
    refused(ssd.causal_conv1d_bwd, {**k, "dy": t(B, L, D, dt=F32)}, {}, ValueError, "dy: dtype")
    refused(ssd.causal_conv1d_bwd, {**k, "dy": t(B, L, D), "dfinal": t(B, W, D)}, {}, ValueError, "dfinal: shape")


def test_conv_step():
    k = dict(x=t(B, D), state=t(S, W - 1, D), w=t(D, W, dt=F32), slots=ints(B))
    for over, match in ((dict(x=t(B, 1, D)), "x: 3 dimensions"), (dict(state=t(S, W, D)), "state: shape"), (dict(state=t(S, W - 1, D, dt=F32)), "state: dtype"),
                        (dict(state_out=t(S, W - 1, D, dt=F32)), "state_out: dtype"), (dict(slots=ints(B, dt=torch.int64)), "slots: dtype"),
                        (dict(x=t(1, D).expand(B, D)), "rows must be apart"), (dict(bias=t(D + 1, dt=F32)), "bias: shape"), (dict(out=t(B, D + 1)), "out: shape")):
        refused(ssd.causal_conv1d_step, k, over, ValueError, match)
    refused(ssd.causal_conv1d_step, k, dict(state=t(1, W - 1, D), slots=None), ssd.SsdError, "nslots")


def norm_inputs():
    return dict(o=t(B, L, D), r=t(B, L, D, dt=F32), w_pre=t(D, dt=F32), w_post=t(D, dt=F32), gate=t(B, D), scale=t(D, dt=F32))


NORM = [
    (dict(o=lambda: t(B, L + 1, D)), "o: shape"), (dict(gate=lambda: t(B + 1, D)), "gate: shape"), (dict(gate=lambda: t(B, D + 1)), "gate: shape"),
    (dict(gate=lambda: t(B, 1, D)), "gate: shape"), (dict(gate=lambda: t(L, D)), "gate: shape"), (dict(gate=lambda: t(B, D, dt=F32)), "gate: dtype"),
    (dict(gate=lambda: t(B, 2 * D)[:, :D]), "gate: must be contiguous"), (dict(w_pre=lambda: t(D)), "w_pre: dtype"), (dict(w_pre=lambda: None), "w_pre is required"),
    (dict(w_pre=lambda: t(D + 1, dt=F32)), "w_pre: shape"), (dict(w_post=lambda: t(D, dt=F64)), "w_post: dtype"), (dict(scale=lambda: t(1, dt=F32)), "scale: shape"),
    (dict(o=lambda: t(B, L, 2 * D)[..., :D]), "o: must be contiguous"), (dict(scale=lambda: t(D, dt=F32).cpu()), "scale: on cpu")]


@pytest.mark.parametrize("over,match", NORM)
def test_norm(over, match):
    over = {k: f() for k, f in over.items()}
    refused(ssd.block_norm, norm_inputs(), over, ValueError, match)
    back = norm_inputs()
    back["r_out"] = back.pop("r")
    refused(ssd.block_norm_bwd, {**back, "dn": t(B, L, D), "dr_out": t(B, L, D, dt=F32)}, over, ValueError, match)


def test_norm_outputs_and_gradients():
    k = norm_inputs()
    for over, match in ((dict(out=t(B, L, D, dt=F32)), "out: dtype"), (dict(out=t(B, D)), "out: shape"), (dict(r_out=t(B, L, D)), "r_out: dtype"),
                        (dict(r=t(B, L, D, dt=F64)), "unsupported dtype"), (dict(r=t(B, L, 2 * D, dt=F32)[..., :D]), "r: must be contiguous")):
        refused(ssd.block_norm, k, over, ValueError, match)
    for over, match in ((dict(eps=-1.0), "eps"), (dict(r=t(B, L, D, dt=F16)), "stream"), (dict(o=None, gate=None), "need o")):
        refused(ssd.block_norm, k, over, ssd.SsdError, match)
    same = t(B, L, D)
    refused(ssd.block_norm, {**k, "r": t(B, L, D)}, dict(out=same, r_out=same), ssd.SsdError, "overlap")
    back = {n: v for n, v in k.items() if n != "r"}
    for over, match in ((dict(dn=t(B, L + 1, D)), "dn: shape"), (dict(dr_out=t(B, L, D)), "dr_out: dtype"), (dict(r_out=t(B, L, D, dt=F32).cpu()), "CUDA")):
        refused(ssd.block_norm_bwd, {**back, "r_out": k["r"], "dn": t(B, L, D), "dr_out": t(B, L, D, dt=F32)}, over, ValueError, match)
