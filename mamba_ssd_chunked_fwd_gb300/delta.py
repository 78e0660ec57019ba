"""Gated delta rule, and the norm of queries and keys: Python binding.

Like ``selective.py``, whose loader and error handling this shares: every step runs
in ``libssd_gb300.so`` on the current stream of the tensors' device, a bad argument
raises ``SsdError`` or ``ValueError``, and no call is recorded by autograd.
"""
from __future__ import annotations

import ctypes

from .selective import _called, _f32, _i32, _i64, _ptr_t, _run, _size, _sized

SSD_NORM_RMS, SSD_NORM_L2 = 0, 1
_NORMS = {"rms": SSD_NORM_RMS, "l2": SSD_NORM_L2}


class SsdDeltaArgs(ctypes.Structure):
    """Mirror of ``ssd_delta_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "L", "H", "G", "N", "P")]
                + [(n, _ptr_t) for n in ("q", "k", "v", "g", "beta", "initial_state", "lengths", "y", "final_state")]
                + [(n, _i64 * 2) for n in ("q_stride", "k_stride", "v_stride", "g_stride", "beta_stride")]
                + [("dtype", _i32), ("g_dtype", _i32), ("beta_dtype", _i32), ("scale", _f32), ("workspace", _ptr_t),
                   ("workspace_bytes", _size)])


class SsdDeltaBwdArgs(ctypes.Structure):
    """Mirror of ``ssd_delta_bwd_args`` in include/ssd.h."""
    _fields_ = ([("fwd", SsdDeltaArgs)]
                + [(n, _ptr_t) for n in ("dy", "dfinal", "dq", "dk", "dv", "dg", "dbeta", "dh0", "workspace")]
                + [("workspace_bytes", _size)])


class SsdDeltaStepArgs(ctypes.Structure):
    """Mirror of ``ssd_delta_step_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "H", "G", "N", "P", "nslots")]
                + [(n, _ptr_t) for n in ("q", "k", "v", "g", "beta", "state", "state_out", "slots", "y")]
                + [(n, _i64) for n in ("q_row", "k_row", "v_row", "g_row", "beta_row")]
                + [("dtype", _i32), ("g_dtype", _i32), ("beta_dtype", _i32), ("scale", _f32)])


class SsdQkNormArgs(ctypes.Structure):
    """Mirror of ``ssd_qk_norm_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "L", "H", "G", "N", "nfreq")]
                + [(n, _ptr_t) for n in ("q", "k", "w_q", "w_k", "freqs", "positions", "q_out", "k_out")]
                + [("q_stride", _i64 * 2), ("k_stride", _i64 * 2), ("dtype", _i32), ("kind", _i32), ("interleaved", _i32),
                   ("eps", _f32)])


class SsdQkNormBwdArgs(ctypes.Structure):
    """Mirror of ``ssd_qk_norm_bwd_args`` in include/ssd.h."""
    _fields_ = ([("fwd", SsdQkNormArgs)]
                + [(n, _ptr_t) for n in ("dq_out", "dk_out", "dq", "dk", "dw_q", "dw_k", "workspace")]
                + [("workspace_bytes", _size)])


SIGNATURES = {
    "ssd_delta_rule_workspace_size": _sized(SsdDeltaArgs),
    "ssd_delta_rule": _called(SsdDeltaArgs),
    "ssd_delta_rule_bwd_workspace_size": _sized(SsdDeltaBwdArgs),
    "ssd_delta_rule_bwd": _called(SsdDeltaBwdArgs),
    "ssd_delta_rule_step": _called(SsdDeltaStepArgs),
    "ssd_qk_norm": _called(SsdQkNormArgs),
    "ssd_qk_norm_bwd_workspace_size": _sized(SsdQkNormBwdArgs),
    "ssd_qk_norm_bwd": _called(SsdQkNormBwdArgs),
}


# ---- gated delta rule --------------------------------------------------------

def delta_rule(q, k, v, g, beta, *, scale=None, initial_states=None, lengths=None, return_final_state=False, out=None):
    """Gated delta rule over prompts on the GPU: for every head h, with the queries
    and keys of group h / (H / G) and the state S of P x N,

        S' = exp(g_t) S_{t-1},   u_t = beta_t (v_t - S' k_t),   S_t = S' + u_t k_t^T,   y_t = scale S_t q_t

    Returns y [B,L,H,P], or (y, final_state [B,H,P,N] fp32).  q, k [B,L,G,N] and v
    [B,L,H,P] share a dtype (fp32, fp16, bf16); g (the decay's logarithm, meant to be
    <= 0) and beta [B,L,H] each have it too or are fp32; all five may be slices of
    wider tensors along the last dimension.  N <= 128.  ``scale``: 1 / sqrt(N) by default.
    initial_states [B,H,P,N] fp32.  ``lengths`` (int32 [B], on the GPU): tokens per
    row; y is 0 past them.  ``out``: y's memory, refused where it overlaps an input.
    16-bit tensors in whole 16-byte pieces (N, P, strides, addresses) run in chunks on the tensor
    cores, all others token by token.  In chunks of fp16, precision is relative to the largest state and value
    of a row of P (gradients: of 128 rows), and q . k must stay below 65504."""
    return _run("delta_rule", "ssd_delta_rule", q, q, k, v, g, beta, scale, initial_states, lengths, return_final_state, out)


def delta_rule_bwd(q, k, v, g, beta, dy, *, scale=None, dfinal=None, initial_states=None, lengths=None, want_dh0=None):
    """Gradients of sum(dy * y) + sum(dfinal * final_state) of ``delta_rule`` with
    these inputs.  Returns a dict: dq, dk, dv, dg, dbeta, in the inputs' types, and dh0
    (fp32) where initial_states is given (``want_dh0`` overrides that)."""
    return _run("delta_rule_bwd", "ssd_delta_rule_bwd", q, q, k, v, g, beta, scale, initial_states, lengths, dy, dfinal, want_dh0)


def delta_rule_step(q, k, v, g, beta, state, *, scale=None, state_out=None, slots=None, out=None):
    """One token of the delta rule for each row: q, k [B,G,N], v [B,H,P], g, beta
    [B,H]; advances ``state`` [S,H,P,N] fp32 in place, or into ``state_out``; returns
    y [B,H,P].  ``slots`` (int32 [B], on the GPU): the row's place in the state pool
    (default its own index); a row whose slot is outside the pool gives 0 and moves no
    state.  Rows must not share a slot."""
    return _run("delta_rule_step", "ssd_delta_rule_step", q, q, k, v, g, beta, state, scale, state_out, slots, out)


# ---- norm of queries and keys ------------------------------------------------

def _norm_kind(norm):
    if norm not in _NORMS:
        raise ValueError(f"norm: {norm!r}, expected 'rms' or 'l2'")
    return _NORMS[norm]


def qk_norm(q, k, *, w_q=None, w_k=None, norm="rms", eps=1e-6, freqs=None, positions=None, interleaved=False, out_q=None,
            out_k=None):
    """Norm of every head of q [B,L,H,N] and k [B,L,G,N], and its rotation by position:

        x' = x / sqrt(mean(x^2) + eps) * w        (norm="l2": the sum in place of the mean)

    then pair i of x' turns by positions * freqs[i]: the pairs (i, R + i) of R = len(freqs), or
    (2 i, 2 i + 1) with ``interleaved``; what follows the first 2 R elements is not turned.
    Returns (q', k'), dense.  q and k share a dtype (fp32, fp16, bf16) and may be slices
    of wider tensors along the last dimension; w_q, w_k [N] and freqs [R] (None: no
    rotation) fp32, N <= 256; ``positions`` int32 [B,L] (default 0 .. L-1).  For single
    tokens: q [B,H,N], k [B,G,N], positions [B], which are required there with freqs.
    ``out_q``, ``out_k`` may be a dense q, k themselves."""
    return _run("qk_norm", "ssd_qk_norm", q, q, k, w_q, w_k, _norm_kind(norm), eps, freqs, positions, interleaved, out_q, out_k)


def qk_norm_bwd(dq_out, dk_out, q, k, *, w_q=None, w_k=None, norm="rms", eps=1e-6, freqs=None, positions=None, interleaved=False):
    """Gradients of sum(dq_out * q') + sum(dk_out * k') of ``qk_norm`` with these
    inputs: a dict of dq, dk, and dw_q, dw_k (fp32) where the weights are given."""
    return _run("qk_norm_bwd", "ssd_qk_norm_bwd", q, q, k, w_q, w_k, _norm_kind(norm), eps, freqs, positions, interleaved, dq_out,
                dk_out)
