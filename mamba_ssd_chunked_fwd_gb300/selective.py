"""Selective scan, its short convolution, and the block norm: Python binding.

Like the rest of the package this only marshals torch tensors into the C ABI of
``include/ssd.h``: every step runs in ``libssd_gb300.so`` on the current stream
of the tensors' device, and a bad argument raises ``SsdError`` (from the
library) or ``ValueError`` (a shape, type or device the binding cannot express).
The functions here pass their arguments on to ``csrc/binding.cpp``, which does
the marshalling; the ctypes structures and ``make_*_args`` are for callers of
the C entries themselves.

No call is recorded by autograd: from inputs that require gradients come results
that carry none (the ``*_bwd`` functions give them), and a state that is updated
in place keeps its version counter.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import threading

import torch

_i64, _i32, _f32, _ptr_t, _size = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class SsdScanArgs(ctypes.Structure):
    """Mirror of ``ssd_scan_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "L", "D", "N", "G")]
                + [(n, _ptr_t) for n in ("x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "initial_state", "lengths",
                                         "y", "final_state")]
                + [(n, _i64 * 2) for n in ("x_stride", "dt_stride", "z_stride", "b_stride", "c_stride")]
                + [("x_dtype", _i32), ("dt_dtype", _i32), ("dt_softplus", _i32), ("dt_min", _f32), ("dt_max", _f32),
                   ("workspace", _ptr_t), ("workspace_bytes", _size)])


class SsdScanBwdArgs(ctypes.Structure):
    """Mirror of ``ssd_scan_bwd_args`` in include/ssd.h."""
    _fields_ = ([("fwd", SsdScanArgs)]
                + [(n, _ptr_t) for n in ("dy", "dfinal", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0",
                                         "workspace")]
                + [("workspace_bytes", _size)])


class SsdScanStepArgs(ctypes.Structure):
    """Mirror of ``ssd_scan_step_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "D", "N", "G", "nslots")]
                + [(n, _ptr_t) for n in ("x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "state", "state_out", "slots",
                                         "y")]
                + [(n, _i64) for n in ("x_row", "dt_row", "z_row", "b_row", "c_row")]
                + [("x_dtype", _i32), ("dt_dtype", _i32), ("dt_softplus", _i32), ("dt_min", _f32), ("dt_max", _f32)])


class SsdConvArgs(ctypes.Structure):
    """Mirror of ``ssd_conv_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "L", "C", "W")] + [("x", _ptr_t), ("x_stride", _i64 * 2)]
                + [(n, _ptr_t) for n in ("w", "bias", "initial_state", "lengths", "y", "final_state")]
                + [("dtype", _i32), ("silu", _i32)])


class SsdConvBwdArgs(ctypes.Structure):
    """Mirror of ``ssd_conv_bwd_args`` in include/ssd.h."""
    _fields_ = ([("fwd", SsdConvArgs)] + [(n, _ptr_t) for n in ("dy", "dfinal", "dx", "dw", "dbias", "dh0", "workspace")]
                + [("workspace_bytes", _size)])


class SsdConvStepArgs(ctypes.Structure):
    """Mirror of ``ssd_conv_step_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("B", "C", "W", "nslots")] + [("x", _ptr_t), ("x_row", _i64)]
                + [(n, _ptr_t) for n in ("w", "bias", "state", "state_out", "slots", "y")]
                + [("dtype", _i32), ("silu", _i32)])


class SsdBlockNormArgs(ctypes.Structure):
    """Mirror of ``ssd_block_norm_args`` in include/ssd.h."""
    _fields_ = ([(n, _i64) for n in ("rows", "D", "rows_per_gate")]
                + [(n, _ptr_t) for n in ("o", "r", "gate", "w_post", "w_pre", "scale", "n", "r_out")]
                + [("dtype", _i32), ("stream_dtype", _i32), ("eps", _f32)])


class SsdBlockNormBwdArgs(ctypes.Structure):
    """Mirror of ``ssd_block_norm_bwd_args`` in include/ssd.h."""
    _fields_ = ([("fwd", SsdBlockNormArgs)]
                + [(n, _ptr_t) for n in ("dn", "dr_out", "d_o", "dr", "dgate", "dw_post", "dw_pre", "dscale", "workspace")]
                + [("workspace_bytes", _size)])


def _sized(cls):
    return [ctypes.POINTER(cls), ctypes.POINTER(_size)]


def _called(cls):
    return [ctypes.POINTER(cls), _ptr_t]


SIGNATURES = {
    "ssd_selective_scan_workspace_size": _sized(SsdScanArgs),
    "ssd_selective_scan": _called(SsdScanArgs),
    "ssd_selective_scan_bwd_workspace_size": _sized(SsdScanBwdArgs),
    "ssd_selective_scan_bwd": _called(SsdScanBwdArgs),
    "ssd_selective_scan_step": _called(SsdScanStepArgs),
    "ssd_causal_conv_carry": _called(SsdConvArgs),
    "ssd_causal_conv_bwd_workspace_size": _sized(SsdConvBwdArgs),
    "ssd_causal_conv_bwd": _called(SsdConvBwdArgs),
    "ssd_causal_conv_step": _called(SsdConvStepArgs),
    "ssd_block_norm": _called(SsdBlockNormArgs),
    "ssd_block_norm_bwd_workspace_size": _sized(SsdBlockNormBwdArgs),
    "ssd_block_norm_bwd": _called(SsdBlockNormBwdArgs),
}

_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_pkg = _ext = None
_lock = threading.Lock()


def _binding():
    """The package and its C++ binding, loaded (and built, if stale) on first use."""
    global _pkg, _ext
    with _lock:
        if _ext is None:
            import mamba_ssd_chunked_fwd_gb300 as pkg
            pkg.load_library()
            spec = importlib.util.spec_from_file_location("_ssd_binding", pkg._build.build_binding())
            ext = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(ext)
            ext.load(pkg.library_path())
            _pkg, _ext = pkg, ext
    return _ext


def _run(name, entry, x, *args):
    """The binding's function ``name`` on x's device and its current stream."""
    fn = getattr(_ext or _binding(), name)
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    if torch.cuda.current_device() == dev:
        out = fn(torch._C._cuda_getCurrentRawStream(dev), *args)
    else:
        with torch.cuda.device(dev):
            out = fn(torch._C._cuda_getCurrentRawStream(dev), *args)
    if type(out) is int:
        _pkg._check(out, entry)
    return out


def _code(t, what):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: unsupported dtype {t.dtype}")
    return code


def _refuse(t, shape, dtype, dev, what):
    """Says which of the checks a tensor fails (none: it is not dense)."""
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, expected CUDA device {dev}")
    raise ValueError(f"{what}: must be contiguous")


def _dense(t, shape, dtype, dev, what):
    """The address of a dense tensor of this shape and type, or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, shape, dtype, dev, what)
    return t.data_ptr()


def _inner_dense(shape, st, lead):
    """Whether the dimensions after the first ``lead`` are dense among themselves."""
    want = 1
    for n, s in zip(reversed(shape[lead:]), reversed(st[lead:])):
        if n != 1 and s != want:
            return False
        want *= n
    return True


_DENSE = (0, 0)


def _tokens(t, shape, dtype, dev, what):
    """(address, (batch stride, token stride)) of a [B,L,...] tensor whose tokens are dense."""
    if t is None:
        return None, _DENSE
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, shape, dtype, dev, what)
    if t.is_contiguous():
        return t.data_ptr(), _DENSE
    st = t.stride()
    if not _inner_dense(shape, st, 2):
        raise ValueError(f"{what}: the values of a token must be contiguous")
    st = (0 if shape[0] == 1 else st[0], 0 if shape[1] == 1 else st[1])
    if st == _DENSE and t.numel():
        if shape[1] != 1:
            raise ValueError(f"{what}: broadcast over every token")
        st = (0, t.numel() // shape[0])  # one token for every sequence; two zeros would mean dense
    return t.data_ptr(), st


def _ndim(t, n, what):
    if t.dim() != n:
        raise ValueError(f"{what}: {t.dim()} dimensions, expected {n}")


def _dt_dtype(x, dt):
    if dt.dtype is not x.dtype and dt.dtype is not torch.float32:
        raise ValueError(f"dt: dtype {dt.dtype}, expected {x.dtype} or torch.float32")
    return dt.dtype


# ---- selective scan ----------------------------------------------------------

def make_scan_args(x, dt, A, B, C, *, y=None, final_state=None, D=None, z=None, dt_bias=None, initial_states=None,
                   lengths=None, dt_softplus=False, dt_limit=(0.0, math.inf)) -> SsdScanArgs:
    """Fill an ``ssd_scan_args`` from tensors (no copies).  x, dt, z [B,L,D] and
    B, C [B,L,G,N] may be strided over batch and tokens."""
    _ndim(x, 3, "x"), _ndim(B, 4, "B"), _ndim(A, 2, "A")
    xs, dev, f32, io = x.shape, x.get_device(), torch.float32, x.dtype
    Bb, L, Dm = xs
    bc = (Bb, L, B.shape[2], B.shape[3])
    N = bc[3]
    code, dtt, state = _code(x, "x"), _dt_dtype(x, dt), (Bb, Dm, N)
    px, sx = _tokens(x, xs, io, dev, "x")
    pdt, sdt = _tokens(dt, xs, dtt, dev, "dt")
    pz, sz = _tokens(z, xs, io, dev, "z")
    pb, sb = _tokens(B, bc, io, dev, "B")
    pc, sc = _tokens(C, bc, io, dev, "C")
    return SsdScanArgs(
        Bb, L, Dm, N, bc[2], px, pdt, _dense(A, (Dm, N), f32, dev, "A"), pb, pc, _dense(D, (Dm,), f32, dev, "D"), pz,
        _dense(dt_bias, (Dm,), f32, dev, "dt_bias"), _dense(initial_states, state, f32, dev, "initial_states"),
        _dense(lengths, (Bb,), torch.int32, dev, "lengths"), _dense(y, xs, io, dev, "y"),
        _dense(final_state, state, f32, dev, "final_state"), sx, sdt, sz, sb, sc, code, _CODES[dtt],
        1 if dt_softplus else 0, dt_limit[0], dt_limit[1])


def selective_scan(x, dt, A, B, C, dt_softplus=False, return_final_state=False, *, D=None, z=None, dt_bias=None,
                   dt_limit=(0.0, math.inf), initial_states=None, lengths=None, out=None):
    """Selective scan over prompts on the GPU: for every channel c of D and state n of N

        h_t = exp(d_t A[c]) h_{t-1} + d_t x_t B_t,   y_t = (h_t . C_t + D x_t) silu(z_t),
        d_t = clamp(softplus(dt_t + dt_bias))

    Returns y [B,L,D], or (y, final_state [B,D,N] fp32).  x, z [B,L,D] and B, C
    [B,L,G,N] share a dtype (fp32, fp16, bf16), dt [B,L,D] has it too or is
    fp32; they may be slices of wider tensors along the last dimension.  A
    [D,N], D, dt_bias [D] and initial_states [B,D,N] are fp32.  ``lengths``
    (int32 [B], on the GPU): tokens per row; y is 0 past them.  ``out``: y's
    memory; it may be x, z or dt itself where that is dense and of y's type, and
    is refused where it overlaps an input otherwise."""
    return _run("selective_scan", "ssd_selective_scan", x, x, dt, A, B, C, dt_softplus, dt_limit[0], dt_limit[1], D, z, dt_bias,
                initial_states, lengths, return_final_state, out)


def selective_scan_bwd(x, dt, A, B, C, dy, dt_softplus=False, *, dfinal=None, D=None, z=None, dt_bias=None,
                       dt_limit=(0.0, math.inf), initial_states=None, lengths=None, want_dh0=None):
    """Gradients of sum(dy * y) + sum(dfinal * final_state) of ``selective_scan``
    with these inputs.  Returns a dict: dx, ddt, dA, dB, dC and, where the
    matching input is given, dD, dz, ddt_bias, dh0 (``want_dh0`` overrides the
    last).  dx, dB, dC, dz have x's dtype, ddt has dt's, the others are fp32."""
    return _run("selective_scan_bwd", "ssd_selective_scan_bwd", x, x, dt, A, B, C, dt_softplus, dt_limit[0], dt_limit[1], D, z,
                dt_bias, initial_states, lengths, dy, dfinal, want_dh0)


def selective_scan_step(x, dt, A, B, C, state, dt_softplus=False, *, state_out=None, slots=None, D=None, z=None,
                        dt_bias=None, dt_limit=(0.0, math.inf), out=None):
    """One token of the scan for each row: x, dt, z [B,D], B, C [B,G,N]; advances
    ``state`` [S,D,N] fp32 in place, or into ``state_out``; returns y [B,D].
    ``slots`` (int32 [B], on the GPU): the row's place in the state pool (default
    its own index); a row whose slot is outside the pool gives 0 and moves no
    state.  Rows must not share a slot."""
    return _run("selective_scan_step", "ssd_selective_scan_step", x, x, dt, A, B, C, state, dt_softplus, dt_limit[0], dt_limit[1],
                state_out, slots, D, z, dt_bias, out)


# ---- its convolution ---------------------------------------------------------

def make_conv_args(x, w, bias=None, *, y=None, final_state=None, initial_state=None, lengths=None, silu=True) -> SsdConvArgs:
    """Fill an ``ssd_conv_args`` from tensors (no copies)."""
    _ndim(x, 3, "x"), _ndim(w, 2, "w")
    xs, W, dev, f32, io = x.shape, w.shape[1], x.get_device(), torch.float32, x.dtype
    Bb, L, Cc = xs
    code, state = _code(x, "x"), (Bb, W - 1, Cc)
    px, sx = _tokens(x, xs, io, dev, "x")
    return SsdConvArgs(
        Bb, L, Cc, W, px, sx, _dense(w, (Cc, W), f32, dev, "w"), _dense(bias, (Cc,), f32, dev, "bias"),
        _dense(initial_state, state, io, dev, "initial_state"), _dense(lengths, (Bb,), torch.int32, dev, "lengths"),
        _dense(y, xs, io, dev, "y"), _dense(final_state, state, io, dev, "final_state"), code, 1 if silu else 0)


def causal_conv1d_carry(x, w, bias=None, silu=True, *, initial_state=None, lengths=None, return_final_state=False, out=None):
    """Depthwise causal conv1d over token-major prompts x [B,L,C] (may be strided
    over batch and tokens), continuing from ``initial_state`` [B,W-1,C] (the
    inputs before the first token; default zeros), then SiLU.  w [C,W], bias [C]
    fp32, W <= 8.  Returns y, or (y, final_state [B,W-1,C] in x's dtype);
    ``lengths`` as in ``selective_scan``."""
    return _run("causal_conv1d_carry", "ssd_causal_conv_carry", x, x, w, bias, silu, initial_state, lengths, return_final_state, out)


def causal_conv1d_bwd(x, w, dy, bias=None, silu=True, *, dfinal=None, initial_state=None, lengths=None, want_dh0=None):
    """Gradients of sum(dy * y) + sum(dfinal * final_state) of
    ``causal_conv1d_carry``: a dict of dx, dw, and dbias and dh0 where bias and
    initial_state are given (``want_dh0`` overrides the last)."""
    return _run("causal_conv1d_bwd", "ssd_causal_conv_bwd", x, x, w, bias, silu, initial_state, lengths, dy, dfinal, want_dh0)


def causal_conv1d_step(x, state, w, bias=None, silu=True, *, state_out=None, slots=None, out=None):
    """One token of the convolution for each row: x [B,C]; advances ``state``
    [S,W-1,C] (x's dtype) in place, or into ``state_out``; returns y [B,C].
    ``slots`` as in ``selective_scan_step``."""
    return _run("causal_conv1d_step", "ssd_causal_conv_step", x, x, state, w, bias, silu, state_out, slots, out)


# ---- block norm --------------------------------------------------------------

def block_norm(o, r, w_pre, *, w_post=None, gate=None, scale=None, eps=1e-5, dtype=None, out=None, r_out=None):
    """The end of one block and the norm before the next:

        r' = r + scale * gate * (o / rms(o) * w_post),   n = r' / rms(r') * w_pre

    Returns (n, r').  o [..., D] (None: only the norm of r, in ``dtype`` or r's);
    the residual stream r has o's dtype or fp32; gate, in o's dtype, has o's
    shape or is [B, D] for o [B, ..., D]; w_post (None: o is added as it is),
    w_pre and scale [D] fp32.  ``r_out`` may be r itself; ``out`` and ``r_out`` are
    refused where they overlap each other, a weight or part of an input."""
    like = None
    if o is None:
        if r_out is not None:
            raise ValueError("r_out needs o")
        if dtype is not None:
            like = torch.empty(0, dtype=dtype)
    elif dtype is not None and dtype is not o.dtype:
        raise ValueError(f"dtype: {dtype}, but n has o's {o.dtype}")
    return _run("block_norm", "ssd_block_norm", r, o, r, w_pre, w_post, gate, scale, eps, like, out, r_out)


def block_norm_bwd(dn, dr_out, o, r_out, w_pre, *, w_post=None, gate=None, scale=None, eps=1e-5):
    """Gradients of sum(dn * n) + sum(dr_out * r') of ``block_norm`` from its
    stored r' (``r_out``): a dict of dr, dw_pre, and with o also do, and dw_post,
    dgate, dscale where those inputs are given.  ``dr_out`` may be None."""
    return _run("block_norm_bwd", "ssd_block_norm_bwd", dn, o, r_out, w_pre, w_post, gate, scale, eps, dn, dr_out)
