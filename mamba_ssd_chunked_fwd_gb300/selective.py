"""Selective scan, its short convolution, and the block norm: Python binding.

Like the rest of the package this only marshals torch tensors into the C ABI of
``include/ssd.h``: every step runs in ``libssd_gb300.so`` on the current stream
of the tensors' device, and a bad argument raises ``SsdError`` (from the
library) or ``ValueError`` (a shape, type or device the binding cannot express).
"""
from __future__ import annotations

import ctypes
import math
import struct

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
    return [_ptr_t, _ptr_t]  # the structure by reference, or its bytes


def _packer(cls):
    """The structure's layout for ``struct.pack``: filling it that way costs a
    fifth of the ctypes constructor, which counts in a call of a few microseconds."""
    code = {_i64: "q", _i32: "i", _f32: "f", _ptr_t: "P", _size: "N"}
    packed = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_))
    pad = ctypes.sizeof(cls) - packed.size  # the structure's tail
    return struct.Struct(packed.format + "%dx" % pad if pad else packed.format).pack


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

_pack_scan_step, _pack_conv_step = _packer(SsdScanStepArgs), _packer(SsdConvStepArgs)
_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_byref = ctypes.byref
_pkg = None


def _host():
    """The package (its loader and error check); imported late, since it imports this module."""
    global _pkg
    if _pkg is None:
        import mamba_ssd_chunked_fwd_gb300 as _pkg_module
        _pkg = _pkg_module
    return _pkg


def _call(name, args, dev):
    """One C entry on the current stream of CUDA device ``dev``; args: a
    reference to its structure, or the structure's bytes."""
    pkg = _pkg or _host()
    fn = getattr(pkg._lib or pkg.load_library(), name)
    if torch.cuda.current_device() == dev:
        status = fn(args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        pkg._check(status, name)


def _work(name, args, t):
    """Sizes args' workspace by the library's query and allocates it on t's
    device; the caller holds the tensor until its call is enqueued."""
    pkg, dev, out = _pkg or _host(), t.get_device(), _size(0)
    fn = getattr(pkg._lib or pkg.load_library(), name)
    if torch.cuda.current_device() == dev:
        status = fn(_byref(args), _byref(out))
    else:
        with torch.cuda.device(dev):
            status = fn(_byref(args), _byref(out))
    if status:
        pkg._check(status, name)
    if not out.value:
        return None
    ws = torch.empty(out.value, device=t.device, dtype=torch.uint8)
    args.workspace, args.workspace_bytes = ws.data_ptr(), out.value
    return ws


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
    """The address of a dense tensor of this shape and type, or 0 for None."""
    if t is None:
        return 0
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
        raise ValueError(f"{what}: broadcast over every token")
    return t.data_ptr(), st


def _rows(t, shape, dtype, dev, what):
    """(address, row stride) of a [B,...] tensor whose rows are dense."""
    if t is None:
        return 0, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, shape, dtype, dev, what)
    if t.is_contiguous():
        return t.data_ptr(), 0
    st = t.stride()
    if not _inner_dense(shape, st, 1):
        raise ValueError(f"{what}: the values of a row must be contiguous")
    if shape[0] == 1:
        return t.data_ptr(), 0
    if st[0] <= 0:
        raise ValueError(f"{what}: rows must be apart")
    return t.data_ptr(), st[0]


def _output(x, out):
    """(tensor, address) of a dense output of x's shape and type: ``out``, or a new one."""
    if out is not None:
        return out, _dense(out, x.shape, x.dtype, x.get_device(), "out")
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    return y, y.data_ptr()


def _ndim(t, n, what):
    if t.dim() != n:
        raise ValueError(f"{what}: {t.dim()} dimensions, expected {n}")


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} takes CUDA tensors")


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
    (int32 [B], on the GPU): tokens per row; y is 0 past them."""
    _cuda(x, "selective_scan")
    y = _output(x, out)[0]
    fin = torch.empty((x.shape[0], x.shape[2], A.shape[1]), device=x.device, dtype=torch.float32) if return_final_state else None
    a = make_scan_args(x, dt, A, B, C, y=y, final_state=fin, D=D, z=z, dt_bias=dt_bias, initial_states=initial_states,
                       lengths=lengths, dt_softplus=dt_softplus, dt_limit=dt_limit)
    ws = _work("ssd_selective_scan_workspace_size", a, x)  # noqa: F841
    _call("ssd_selective_scan", _byref(a), x.get_device())
    return (y, fin) if return_final_state else y


def selective_scan_bwd(x, dt, A, B, C, dy, dt_softplus=False, *, dfinal=None, D=None, z=None, dt_bias=None,
                       dt_limit=(0.0, math.inf), initial_states=None, lengths=None, want_dh0=None):
    """Gradients of sum(dy * y) + sum(dfinal * final_state) of ``selective_scan``
    with these inputs.  Returns a dict: dx, ddt, dA, dB, dC and, where the
    matching input is given, dD, dz, ddt_bias, dh0 (``want_dh0`` overrides the
    last).  dx, dB, dC, dz have x's dtype, ddt has dt's, the others are fp32."""
    _cuda(x, "selective_scan_bwd")
    dev, f32 = x.device, torch.float32

    def like(t):
        return torch.empty(t.shape, device=dev, dtype=t.dtype)

    a = SsdScanBwdArgs()
    a.fwd = make_scan_args(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, initial_states=initial_states, lengths=lengths,
                           dt_softplus=dt_softplus, dt_limit=dt_limit)
    state = (x.shape[0], x.shape[2], A.shape[1])
    a.dy = _dense(dy, x.shape, x.dtype, x.get_device(), "dy")
    a.dfinal = _dense(dfinal, state, f32, x.get_device(), "dfinal")
    g = {"dx": like(x), "ddt": like(dt), "dA": like(A), "dB": like(B), "dC": like(C)}
    if D is not None:
        g["dD"] = like(D)
    if z is not None:
        g["dz"] = like(z)
    if dt_bias is not None:
        g["ddt_bias"] = like(dt_bias)
    if want_dh0 if want_dh0 is not None else initial_states is not None:
        g["dh0"] = torch.empty(state, device=dev, dtype=f32)
    for k, t in g.items():
        setattr(a, k, t.data_ptr())
    ws = _work("ssd_selective_scan_bwd_workspace_size", a, x)  # noqa: F841
    _call("ssd_selective_scan_bwd", _byref(a), x.get_device())
    return g


def selective_scan_step(x, dt, A, B, C, state, dt_softplus=False, *, state_out=None, slots=None, D=None, z=None,
                        dt_bias=None, dt_limit=(0.0, math.inf), out=None):
    """One token of the scan for each row: x, dt, z [B,D], B, C [B,G,N]; advances
    ``state`` [S,D,N] fp32 in place, or into ``state_out``; returns y [B,D].
    ``slots`` (int32 [B], on the GPU): the row's place in the state pool (default
    its own index); a row whose slot is outside the pool gives 0 and moves no
    state.  Rows must not share a slot."""
    _cuda(x, "selective_scan_step")
    _ndim(x, 2, "x"), _ndim(B, 3, "B"), _ndim(state, 3, "state"), _ndim(A, 2, "A")
    xs, dev, f32, io = x.shape, x.get_device(), torch.float32, x.dtype
    Bb, Dm = xs
    bc = (Bb, B.shape[1], B.shape[2])
    pool = (state.shape[0], Dm, bc[2])
    code, dtt = _code(x, "x"), _dt_dtype(x, dt)
    y, py = _output(x, out)
    px, rx = _rows(x, xs, io, dev, "x")
    pdt, rdt = _rows(dt, xs, dtt, dev, "dt")
    pz, rz = _rows(z, xs, io, dev, "z")
    pb, rb = _rows(B, bc, io, dev, "B")
    pc, rc = _rows(C, bc, io, dev, "C")
    ps = _dense(state, pool, f32, dev, "state")
    a = _pack_scan_step(
        Bb, Dm, bc[2], bc[1], pool[0], px, pdt, _dense(A, (Dm, bc[2]), f32, dev, "A"), pb, pc,
        _dense(D, (Dm,), f32, dev, "D"), pz, _dense(dt_bias, (Dm,), f32, dev, "dt_bias"), ps,
        ps if state_out is None else _dense(state_out, pool, f32, dev, "state_out"),
        _dense(slots, (Bb,), torch.int32, dev, "slots"), py, rx, rdt, rz, rb, rc, code,
        _CODES[dtt], 1 if dt_softplus else 0, dt_limit[0], dt_limit[1])
    _call("ssd_selective_scan_step", a, dev)
    return y


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
    _cuda(x, "causal_conv1d_carry")
    y = _output(x, out)[0]
    fin = torch.empty((x.shape[0], w.shape[1] - 1, x.shape[2]), device=x.device, dtype=x.dtype) if return_final_state else None
    a = make_conv_args(x, w, bias, y=y, final_state=fin, initial_state=initial_state, lengths=lengths, silu=silu)
    _call("ssd_causal_conv_carry", _byref(a), x.get_device())
    return (y, fin) if return_final_state else y


def causal_conv1d_bwd(x, w, dy, bias=None, silu=True, *, dfinal=None, initial_state=None, lengths=None, want_dh0=None):
    """Gradients of sum(dy * y) + sum(dfinal * final_state) of
    ``causal_conv1d_carry``: a dict of dx, dw, and dbias and dh0 where bias and
    initial_state are given (``want_dh0`` overrides the last)."""
    _cuda(x, "causal_conv1d_bwd")
    dev = x.device
    a = SsdConvBwdArgs()
    a.fwd = make_conv_args(x, w, bias, initial_state=initial_state, lengths=lengths, silu=silu)
    state = (x.shape[0], w.shape[1] - 1, x.shape[2])
    a.dy = _dense(dy, x.shape, x.dtype, x.get_device(), "dy")
    a.dfinal = _dense(dfinal, state, x.dtype, x.get_device(), "dfinal")
    g = {"dx": torch.empty(x.shape, device=dev, dtype=x.dtype), "dw": torch.empty_like(w)}
    if bias is not None:
        g["dbias"] = torch.empty_like(bias)
    if want_dh0 if want_dh0 is not None else initial_state is not None:
        g["dh0"] = torch.empty(state, device=dev, dtype=x.dtype)
    for k, t in g.items():
        setattr(a, k, t.data_ptr())
    ws = _work("ssd_causal_conv_bwd_workspace_size", a, x)  # noqa: F841
    _call("ssd_causal_conv_bwd", _byref(a), x.get_device())
    return g


def causal_conv1d_step(x, state, w, bias=None, silu=True, *, state_out=None, slots=None, out=None):
    """One token of the convolution for each row: x [B,C]; advances ``state``
    [S,W-1,C] (x's dtype) in place, or into ``state_out``; returns y [B,C].
    ``slots`` as in ``selective_scan_step``."""
    _cuda(x, "causal_conv1d_step")
    _ndim(x, 2, "x"), _ndim(w, 2, "w"), _ndim(state, 3, "state")
    xs, W, dev, f32, io = x.shape, w.shape[1], x.get_device(), torch.float32, x.dtype
    Bb, Cc = xs
    pool = (state.shape[0], W - 1, Cc)
    code = _code(x, "x")
    y, py = _output(x, out)
    px, rx = _rows(x, xs, io, dev, "x")
    ps = _dense(state, pool, io, dev, "state")
    a = _pack_conv_step(
        Bb, Cc, W, pool[0], px, rx, _dense(w, (Cc, W), f32, dev, "w"), _dense(bias, (Cc,), f32, dev, "bias"), ps,
        ps if state_out is None else _dense(state_out, pool, io, dev, "state_out"),
        _dense(slots, (Bb,), torch.int32, dev, "slots"), py, code, 1 if silu else 0)
    _call("ssd_causal_conv_step", a, dev)
    return y


# ---- block norm --------------------------------------------------------------

def _norm_args(o, r, w_pre, w_post, gate, scale, eps, like):
    """The shared part; ``like`` is a tensor of o's shape and dtype."""
    if r.dim() < 1:
        raise ValueError("r: at least one dimension")
    D, dev, f32 = r.shape[-1], r.get_device(), torch.float32
    rows = r.numel() // max(D, 1)
    a = SsdBlockNormArgs()
    a.rows, a.D, a.rows_per_gate = rows, D, 1
    a.dtype, a.stream_dtype = _code(like, "o"), _code(r, "r")
    a.o = _dense(o, r.shape, like.dtype, dev, "o")
    if gate is not None:
        lead = 1
        if gate.shape != r.shape:  # [B, D] for [B, ..., D]
            if r.dim() < 2 or gate.shape != (r.shape[0], D):
                raise ValueError(f"gate: shape {tuple(gate.shape)}, expected {tuple(r.shape)} or {(r.shape[0], D)}")
            lead = rows // max(r.shape[0], 1)
        a.rows_per_gate = lead
        a.gate = _dense(gate, gate.shape, like.dtype, dev, "gate")
    a.w_post = _dense(w_post, (D,), f32, dev, "w_post")
    a.w_pre = _dense(w_pre, (D,), f32, dev, "w_pre")
    a.scale = _dense(scale, (D,), f32, dev, "scale")
    a.eps = float(eps)
    return a


def block_norm(o, r, w_pre, *, w_post=None, gate=None, scale=None, eps=1e-5, dtype=None, out=None, r_out=None):
    """The end of one block and the norm before the next:

        r' = r + scale * gate * (o / rms(o) * w_post),   n = r' / rms(r') * w_pre

    Returns (n, r').  o [..., D] (None: only the norm of r, in ``dtype`` or r's);
    the residual stream r has o's dtype or fp32; gate, in o's dtype, has o's
    shape or is [B, D] for o [B, ..., D]; w_post (None: o is added as it is),
    w_pre and scale [D] fp32.  ``r_out`` may be r itself."""
    _cuda(r, "block_norm")
    like = o if o is not None else torch.empty(0, device=r.device, dtype=dtype or r.dtype)
    a = _norm_args(o, r, w_pre, w_post, gate, scale, eps, like)
    n = out if out is not None else torch.empty(r.shape, device=r.device, dtype=like.dtype)
    dev = r.get_device()
    a.r = _dense(r, r.shape, r.dtype, dev, "r")
    a.n = _dense(n, r.shape, like.dtype, dev, "out")
    if o is not None:
        r_out = r_out if r_out is not None else torch.empty_like(r)
        a.r_out = _dense(r_out, r.shape, r.dtype, dev, "r_out")
    _call("ssd_block_norm", _byref(a), dev)
    return n, (r_out if o is not None else r)


def block_norm_bwd(dn, dr_out, o, r_out, w_pre, *, w_post=None, gate=None, scale=None, eps=1e-5):
    """Gradients of sum(dn * n) + sum(dr_out * r') of ``block_norm`` from its
    stored r' (``r_out``): a dict of dr, dw_pre, and with o also do, and dw_post,
    dgate, dscale where those inputs are given.  ``dr_out`` may be None."""
    _cuda(dn, "block_norm_bwd")
    dev = dn.get_device()
    a = SsdBlockNormBwdArgs()
    a.fwd = _norm_args(o, r_out, w_pre, w_post, gate, scale, eps, dn)
    a.fwd.r_out = _dense(r_out, r_out.shape, r_out.dtype, dev, "r_out")
    a.dn = _dense(dn, r_out.shape, dn.dtype, dev, "dn")
    a.dr_out = _dense(dr_out, r_out.shape, r_out.dtype, dev, "dr_out")
    g = {"dr": torch.empty_like(r_out), "dw_pre": torch.empty_like(w_pre)}
    if o is not None:
        g["do"] = torch.empty_like(o)
    for name, t in (("dw_post", w_post), ("dgate", gate), ("dscale", scale)):
        if t is not None:
            g[name] = torch.empty_like(t)
    for k, t in g.items():
        setattr(a, "d_o" if k == "do" else k, t.data_ptr())
    ws = _work("ssd_block_norm_bwd_workspace_size", a, dn)  # noqa: F841
    _call("ssd_block_norm_bwd", _byref(a), dev)
    return g
