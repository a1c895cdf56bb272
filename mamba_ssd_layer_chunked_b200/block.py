"""Python binding of the operators around the scan (see include/ssd.h): the
short causal convolution, the selective scan with a decay per channel and state,
and the norms of a block. Argument marshalling only, as in ssd.py.

Activations may be slices of a projection's output: their last dimension is
contiguous, the others may have any stride. Every call runs on the device of its
tensors and on that device's current torch stream, or on ``stream``; outputs and
workspaces are allocated on the stream the call runs on. Inputs must be ready on
that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from . import ssd as _ssd

_DTYPES = {torch.float32: _ssd.SSD_DTYPE_F32, torch.bfloat16: _ssd.SSD_DTYPE_BF16}
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_i64 = ctypes.c_int64
_HERE = contextlib.nullcontext()


class ConvProblem(ctypes.Structure):
    """Mirror of ssd_conv_problem."""

    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("width", _i64), ("nseq", _i64),
                ("x_stride", _i64 * 2), ("split", _i64 * 3), ("dtype", ctypes.c_int), ("act", ctypes.c_int)]


class SelectiveProblem(ctypes.Structure):
    """Mirror of ssd_selective_problem."""

    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("dstate", _i64), ("ngroups", _i64),
                ("nseq", _i64), ("u_stride", _i64 * 2), ("dt_stride", _i64 * 2), ("z_stride", _i64 * 2),
                ("B_stride", _i64 * 2), ("C_stride", _i64 * 2), ("dtype", ctypes.c_int),
                ("dt_softplus", ctypes.c_int32)]


class NormProblem(ctypes.Structure):
    """Mirror of ssd_norm_problem."""

    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("ngroups", _i64), ("x_stride", _i64 * 2),
                ("z_stride", _i64 * 2), ("dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("alpha", ctypes.c_float), ("gate_first", ctypes.c_int32)]


def declare(lib):
    """Argument types of the C functions this module calls."""
    vp, P = ctypes.c_void_p, ctypes.POINTER
    for name, argtypes, restype in (
            ("ssd_causal_conv", [P(ConvProblem)] + [vp] * 10, ctypes.c_int),
            ("ssd_conv_step", [P(ConvProblem)] + [vp] * 8, ctypes.c_int),
            ("ssd_selective_scan_workspace_bytes", [P(SelectiveProblem)], ctypes.c_size_t),
            ("ssd_selective_scan", [P(SelectiveProblem)] + [vp] * 13 + [ctypes.c_size_t, vp], ctypes.c_int),
            ("ssd_selective_step", [P(SelectiveProblem)] + [vp] * 11, ctypes.c_int),
            ("ssd_gated_norm", [P(NormProblem)] + [vp] * 5, ctypes.c_int),
            ("ssd_add_norm", [P(NormProblem)] + [vp] * 7, ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = argtypes, restype


# ---- checks ------------------------------------------------------------------

def _dtype(x: torch.Tensor, name: str) -> int:
    try:
        return _DTYPES[x.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {x.dtype} of {name} (float32 or bfloat16)") from None


def _need(t: Optional[torch.Tensor], name: str, shape, dtype, device, dense=True) -> Optional[int]:
    """The address of t after checking it (None for an absent tensor)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr()


def _lead(x: torch.Tensor, name: str):
    """The device of the call's first tensor, which must be a CUDA tensor."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return x.device


def _run_on(device: torch.device, stream):
    """A context in which `device` is current, and `stream` where it is given."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _raw_stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _nseq(seq_idx, nseq) -> int:
    if nseq is None:
        if seq_idx is not None:
            raise ValueError("nseq is required with seq_idx (the number of sequences per row)")
        return 1
    return int(nseq)


def _split(channels: int, splits: Optional[Sequence[int]]):
    if splits is None:
        return (channels, 0, 0)
    splits = tuple(int(n) for n in splits)
    if not 1 <= len(splits) <= 3 or min(splits) < 1 or sum(splits) != channels:
        raise ValueError(f"splits must be 1 to 3 positive channel counts that sum to {channels}")
    return splits + (0,) * (3 - len(splits))


def _outputs(lead, split, x, out, as_tuple):
    """The outputs' tensors (allocated, or checked) and their three addresses."""
    shapes = [torch.Size((*lead, n)) for n in split if n]
    if out is None:
        outs = tuple(torch.empty(s, dtype=x.dtype, device=x.device) for s in shapes)
        ptrs = [o.data_ptr() for o in outs]
    else:
        outs = tuple(out) if as_tuple else (out,)
        if len(outs) != len(shapes):
            raise ValueError(f"out must hold {len(shapes)} tensors")
        ptrs = [_need(o, f"out[{i}]", s, x.dtype, x.device) for i, (o, s) in enumerate(zip(outs, shapes))]
    return outs, ptrs + [None] * (3 - len(ptrs))


Outputs = Union[torch.Tensor, Tuple[torch.Tensor, ...]]


# ---- the short causal convolution ----------------------------------------------

def causal_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                init_states: Optional[torch.Tensor] = None, seq_idx: Optional[torch.Tensor] = None,
                nseq: Optional[int] = None, activation: Optional[str] = "silu",
                splits: Optional[Sequence[int]] = None, return_final_states: bool = True, out: Optional[Outputs] = None,
                final_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[Outputs, Optional[torch.Tensor]]:
    """The short causal convolution of every channel of x [b, T, C] with its own
    taps weight [C, W] fp32 (W = 2, 3 or 4), bias [C] fp32 and the activation
    ("silu" or None), restarted at every sequence of seq_idx [b, T] int32.

    Returns (y, final windows). With splits (up to three channel counts that sum
    to C) y is a tuple of tensors [b, T, splits[i]] in channel order, as ssd_fwd
    takes them; else one tensor [b, T, C]. Windows are the last W - 1 inputs of a
    sequence, [b, nseq, W-1, C] in x's dtype, oldest first: init_states come
    before each sequence's first token (zero when None), the final ones are None
    unless return_final_states."""
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("shapes: x [b,T,C], weight [C,W]")
    device, dtype = _lead(x, "x"), _dtype(x, "x")
    b, T, C = x.shape
    W, nseq = weight.shape[1], _nseq(seq_idx, nseq)
    if C > 1 and x.stride(2) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    split = _split(C, splits)
    windows = torch.Size((b, nseq, W - 1, C))
    ptrs = (x.data_ptr(), _need(weight, "weight", (C, W), torch.float32, device),
            _need(bias, "bias", (C,), torch.float32, device),
            _need(init_states, "init_states", windows, x.dtype, device),
            _need(seq_idx, "seq_idx", (b, T), torch.int32, device))
    p = ConvProblem(b, T, C, W, nseq, (x.stride(0), x.stride(1)), split, dtype, _activation(activation))
    with _run_on(device, stream):
        outs, outp = _outputs((b, T), split, x, out, splits is not None)
        final, finp = None, None
        if return_final_states:
            final = torch.empty(windows, dtype=x.dtype, device=device) if final_out is None else final_out
            finp = _need(final, "final_out", windows, x.dtype, device)
        st = _ssd.lib().ssd_causal_conv(ctypes.byref(p), *ptrs, *outp, finp, _raw_stream(device))
    _ssd._check(st, "ssd_causal_conv")
    return (outs if splits is not None else outs[0]), final


def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or None, not {name!r}")
    return _ACTIVATIONS[name]


def conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
              activation: Optional[str] = "silu", splits: Optional[Sequence[int]] = None,
              out: Optional[Outputs] = None, stream=None) -> Outputs:
    """One token of causal_conv for every batch row: x [b, C], with the window
    state [b, W-1, C] (x's dtype) updated in place. Returns y [b, C], or a tuple
    of [b, splits[i]] with splits."""
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("shapes: x [b,C], weight [C,W]")
    device, dtype = _lead(x, "x"), _dtype(x, "x")
    b, C = x.shape
    W = weight.shape[1]
    if C > 1 and x.stride(1) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    split = _split(C, splits)
    ptrs = (x.data_ptr(), _need(weight, "weight", (C, W), torch.float32, device),
            _need(bias, "bias", (C,), torch.float32, device), _need(state, "state", (b, W - 1, C), x.dtype, device))
    p = ConvProblem(b, 1, C, W, 1, (x.stride(0), 0), split, dtype, _activation(activation))
    with _run_on(device, stream):
        outs, outp = _outputs((b,), split, x, out, splits is not None)
        st = _ssd.lib().ssd_conv_step(ctypes.byref(p), *ptrs, *outp, _raw_stream(device))
    _ssd._check(st, "ssd_conv_step")
    return outs if splits is not None else outs[0]


# ---- the selective scan ----------------------------------------------------------

def _selective(u, dt, A, B, C, D, z, dt_bias, lead):
    """Checked addresses (u, dt, A, B, C, D, z, dt_bias), sizes and strides of a selective call."""
    k = len(lead)
    device = _lead(u, "u")
    _dtype(u, "u")
    ch = u.shape[-1]
    if A.dim() != 2 or B.dim() != k + 2:
        raise ValueError("shapes: A [channels,N], B and C [b,T,G,N] ([b,G,N] for a step)")
    N, G = A.shape[1], B.shape[-2]
    acts, bc = torch.Size((*lead, ch)), torch.Size((*lead, G, N))
    for t, name in ((B, "B"), (C, "C")):
        if t.dim() == k + 2 and G > 1 and t.stride(-2) != N:
            raise ValueError(f"the groups of {name} must be contiguous (stride N)")
    f32 = torch.float32
    ptrs = (_need(u, "u", acts, u.dtype, device, False), _need(dt, "dt", acts, u.dtype, device, False),
            _need(A, "A", (ch, N), f32, device), _need(B, "B", bc, u.dtype, device, False),
            _need(C, "C", bc, u.dtype, device, False), _need(D, "D", (ch,), f32, device),
            _need(z, "z", acts, u.dtype, device, False), _need(dt_bias, "dt_bias", (ch,), f32, device))
    strides = [(t.stride(0), t.stride(1) if k == 2 else 0) if t is not None else (0, 0) for t in (u, dt, z, B, C)]
    return ptrs, (ch, N, G), strides


def selective_scan(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                   init_states: Optional[torch.Tensor] = None, seq_idx: Optional[torch.Tensor] = None,
                   nseq: Optional[int] = None, return_final_states: bool = True, out: Optional[torch.Tensor] = None,
                   final_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The selective scan with a decay per channel and state:

        delta = softplus(dt + dt_bias),  h[n] <- exp(delta A[c, n]) h[n] + delta u B[n]
        y = (sum_n C[n] h[n] + D u) * silu(z)

    u, dt, z [b, T, channels], B, C [b, T, G, N] in one dtype (float32 or
    bfloat16), A [channels, N], D, dt_bias [channels] fp32. Returns y
    [b, T, channels] and the final states [b, nseq, N, channels] fp32 (None unless
    return_final_states); init_states and seq_idx as in ssd_fwd. dt_softplus=False
    takes dt + dt_bias as delta."""
    if u.dim() != 3:
        raise ValueError("u must be [b, T, channels]")
    b, T = u.shape[:2]
    ptrs, (ch, N, G), strides = _selective(u, dt, A, B, C, D, z, dt_bias, (b, T))
    nseq, device = _nseq(seq_idx, nseq), u.device
    states = torch.Size((b, nseq, N, ch))
    initp = _need(init_states, "init_states", states, torch.float32, device)
    idsp = _need(seq_idx, "seq_idx", (b, T), torch.int32, device)
    p = SelectiveProblem(b, T, ch, N, G, nseq, *strides, _DTYPES[u.dtype], int(bool(dt_softplus)))
    lib = _ssd.lib()
    with _run_on(device, stream):
        y = torch.empty((b, T, ch), dtype=u.dtype, device=device) if out is None else out
        yp = _need(y, "out", (b, T, ch), u.dtype, device)
        final, finp = None, None
        if return_final_states:
            final = torch.empty(states, dtype=torch.float32, device=device) if final_out is None else final_out
            finp = _need(final, "final_out", states, torch.float32, device)
        need = lib.ssd_selective_scan_workspace_bytes(ctypes.byref(p))
        if workspace is None and 0 < need < ctypes.c_size_t(-1).value:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        wsp = None if workspace is None else _need(workspace, "workspace", workspace.shape, workspace.dtype, device)
        size = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = lib.ssd_selective_scan(ctypes.byref(p), *ptrs, initp, idsp, yp, finp, wsp, size, _raw_stream(device))
    _ssd._check(st, "ssd_selective_scan")
    return y, final


def selective_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   state: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of selective_scan for every batch row: u, dt, z [b, channels],
    B, C [b, G, N], with the state [b, N, channels] fp32 updated in place.
    Returns y [b, channels]."""
    if u.dim() != 2:
        raise ValueError("u must be [b, channels]")
    b = u.shape[0]
    ptrs, (ch, N, G), strides = _selective(u, dt, A, B, C, D, z, dt_bias, (b,))
    device = u.device
    sp = _need(state, "state", (b, N, ch), torch.float32, device)
    p = SelectiveProblem(b, 1, ch, N, G, 1, *strides, _DTYPES[u.dtype], int(bool(dt_softplus)))
    with _run_on(device, stream):
        y = torch.empty((b, ch), dtype=u.dtype, device=device) if out is None else out
        yp = _need(y, "out", (b, ch), u.dtype, device)
        st = _ssd.lib().ssd_selective_step(ctypes.byref(p), *ptrs, sp, yp, _raw_stream(device))
    _ssd._check(st, "ssd_selective_step")
    return y


# ---- norms -------------------------------------------------------------------------

def _rows(x: torch.Tensor, name: str):
    """(batch, tokens) of a tensor [rows, channels] or [b, T, channels]."""
    if x.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows, channels] or [b, T, channels]")
    return (1, x.shape[0]) if x.dim() == 2 else (x.shape[0], x.shape[1])


def _row_strides(t: Optional[torch.Tensor]):
    if t is None:
        return (0, 0)
    return (0, t.stride(0)) if t.dim() == 2 else (t.stride(0), t.stride(1))


def gated_norm(x: torch.Tensor, weight: torch.Tensor, z: Optional[torch.Tensor] = None, ngroups: int = 1,
               eps: float = 1e-5, gate_first: bool = True, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """The root-mean-square norm over each of ngroups groups of channels, times
    weight [channels] fp32, of x * silu(z) (gate_first), or of x and times silu(z)
    afterwards; without z the plain norm. x and z [rows, channels] or
    [b, T, channels] in one dtype (float32 or bfloat16), which the result has too."""
    device, dtype = _lead(x, "x"), _dtype(x, "x")
    b, T = _rows(x, "x")
    ch = x.shape[-1]
    ptrs = (_need(x, "x", x.shape, x.dtype, device, False), _need(z, "z", x.shape, x.dtype, device, False),
            _need(weight, "weight", (ch,), torch.float32, device))
    p = NormProblem(b, T, ch, int(ngroups), _row_strides(x), _row_strides(z), dtype, dtype, eps, 1.0,
                    int(bool(gate_first)))
    with _run_on(device, stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=device) if out is None else out
        yp = _need(y, "out", x.shape, x.dtype, device)
        st = _ssd.lib().ssd_gated_norm(ctypes.byref(p), *ptrs, yp, _raw_stream(device))
    _ssd._check(st, "ssd_gated_norm")
    return y


def add_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
             scale: Union[float, torch.Tensor] = 1.0, eps: float = 1e-5,
             residual_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The norm before a block with the residual sum in front of it:

        r = residual + scale * x,   out = weight * r / sqrt(mean(r^2) + eps)

    Returns (out, r). x [rows, channels] or [b, T, channels], float32 or bfloat16;
    scale a number or an fp32 tensor [channels]; the residual is fp32 or of x's
    dtype (without one, r has residual_dtype, fp32 by default). The norm is taken of
    the unrounded sum. residual_out=residual updates a dense residual in place."""
    device, dtype = _lead(x, "x"), _dtype(x, "x")
    b, T = _rows(x, "x")
    ch = x.shape[-1]
    rdt = residual.dtype if residual is not None else (residual_dtype or torch.float32)
    if residual_dtype is not None and residual_dtype != rdt:
        raise TypeError(f"residual_dtype is {residual_dtype}, the residual {rdt}")
    if rdt not in (torch.float32, x.dtype):
        raise TypeError(f"the residual must be float32 or {x.dtype}, not {rdt}")
    per_channel = isinstance(scale, torch.Tensor)
    ptrs = (_need(x, "x", x.shape, x.dtype, device, False),
            _need(residual, "residual", x.shape, rdt, device, False),
            _need(weight, "weight", (ch,), torch.float32, device),
            _need(scale, "scale", (ch,), torch.float32, device) if per_channel else None)
    p = NormProblem(b, T, ch, 1, _row_strides(x), _row_strides(residual), dtype, _DTYPES[rdt], eps,
                    1.0 if per_channel else scale, 0)
    with _run_on(device, stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=device) if out is None else out
        r = torch.empty(x.shape, dtype=rdt, device=device) if residual_out is None else residual_out
        yp, rp = _need(y, "out", x.shape, x.dtype, device), _need(r, "residual_out", x.shape, rdt, device)
        st = _ssd.lib().ssd_add_norm(ctypes.byref(p), *ptrs, yp, rp, _raw_stream(device))
    _ssd._check(st, "ssd_add_norm")
    return y, r
