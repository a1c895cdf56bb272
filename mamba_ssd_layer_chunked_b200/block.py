"""Python binding of the operators around the scan (see include/ssd.h): the
short causal convolution, the selective scan with a decay per channel and state,
and the norms of a block. Argument marshalling only, as in ssd.py.

Activations may be slices of a projection's output: their last dimension is
contiguous, the others may have any stride. Every call runs on the device of its
tensors and on that device's current torch stream, or on ``stream``; outputs are
allocated on the stream the call runs on. Inputs must be ready on that stream;
the memory of inputs and of given outputs is kept until it is done with them.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from . import ssd as _ssd

_DTYPES = {torch.float32: _ssd.SSD_DTYPE_F32, torch.bfloat16: _ssd.SSD_DTYPE_BF16}
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_i64 = ctypes.c_int64
_fn = None  # the loaded library


class ConvProblem(ctypes.Structure):
    """Mirror of ssd_conv_problem (its small arrays as one field per element)."""

    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("width", _i64), ("nseq", _i64),
                ("x_batch_stride", _i64), ("x_token_stride", _i64), ("split0", _i64), ("split1", _i64),
                ("split2", _i64), ("dtype", ctypes.c_int), ("act", ctypes.c_int)]


class SelectiveProblem(ctypes.Structure):
    """Mirror of ssd_selective_problem."""

    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("dstate", _i64), ("ngroups", _i64),
                ("nseq", _i64), ("u_batch_stride", _i64), ("u_token_stride", _i64), ("dt_batch_stride", _i64),
                ("dt_token_stride", _i64), ("z_batch_stride", _i64), ("z_token_stride", _i64),
                ("B_batch_stride", _i64), ("B_token_stride", _i64), ("C_batch_stride", _i64),
                ("C_token_stride", _i64), ("dtype", ctypes.c_int), ("dt_softplus", ctypes.c_int32)]


class NormProblem(ctypes.Structure):
    """Mirror of ssd_norm_problem."""

    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("ngroups", _i64),
                ("x_batch_stride", _i64), ("x_token_stride", _i64), ("z_batch_stride", _i64),
                ("z_token_stride", _i64), ("dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("alpha", ctypes.c_float), ("gate_first", ctypes.c_int32)]


def declare(lib):
    """Take the loaded library, and declare the argument types of the C functions this module calls."""
    global _fn
    _fn = lib
    vp, P = ctypes.c_void_p, ctypes.POINTER
    for name, argtypes, restype in (
            ("ssd_causal_conv", [P(ConvProblem)] + [vp] * 10, ctypes.c_int),
            ("ssd_conv_step", [P(ConvProblem)] + [vp] * 8, ctypes.c_int),
            ("ssd_selective_scan", [P(SelectiveProblem)] + [vp] * 13, ctypes.c_int),
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
    if (t.dtype is dtype and t.shape == shape and t.device == device
            and (t.is_contiguous() or (not dense and t.stride(-1) == 1))):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr()


# torch's own calls behind the public ones, which cost several times as much per call; a torch built without
# CUDA has neither, and no tensor that would reach them.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(x: torch.Tensor, stream) -> bool:
    """Whether a call on x has to change the current device or stream first."""
    return stream is not None or not x.is_cuda or x.get_device() != _current_device()


def _run_on(stream, x: torch.Tensor, *others):
    """A context in which x's device is current, and `stream` where it is given:
    the call's tensors, given outputs among them (tensors or tuples of tensors),
    are then recorded as used on it, so that their memory is not reused before it
    is done."""
    if not x.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if stream is None:
        return torch.cuda.device(x.device)
    if stream.device != x.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {x.device}")
    for t in (x, *others):
        for v in t if isinstance(t, (tuple, list)) else (t,):
            if isinstance(v, torch.Tensor) and v.is_cuda:
                v.record_stream(stream)
    return torch.cuda.stream(stream)


def _like(x: torch.Tensor) -> torch.Tensor:
    """A dense tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _nseq(seq_idx, nseq) -> int:
    if nseq is None:
        if seq_idx is not None:
            raise ValueError("nseq is required with seq_idx (the number of sequences per row)")
        return 1
    return int(nseq)


def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or None, not {name!r}")
    return _ACTIVATIONS[name]


def _split(channels: int, splits: Optional[Sequence[int]]):
    if splits is None:
        return (channels, 0, 0)
    splits = tuple(int(n) for n in splits)
    if not 1 <= len(splits) <= 3 or min(splits) < 1 or sum(splits) != channels:
        raise ValueError(f"splits must be 1 to 3 positive channel counts that sum to {channels}")
    return splits + (0,) * (3 - len(splits))


def _outputs(lead, split, x, out, as_tuple):
    """The outputs' tensors (allocated, or checked) and their three addresses."""
    if out is None:
        outs = [x.new_empty((*lead, n)) for n in split if n] if as_tuple else [_like(x)]
        ptrs = [o.data_ptr() for o in outs]
    else:
        outs = tuple(out) if as_tuple else (out,)
        shapes = [(*lead, n) for n in split if n]
        if len(outs) != len(shapes):
            raise ValueError(f"out must hold {len(shapes)} tensors")
        ptrs = [_need(o, f"out[{i}]", s, x.dtype, x.device) for i, (o, s) in enumerate(zip(outs, shapes))]
    while len(ptrs) < 3:
        ptrs.append(None)
    return (tuple(outs) if as_tuple else outs[0]), ptrs


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
    if _elsewhere(x, stream):
        with _run_on(stream, x, weight, bias, init_states, seq_idx, out, final_out):
            return causal_conv(x, weight, bias, init_states, seq_idx, nseq, activation, splits, return_final_states,
                               out, final_out)
    device, dtype = x.device, x.dtype
    b, T, C = x.shape
    W, nseq = weight.shape[1], _nseq(seq_idx, nseq)
    split, windows = _split(C, splits), (b, nseq, W - 1, C)
    xp = _need(x, "x", x.shape, dtype, device, False)
    p = ConvProblem(b, T, C, W, nseq, x.stride(0), x.stride(1), *split, _dtype(x, "x"), _activation(activation))
    ptrs = (_need(weight, "weight", (C, W), torch.float32, device), _need(bias, "bias", (C,), torch.float32, device),
            _need(init_states, "init_states", windows, dtype, device),
            _need(seq_idx, "seq_idx", (b, T), torch.int32, device))
    outs, outp = _outputs((b, T), split, x, out, splits is not None)
    final, finp = None, None
    if return_final_states:
        final = x.new_empty(windows) if final_out is None else final_out
        finp = _need(final, "final_out", windows, dtype, device)
    _ssd._check(_fn.ssd_causal_conv(ctypes.byref(p), xp, *ptrs, *outp, finp, _raw_stream(device.index)),
                "ssd_causal_conv")
    return outs, final


def conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
              activation: Optional[str] = "silu", splits: Optional[Sequence[int]] = None,
              out: Optional[Outputs] = None, stream=None) -> Outputs:
    """One token of causal_conv for every batch row: x [b, C], with the window
    state [b, W-1, C] (x's dtype) updated in place. Returns y [b, C], or a tuple
    of [b, splits[i]] with splits."""
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("shapes: x [b,C], weight [C,W]")
    if _elsewhere(x, stream):
        with _run_on(stream, x, state, weight, bias, out):
            return conv_step(x, state, weight, bias, activation, splits, out)
    device, dtype = x.device, x.dtype
    b, C = x.shape
    W = weight.shape[1]
    split = _split(C, splits)
    xp = _need(x, "x", x.shape, dtype, device, False)
    p = ConvProblem(b, 1, C, W, 1, x.stride(0), 0, *split, _dtype(x, "x"), _activation(activation))
    ptrs = (_need(weight, "weight", (C, W), torch.float32, device), _need(bias, "bias", (C,), torch.float32, device),
            _need(state, "state", (b, W - 1, C), dtype, device))
    outs, outp = _outputs((b,), split, x, out, splits is not None)
    _ssd._check(_fn.ssd_conv_step(ctypes.byref(p), xp, *ptrs, *outp, _raw_stream(device.index)), "ssd_conv_step")
    return outs


# ---- the selective scan ----------------------------------------------------------

def _selective(u, dt, A, B, C, D, z, dt_bias):
    """Checked addresses (u, dt, A, B, C, D, z, dt_bias), sizes and strides of a selective call."""
    dtype, device, acts = u.dtype, u.device, u.shape
    k, ch = len(acts) - 1, acts[-1]
    if A.dim() != 2 or B.dim() != k + 2:
        raise ValueError("shapes: A [channels,N], B and C [b,T,G,N] ([b,G,N] for a step)")
    N, G = A.shape[1], B.shape[-2]
    bc, f32 = (*acts[:-1], G, N), torch.float32
    ptrs = (_need(u, "u", acts, dtype, device, False), _need(dt, "dt", acts, dtype, device, False),
            _need(A, "A", (ch, N), f32, device), _need(B, "B", bc, dtype, device, False),
            _need(C, "C", bc, dtype, device, False), _need(D, "D", (ch,), f32, device),
            _need(z, "z", acts, dtype, device, False), _need(dt_bias, "dt_bias", (ch,), f32, device))
    if G > 1 and (B.stride(-2) != N or C.stride(-2) != N):
        raise ValueError("the groups of B and of C must be contiguous (stride N)")
    strides = []
    for t in (u, dt, z, B, C):
        if t is None:
            strides += (0, 0)
        else:
            strides += (t.stride(0), t.stride(1) if k == 2 else 0)
    return ptrs, ch, N, G, strides


def selective_scan(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                   init_states: Optional[torch.Tensor] = None, seq_idx: Optional[torch.Tensor] = None,
                   nseq: Optional[int] = None, return_final_states: bool = True, out: Optional[torch.Tensor] = None,
                   final_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
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
    if _elsewhere(u, stream):
        with _run_on(stream, u, dt, A, B, C, D, z, dt_bias, init_states, seq_idx, out, final_out):
            return selective_scan(u, dt, A, B, C, D, z, dt_bias, dt_softplus, init_states, seq_idx, nseq,
                                  return_final_states, out, final_out)
    dtype = _dtype(u, "u")
    ptrs, ch, N, G, strides = _selective(u, dt, A, B, C, D, z, dt_bias)
    (b, T, _), device, nseq = u.shape, u.device, _nseq(seq_idx, nseq)
    states = (b, nseq, N, ch)
    initp = _need(init_states, "init_states", states, torch.float32, device)
    idsp = _need(seq_idx, "seq_idx", (b, T), torch.int32, device)
    p = ctypes.byref(SelectiveProblem(b, T, ch, N, G, nseq, *strides, dtype, 1 if dt_softplus else 0))
    y = _like(u) if out is None else out
    yp = y.data_ptr() if out is None else _need(y, "out", u.shape, u.dtype, device)
    final, finp = None, None
    if return_final_states:
        final = u.new_empty(states, dtype=torch.float32) if final_out is None else final_out
        finp = _need(final, "final_out", states, torch.float32, device)
    _ssd._check(_fn.ssd_selective_scan(p, *ptrs, initp, idsp, yp, finp, _raw_stream(device.index)),
                "ssd_selective_scan")
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
    if _elsewhere(u, stream):
        with _run_on(stream, u, dt, A, B, C, state, D, z, dt_bias, out):
            return selective_step(u, dt, A, B, C, state, D, z, dt_bias, dt_softplus, out)
    dtype = _dtype(u, "u")
    ptrs, ch, N, G, strides = _selective(u, dt, A, B, C, D, z, dt_bias)
    b, device = u.shape[0], u.device
    sp = _need(state, "state", (b, N, ch), torch.float32, device)
    p = SelectiveProblem(b, 1, ch, N, G, 1, *strides, dtype, 1 if dt_softplus else 0)
    y = _like(u) if out is None else out
    yp = y.data_ptr() if out is None else _need(y, "out", u.shape, u.dtype, device)
    _ssd._check(_fn.ssd_selective_step(ctypes.byref(p), *ptrs, sp, yp, _raw_stream(device.index)),
                "ssd_selective_step")
    return y


# ---- norms -------------------------------------------------------------------------

def _rows(x: torch.Tensor, z: Optional[torch.Tensor]):
    """batch, tokens, channels, and the two strides of x and of z (of x's shape, or None)."""
    if x.dim() == 3:
        zs = (z.stride(0), z.stride(1)) if z is not None else (0, 0)
        return (*x.shape, x.stride(0), x.stride(1)), zs
    if x.dim() == 2:
        zs = (0, z.stride(0)) if z is not None else (0, 0)
        return (1, *x.shape, 0, x.stride(0)), zs
    raise ValueError("x must be [rows, channels] or [b, T, channels]")


def gated_norm(x: torch.Tensor, weight: torch.Tensor, z: Optional[torch.Tensor] = None, ngroups: int = 1,
               eps: float = 1e-5, gate_first: bool = True, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """The root-mean-square norm over each of ngroups groups of channels, times
    weight [channels] fp32, of x * silu(z) (gate_first), or of x and times silu(z)
    afterwards; without z the plain norm. x and z [rows, channels] or
    [b, T, channels] in one dtype (float32 or bfloat16), which the result has too."""
    if _elsewhere(x, stream):
        with _run_on(stream, x, weight, z, out):
            return gated_norm(x, weight, z, ngroups, eps, gate_first, out)
    dtype, device, shape = x.dtype, x.device, x.shape
    xp, zp = _need(x, "x", shape, dtype, device, False), _need(z, "z", shape, dtype, device, False)
    (b, T, ch, xs0, xs1), zs = _rows(x, z)
    wp = _need(weight, "weight", (ch,), torch.float32, device)
    code = _dtype(x, "x")
    p = NormProblem(b, T, ch, int(ngroups), xs0, xs1, *zs, code, code, eps, 1.0, 1 if gate_first else 0)
    y = _like(x) if out is None else out
    yp = y.data_ptr() if out is None else _need(y, "out", shape, dtype, device)
    _ssd._check(_fn.ssd_gated_norm(ctypes.byref(p), xp, zp, wp, yp, _raw_stream(device.index)), "ssd_gated_norm")
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
    if _elsewhere(x, stream):
        with _run_on(stream, x, weight, residual, scale, out, residual_out):
            return add_norm(x, weight, residual, scale, eps, residual_dtype, out, residual_out)
    dtype, device, shape, code = x.dtype, x.device, x.shape, _dtype(x, "x")
    rdt = residual.dtype if residual is not None else (residual_dtype or torch.float32)
    if residual_dtype is not None and residual_dtype != rdt:
        raise TypeError(f"residual_dtype is {residual_dtype}, the residual {rdt}")
    if rdt is not torch.float32 and rdt is not dtype:
        raise TypeError(f"the residual must be float32 or {dtype}, not {rdt}")
    xp, rp = _need(x, "x", shape, dtype, device, False), _need(residual, "residual", shape, rdt, device, False)
    (b, T, ch, xs0, xs1), rs = _rows(x, residual)
    wp, sp = _need(weight, "weight", (ch,), torch.float32, device), None
    per_channel = isinstance(scale, torch.Tensor)  # not rebound: the tensor lives until the launch
    if per_channel:
        sp = _need(scale, "scale", (ch,), torch.float32, device)
    p = NormProblem(b, T, ch, 1, xs0, xs1, *rs, code, _DTYPES[rdt], eps, 1.0 if per_channel else scale, 0)
    y = _like(x) if out is None else out
    yp = y.data_ptr() if out is None else _need(y, "out", shape, dtype, device)
    if residual_out is not None:
        r = residual_out
    else:
        r = _like(residual) if residual is not None else x.new_empty(shape, dtype=rdt)
    rop = r.data_ptr() if residual_out is None else _need(r, "residual_out", shape, rdt, device)
    _ssd._check(_fn.ssd_add_norm(ctypes.byref(p), xp, rp, wp, sp, yp, rop, _raw_stream(device.index)), "ssd_add_norm")
    return y, r
