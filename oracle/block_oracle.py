"""fp64 definitions of the operators around the scan (test infrastructure only):
the short causal convolution, the selective scan with a decay per channel and
state, the gated norm and the norm before a block. One loop over tokens each,
nothing shared with the product.

``selective_scan`` also carries a bound for a 32-bit evaluation of itself: per
step, the rounding of exp(delta A), of delta and of each product and sum are
relative errors of a few 2^-24 of the terms' absolute values, so with
    q_t = a_t q_{t-1} + |delta u B|   (the state of the absolute values)
    m_t = a_t m_{t-1} + q_t           (all earlier steps' q, decayed to t)
the state is off by at most a small multiple of 2^-24 m_t. (A relative error r of
delta moves a = exp(-x) by x a r <= r / e, so it needs no term of its own.)
"""
from __future__ import annotations

import numpy as np


def silu(v):
    v = np.asarray(v, dtype=np.float64)
    return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(np.asarray(v, dtype=np.float64), 0.0)


def _ids(seq_idx, b, T):
    return np.zeros((b, T), dtype=np.int64) if seq_idx is None else np.asarray(seq_idx, dtype=np.int64)


def causal_conv(x, weight, bias=None, init_states=None, seq_idx=None, nseq=1, act=True):
    """(y [b, T, C], final windows [b, nseq, W-1, C])."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    b, T, C = x.shape
    W = weight.shape[1]
    ids = _ids(seq_idx, b, T)
    final = np.zeros((b, nseq, W - 1, C)) if init_states is None else np.array(init_states, np.float64)
    y = np.zeros_like(x)
    for r in range(b):
        for t in range(T):
            s = ids[r, t]
            seen = np.concatenate([final[r, s], x[r, t][None]])  # W inputs, oldest first
            y[r, t] = (seen * weight.T).sum(0)
            final[r, s] = seen[1:]
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return (silu(y) if act else y), final


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, init_states=None, seq_idx=None,
                   nseq=1, bounds=False):
    """(y [b, T, c], final states [b, nseq, N, c]), and with bounds=True the two
    multiples of 2^-24 (before the output's own rounding) described above."""
    f = lambda v: np.asarray(v, np.float64)  # noqa: E731
    u, A, B, C = f(u), f(A), f(B), f(C)
    b, T, c = u.shape
    N, G = A.shape[1], B.shape[2]
    delta = f(dt) + (0.0 if dt_bias is None else f(dt_bias))
    if dt_softplus:
        delta = softplus(delta)
    Bc = np.repeat(B, c // G, axis=2).transpose(0, 1, 3, 2)  # [b, T, N, c]
    Cc = np.repeat(C, c // G, axis=2).transpose(0, 1, 3, 2)
    ids = _ids(seq_idx, b, T)
    final = np.zeros((b, nseq, N, c)) if init_states is None else np.array(init_states, np.float64)
    q, m = np.abs(final), np.zeros_like(final)
    y, ybound = np.zeros_like(u), np.zeros_like(u)
    for r in range(b):
        for t in range(T):
            s = ids[r, t]
            a = np.exp(delta[r, t] * A.T)
            v = (delta[r, t] * u[r, t]) * Bc[r, t]
            final[r, s] = a * final[r, s] + v
            q[r, s] = a * q[r, s] + np.abs(v)
            m[r, s] = a * m[r, s] + q[r, s]
            y[r, t] = (Cc[r, t] * final[r, s]).sum(0)
            ybound[r, t] = (np.abs(Cc[r, t]) * m[r, s]).sum(0)
    if D is not None:
        y += f(D) * u
        ybound += np.abs(f(D) * u)
    if z is not None:
        y *= silu(z)
        ybound = ybound * np.abs(silu(z)) + np.abs(y)
    return (y, final, ybound, m) if bounds else (y, final)


def gated_norm(x, weight, z=None, ngroups=1, eps=1e-5, gate_first=True):
    x = np.asarray(x, np.float64)
    if z is not None and gate_first:
        x = x * silu(z)
    g = x.reshape(*x.shape[:-1], ngroups, -1)
    g = g / np.sqrt((g * g).mean(-1, keepdims=True) + eps)
    y = g.reshape(x.shape) * np.asarray(weight, np.float64)
    return y * silu(z) if z is not None and not gate_first else y


def add_norm(x, weight, residual=None, scale=1.0, eps=1e-5):
    r = np.asarray(x, np.float64) * np.asarray(scale, np.float64)
    if residual is not None:
        r = r + np.asarray(residual, np.float64)
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64), r
