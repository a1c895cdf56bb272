"""The operators around the scan without a GPU: pins of their fp64 definitions,
and what the entry points refuse. The C functions are called with fake device
addresses only where a host check rejects the call first."""
import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_layer_chunked_b200 as ssd
from mamba_ssd_layer_chunked_b200 import block
import oracle
from oracle import block_oracle as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
BF16, F32 = ssd.ssd.SSD_DTYPE_BF16, ssd.ssd.SSD_DTYPE_F32


def FAKE(i):
    return 0x100000000 * (i + 1)  # far apart: no two fake tensors overlap


# --------------------------------------------------------------------------- #
# Pins of the definitions
# --------------------------------------------------------------------------- #

def test_conv_definition_on_a_small_example():
    x = np.array([1.0, 2.0, 3.0, 4.0]).reshape(1, 4, 1)
    w = np.array([[1.0, 10.0, 100.0]])  # the last tap meets the token itself
    y, final = ref.causal_conv(x, w, act=False)
    assert y.ravel().tolist() == [100.0, 210.0, 321.0, 432.0]
    assert final.ravel().tolist() == [3.0, 4.0]
    # a second sequence from the third token on, with an initial window
    ids = np.array([[0, 0, 1, 1]])
    init = np.array([[[[0.0], [0.0]], [[7.0], [8.0]]]])
    y, final = ref.causal_conv(x, w, init_states=init, seq_idx=ids, nseq=2, act=False)
    assert y.ravel().tolist() == [100.0, 210.0, 387.0, 438.0]
    assert final.ravel().tolist() == [1.0, 2.0, 3.0, 4.0]


def test_selective_definition_is_the_ssd_recurrence_for_a_decay_per_head():
    """With A constant over a head's channels and states, the selective scan of
    u is the SSD scan of X = delta u with log a = delta A."""
    rng = np.random.default_rng(3)
    b, T, H, P, N, G = 2, 9, 4, 3, 5, 2
    u = rng.normal(size=(b, T, H, P))
    dt = rng.normal(size=(b, T, H))
    A = -rng.uniform(0.5, 2.0, H)
    B, C = rng.normal(size=(b, T, G, N)), rng.normal(size=(b, T, G, N))
    D, h0 = rng.normal(size=H), rng.normal(size=(b, 2, H, N, P))
    ids = np.array([[0] * 4 + [1] * 5, [0] * 9])
    log_a, X = oracle.discretize(dt, A, u)
    Y, F = oracle.ssd_reference(X, log_a, B, C, None, h0, ids, nseq=2)
    Y = Y + D[:, None] * u
    rep = lambda v: np.repeat(v, P, axis=-1)  # noqa: E731
    y, final = ref.selective_scan(u.reshape(b, T, H * P), rep(dt), np.repeat(rep(A)[:, None], N, axis=1), B, C,
                                  D=rep(D), init_states=h0.transpose(0, 1, 3, 2, 4).reshape(b, 2, N, H * P),
                                  seq_idx=ids, nseq=2)
    assert np.allclose(y, Y.reshape(b, T, H * P), rtol=1e-12, atol=1e-12)
    assert np.allclose(final, F.transpose(0, 1, 3, 2, 4).reshape(b, 2, N, H * P), rtol=1e-12, atol=1e-12)


def test_norm_definitions():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    assert np.allclose(ref.gated_norm(x, np.ones(4), eps=0.0), x / 2.5)
    g = np.array([[3.0, 4.0, 6.0, 8.0]])
    assert np.allclose(ref.gated_norm(g, np.ones(4), ngroups=2, eps=0.0), g / np.sqrt([[12.5, 12.5, 50.0, 50.0]]))
    z = np.array([[0.0, 50.0, 50.0, 0.0]])  # silu: 0, 50, 50, 0
    assert np.allclose(ref.gated_norm(g, np.ones(4), z=z, eps=0.0), [[0.0, 0.8, 1.2, 0.0]] / np.sqrt(0.52))
    y, r = ref.add_norm(x, 2 * np.ones(4), residual=np.ones((1, 4)), scale=2.0, eps=0.0)
    assert r.tolist() == [[7.0, 9.0, 1.0, 1.0]] and np.allclose(y, 2 * r / np.sqrt(33.0))


# --------------------------------------------------------------------------- #
# Refusals of the C ABI
# --------------------------------------------------------------------------- #

def test_struct_sizes():
    assert ctypes.sizeof(block.ConvProblem) == 8 * 10 + 2 * 4
    assert ctypes.sizeof(block.SelectiveProblem) == 8 * 16 + 2 * 4
    assert ctypes.sizeof(block.NormProblem) == 8 * 8 + 6 * 4  # five 4-byte fields, padded


def _change(p, **kw):
    """Fields of a problem set; x_stride=(batch, token) and split=(a, b, c) set one field per element."""
    for k, v in kw.items():
        if k == "split":
            p.split0, p.split1, p.split2 = v
        elif k.endswith("_stride"):
            setattr(p, k[:-6] + "batch_stride", v[0])
            setattr(p, k[:-6] + "token_stride", v[1])
        else:
            assert k in dict(p._fields_)
            setattr(p, k, v)
    return p


def conv_problem(**kw):
    return _change(block.ConvProblem(2, 64, 96, 4, 1, 64 * 96, 96, 64, 16, 16, BF16, 1), **kw)


def conv(p, x=FAKE(0), weight=FAKE(1), bias=None, init=None, seq=None, out0=FAKE(2), out1=FAKE(3), out2=FAKE(4),
         final=None):
    return ssd.lib().ssd_causal_conv(None if p is None else ctypes.byref(p), x, weight, bias, init, seq, out0, out1,
                                     out2, final, None)


def step(p, x=FAKE(0), weight=FAKE(1), bias=None, state=FAKE(5), out0=FAKE(2), out1=FAKE(3), out2=FAKE(4)):
    return ssd.lib().ssd_conv_step(None if p is None else ctypes.byref(p), x, weight, bias, state, out0, out1, out2,
                                   None)


@pytest.mark.parametrize("field,value,expect", [
    ("batch", 0, INVALID), ("seqlen", 0, INVALID), ("channels", 0, INVALID), ("width", 0, INVALID),
    ("width", 1, UNSUPPORTED), ("width", 5, UNSUPPORTED), ("nseq", 0, INVALID), ("nseq", 2, INVALID),
    ("dtype", 7, INVALID), ("act", 2, INVALID), ("x_stride", (-1, 96), INVALID), ("x_stride", (0, 1 << 41), UNSUPPORTED),
    ("split", (96, 1, 0), INVALID), ("split", (0, 96, 0), INVALID), ("split", (64, 0, 32), INVALID),
    ("split", (128, -16, -16), INVALID), ("channels", 1 << 21, UNSUPPORTED), ("seqlen", (1 << 30) + 1, UNSUPPORTED),
    ("batch", 1 << 30, UNSUPPORTED)])
def test_conv_refuses_bad_problems(field, value, expect):
    assert conv(conv_problem(**{field: value})) == expect
    if field not in ("seqlen", "nseq") and (field, expect) != ("batch", UNSUPPORTED):
        assert step(conv_problem(**{field: value})) == expect


@pytest.mark.parametrize("arg", ["x", "weight", "out0", "out1", "out2"])
def test_conv_refuses_missing_pointers(arg):
    assert conv(conv_problem(), **{arg: None}) == INVALID
    assert step(conv_problem(), **{arg: None}) == INVALID


def test_conv_refuses_misaligned_overlapping_and_surplus_tensors():
    p = conv_problem()
    assert conv(None) == INVALID and step(None) == INVALID and step(p, state=None) == INVALID
    assert conv(p, x=FAKE(0) + 1) == INVALID and conv(p, weight=FAKE(1) + 2) == INVALID
    assert conv(p, seq=FAKE(6) + 2) == INVALID and step(p, state=FAKE(5) + 1) == INVALID
    # an output for a part that does not exist
    assert conv(conv_problem(split=(96, 0, 0))) == INVALID
    # outputs on the input, on each other, and final windows on the initial ones
    assert conv(p, out0=FAKE(0) + 4096) == INVALID
    assert conv(p, out1=FAKE(2) + 16) == INVALID
    assert conv(p, init=FAKE(6), final=FAKE(6)) == INVALID
    assert step(p, out0=FAKE(5)) == INVALID
    # the rows between a strided input's first and last token belong to it
    q = conv_problem(x_stride=(64 * 400, 400))
    assert conv(q, out0=FAKE(0) + 2 * 100) == INVALID


def selective_problem(**kw):
    p = block.SelectiveProblem(2, 64, 96, 16, 2, 1, *[64 * 96, 96] * 3, *[64 * 32, 32] * 2, BF16, 1)
    return _change(p, **kw)


def scan(p, u=FAKE(0), dt=FAKE(1), A=FAKE(2), B=FAKE(3), C=FAKE(4), D=None, z=None, bias=None, init=None, seq=None,
         y=FAKE(5), final=None):
    return ssd.lib().ssd_selective_scan(None if p is None else ctypes.byref(p), u, dt, A, B, C, D, z, bias, init, seq,
                                        y, final, None)


def scan_step(p, u=FAKE(0), dt=FAKE(1), A=FAKE(2), B=FAKE(3), C=FAKE(4), D=None, z=None, bias=None, state=FAKE(6),
              y=FAKE(5)):
    return ssd.lib().ssd_selective_step(None if p is None else ctypes.byref(p), u, dt, A, B, C, D, z, bias, state, y,
                                        None)


@pytest.mark.parametrize("field,value,expect", [
    ("batch", 0, INVALID), ("seqlen", 0, INVALID), ("channels", 0, INVALID), ("dstate", 0, INVALID),
    ("dstate", 257, UNSUPPORTED), ("ngroups", 0, INVALID), ("ngroups", 5, INVALID), ("nseq", 0, INVALID),
    ("nseq", 3, INVALID), ("dtype", 9, INVALID), ("channels", 1 << 21, UNSUPPORTED), ("u_stride", (-4, 1), INVALID),
    ("C_stride", (1 << 41, 0), UNSUPPORTED), ("seqlen", (1 << 30) + 1, UNSUPPORTED)])
def test_selective_refuses_bad_problems(field, value, expect):
    p = selective_problem(**{field: value})
    assert scan(p) == expect
    if field not in ("seqlen", "nseq"):
        assert scan_step(p) == expect


@pytest.mark.parametrize("arg", ["u", "dt", "A", "B", "C", "y"])
def test_selective_refuses_missing_pointers(arg):
    assert scan(selective_problem(), **{arg: None}) == INVALID
    assert scan_step(selective_problem(), **{arg: None}) == INVALID


def test_selective_refuses_misaligned_and_overlapping_tensors():
    p = selective_problem()
    assert scan(None) == INVALID and scan_step(None) == INVALID and scan_step(p, state=None) == INVALID
    assert scan(p, u=FAKE(0) + 1) == INVALID and scan(p, A=FAKE(2) + 2) == INVALID
    assert scan(p, seq=FAKE(7) + 1) == INVALID and scan_step(p, state=FAKE(6) + 2) == INVALID
    assert scan(p, y=FAKE(0)) == INVALID and scan(p, z=FAKE(7), y=FAKE(7) + 64) == INVALID
    assert scan(p, init=FAKE(7), final=FAKE(7)) == INVALID
    assert scan_step(p, y=FAKE(6)) == INVALID and scan_step(p, D=FAKE(6)) == INVALID


def norm_problem(**kw):
    return _change(block.NormProblem(2, 64, 96, 1, *[64 * 96, 96] * 2, BF16, F32, 1e-5, 1.0, 1), **kw)


def gnorm(p, x=FAKE(0), z=FAKE(1), w=FAKE(2), out=FAKE(3)):
    return ssd.lib().ssd_gated_norm(None if p is None else ctypes.byref(p), x, z, w, out, None)


def anorm(p, x=FAKE(0), r=FAKE(1), w=FAKE(2), s=None, out=FAKE(3), rout=FAKE(4)):
    return ssd.lib().ssd_add_norm(None if p is None else ctypes.byref(p), x, r, w, s, out, rout, None)


@pytest.mark.parametrize("field,value,expect", [
    ("batch", 0, INVALID), ("seqlen", -1, INVALID), ("channels", 0, INVALID), ("ngroups", 0, INVALID),
    ("ngroups", 7, INVALID), ("dtype", 2, INVALID), ("eps", -1.0, INVALID), ("eps", float("nan"), INVALID),
    ("eps", float("inf"), INVALID), ("channels", 32769, UNSUPPORTED), ("x_stride", (0, -1), INVALID),
    ("z_stride", (0, -1), INVALID), ("seqlen", (1 << 30) + 1, UNSUPPORTED)])
def test_norms_refuse_bad_problems(field, value, expect):
    assert gnorm(norm_problem(**{field: value})) == expect
    assert anorm(norm_problem(**{field: value})) == expect


def test_norms_refuse_bad_tensors():
    p = norm_problem()
    assert gnorm(None) == INVALID and anorm(None) == INVALID
    for arg in ("x", "w", "out"):
        assert gnorm(p, **{arg: None}) == INVALID and anorm(p, **{arg: None}) == INVALID
    assert anorm(p, rout=None) == INVALID
    assert gnorm(p, z=FAKE(1) + 1) == INVALID and anorm(p, r=FAKE(1) + 2) == INVALID
    assert gnorm(p, out=FAKE(0)) == INVALID and gnorm(p, out=FAKE(1) + 32) == INVALID
    assert anorm(p, out=FAKE(4)) == INVALID and anorm(p, s=FAKE(3)) == INVALID
    assert anorm(norm_problem(ngroups=2)) == INVALID
    assert anorm(norm_problem(dtype=F32, residual_dtype=BF16)) == INVALID
    # the residual in place only where it is dense
    assert anorm(norm_problem(z_stride=(64 * 100, 100)), rout=FAKE(1)) == INVALID
    assert anorm(p, rout=FAKE(1) + 4) == INVALID


# --------------------------------------------------------------------------- #
# Refusals of the Python binding
# --------------------------------------------------------------------------- #

def test_binding_refuses_cpu_tensors_and_bad_shapes():
    x, w = torch.zeros(2, 8, 32), torch.zeros(32, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.causal_conv(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.conv_step(x[:, 0], torch.zeros(2, 3, 32), w)
    with pytest.raises(ValueError, match="shapes"):
        ssd.causal_conv(x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.gated_norm(x, torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.add_norm(x, torch.zeros(32))
    A, B = torch.zeros(32, 4), torch.zeros(2, 8, 1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError, match="channels"):
        ssd.selective_step(x, x, A, B, B, torch.zeros(2, 4, 32))


def test_binding_helpers_refuse():
    cpu = torch.device("cpu")
    t = torch.zeros(4, 6)
    assert block._need(None, "t", (4, 6), torch.float32, cpu) is None
    with pytest.raises(TypeError):
        block._need(t, "t", (4, 6), torch.bfloat16, cpu)
    with pytest.raises(ValueError, match="shape"):
        block._need(t, "t", (4, 7), torch.float32, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        block._need(t[:, :3], "t", (4, 3), torch.float32, cpu)
    with pytest.raises(ValueError, match="last dimension"):
        block._need(t.t(), "t", (6, 4), torch.float32, cpu, dense=False)
    assert block._need(t[:, :3], "t", (4, 3), torch.float32, cpu, dense=False) == t.data_ptr()
    with pytest.raises(ValueError, match="is on"):
        block._need(t, "t", (4, 6), torch.float32, torch.device("cuda", 0))
    for bad in ([], [3, 4], [10, 0], [1, 2, 3, 4], [11, -1]):
        with pytest.raises(ValueError, match="splits"):
            block._split(10, bad)
    assert block._split(10, [7, 3]) == (7, 3, 0) and block._split(10, None) == (10, 0, 0)
    with pytest.raises(ValueError, match="nseq"):
        block._nseq(t, None)
    with pytest.raises(ValueError, match="activation"):
        block._activation("gelu")
    with pytest.raises(TypeError, match="dtype"):
        block._dtype(t.half(), "x")
