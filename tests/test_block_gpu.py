"""The operators around the scan on the GPU against their fp64 definitions
(oracle.block_oracle), alone and as a block runs them.

Tolerances, elementwise. An output in bf16 is rounded once: 2^-8 of its value (half
a step of torch.finfo). What comes before is fp32: a few roundings of 2^-24 of
the terms' absolute sum. ``FP32`` = 2^-20 covers 16 such roundings: a convolution
has W + 1 products and sums, a gate's exponential and division fewer than 8.
silu turns an error e of its argument v into at most (1 + |v|) e, and its
exponential, whose argument is rounded, has a relative error of (1 + |v|) 2^-24:
hence the factors 1 + |v|. The selective scan's bound is the oracle's multiple
of 2^-24; per step it counts the rounding of the product delta A (1, and x e^-x <= 1),
of A log2 e (1), of delta (softplus: 4), the hardware exponential (4) and the
multiply-adds (4): FP32 again.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_layer_chunked_b200 as ssd
import oracle
from oracle import block_oracle as ref
from tests.gpu_util import assert_close

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -20
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(rng, *shape, dtype="f32", scale=1.0, shift=0.0):
    """A CPU tensor in the dtype, and so the values that both sides see."""
    return torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32)).to(DT[dtype])


def cuda(t):
    return None if t is None else t.cuda()


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, bound, dtype, what):
    """|got - want| <= half a step of the output's type + bound, everywhere."""
    got = num(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), what
    lim = HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7) + bound + 1e-37
    over = np.abs(got - want) - lim
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what} at {i}: {got[i]!r} for {want[i]!r}, off by {abs(got[i] - want[i]):.3e} > {lim[i]:.3e}"


def sliced(t, before, after):
    """The same values as a slice of a wider tensor on the GPU (its neighbours are NaN)."""
    wide = torch.full((*t.shape[:-1], before + t.shape[-1] + after), float("nan"), dtype=t.dtype, device="cuda")
    v = wide[..., before:before + t.shape[-1]]
    v.copy_(t)
    return v


def ids_of(lengths, T):
    """seq_idx rows from lists of sequence lengths (0: an id that does not occur)."""
    rows = [np.repeat(np.arange(len(l), dtype=np.int32), l) for l in lengths]
    assert all(r.shape == (T,) for r in rows)
    return torch.from_numpy(np.stack(rows))


# --------------------------------------------------------------------------- #
# The short convolution
# --------------------------------------------------------------------------- #

# (b, T, C, W, dtype, lengths per row, nseq, splits, (before, after) of the slice, bias, act)
CONV = {
    "one_token": (1, 1, 16, 4, "bf16", None, 1, None, (0, 0), True, "silu"),
    "one_channel": (2, 5, 1, 4, "f32", None, 1, None, (0, 0), False, None),
    "shorter_than_window": (3, 2, 24, 4, "f32", None, 1, None, (0, 0), True, "silu"),
    "w2": (2, 70, 40, 2, "bf16", None, 1, [24, 8, 8], (8, 16), True, "silu"),
    "w3_f32": (2, 65, 36, 3, "f32", None, 1, [20, 16], (4, 8), False, "silu"),
    "odd_channels": (2, 33, 37, 4, "bf16", None, 1, [30, 4, 3], (1, 2), True, "silu"),
    "even_channels": (2, 41, 54, 4, "bf16", None, 1, [50, 2, 2], (2, 4), True, None),
    "odd_channels_f32": (1, 33, 7, 3, "f32", None, 1, None, (3, 0), True, "silu"),
    "tile_edges": (2, 129, 64, 4, "bf16", None, 1, None, (0, 0), True, "silu"),
    "packed": (2, 100, 48, 4, "bf16", [[40, 60], [1, 99]], 2, [16, 16, 16], (16, 8), True, "silu"),
    "packed_short": (2, 40, 16, 4, "f32", [[1, 1, 1, 2, 3, 32], [8, 8, 8, 7, 1, 8]], 6, None, (0, 0), True, "silu"),
    "packed_absent": (2, 34, 20, 3, "bf16", [[0, 10, 0, 0, 24, 0], [34, 0, 0, 0, 0, 0]], 6, None, (0, 0), True, None),
    "packed_cut_at_tiles": (1, 97, 9, 4, "bf16", [[32, 32, 1, 31, 1]], 7, None, (0, 0), False, "silu"),
}


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("name", sorted(CONV))
def test_causal_conv(name, init):
    b, T, C, W, dt, lengths, nseq, splits, pad, has_bias, act = CONV[name]
    rng = np.random.default_rng(len(name) + 100 * init)
    x, w = rand(rng, b, T, C, dtype=dt), rand(rng, C, W, scale=0.7)
    bias = rand(rng, C) if has_bias else None
    h0 = rand(rng, b, nseq, W - 1, C, dtype=dt) if init else None
    ids = None if lengths is None else ids_of(lengths, T)
    want, wfinal = ref.causal_conv(num(x), num(w), num(bias), num(h0), ids, nseq, act == "silu")
    size, _ = ref.causal_conv(np.abs(num(x)), np.abs(num(w)), None if bias is None else np.abs(num(bias)),
                              None if h0 is None else np.abs(num(h0)), ids, nseq, False)
    y, final = ssd.causal_conv(sliced(x, *pad), cuda(w), cuda(bias), init_states=cuda(h0), seq_idx=cuda(ids),
                               nseq=nseq, activation=act, splits=splits)
    y = torch.cat(y, -1) if splits else y
    close(y, want, FP32 * size * (1 + size if act else 1), dt, "y")
    assert np.array_equal(num(final), wfinal)  # windows are copies of inputs


@pytest.mark.parametrize("C,W,dt,splits,pad", [(48, 4, "bf16", [16, 16, 16], (8, 8)), (37, 4, "bf16", None, (0, 1)),
                                               (20, 3, "f32", [12, 8], (4, 0)), (5, 2, "f32", None, (1, 1)),
                                               (54, 2, "bf16", [50, 4], (2, 2))])
def test_conv_steps_continue_a_prompt(C, W, dt, splits, pad):
    """A prompt, then single tokens from its final windows: one prompt of all of them."""
    b, T, T0 = 3, 19, 12
    rng = np.random.default_rng(C)
    x, w, bias = rand(rng, b, T, C, dtype=dt), rand(rng, C, W, scale=0.7), rand(rng, C)
    want, wfinal = ref.causal_conv(num(x), num(w), num(bias))
    size, _ = ref.causal_conv(np.abs(num(x)), np.abs(num(w)), np.abs(num(bias)), act=False)
    y0, final = ssd.causal_conv(x[:, :T0].cuda(), cuda(w), cuda(bias))
    state, ys = final[:, 0].contiguous(), [y0]
    for t in range(T0, T):
        y = ssd.conv_step(sliced(x[:, t], *pad), state, cuda(w), cuda(bias), splits=splits)
        ys.append((torch.cat(y, -1) if splits else y)[:, None])
    close(torch.cat(ys, 1), want, FP32 * size * (1 + size), dt, "y")
    assert np.array_equal(num(state), wfinal[:, 0])


def test_conv_takes_rows_more_than_2_31_elements_apart():
    """Offsets of a long strided input pass 32 bits: three tokens, 2^30 + 8 elements apart."""
    stride, C = (1 << 30) + 8, 16
    big = torch.empty(2 * stride + C, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, 3, C), (0, stride, 1))
    rng = np.random.default_rng(5)
    v, w = rand(rng, 1, 3, C, dtype="bf16"), rand(rng, C, 4)
    x.copy_(v)
    want, wfinal = ref.causal_conv(num(v), num(w), act=False)
    size, _ = ref.causal_conv(np.abs(num(v)), np.abs(num(w)), act=False)
    y, final = ssd.causal_conv(x, cuda(w), activation=None)
    close(y, want, FP32 * size, "bf16", "y")
    assert np.array_equal(num(final), wfinal)
    z = ssd.gated_norm(x, torch.ones(C, device="cuda"))
    nwant = ref.gated_norm(num(v), np.ones(C))
    close(z, nwant, FP32 * np.abs(nwant), "bf16", "norm")


# --------------------------------------------------------------------------- #
# The selective scan
# --------------------------------------------------------------------------- #

# (b, T, channels, N, G, dtype, lengths per row, nseq, (before, after), has D, z, bias, softplus)
SCAN = {
    "one_token": (1, 1, 8, 16, 1, "f32", None, 1, (0, 0), True, True, True, True),
    "one_channel_one_state": (2, 37, 1, 1, 1, "f32", None, 1, (1, 2), True, True, True, True),
    "bare": (2, 40, 33, 5, 1, "f32", None, 1, (0, 0), False, False, False, False),
    "tile_edges": (1, 97, 64, 16, 1, "bf16", None, 1, (0, 8), True, True, True, True),
    "groups": (2, 33, 72, 8, 3, "bf16", None, 1, (3, 5), True, True, False, True),
    "groups_f32": (1, 64, 70, 16, 2, "f32", None, 1, (2, 2), False, True, True, True),
    "many_states": (1, 20, 36, 64, 1, "f32", None, 1, (0, 0), True, False, True, True),
    "odd_states": (2, 31, 40, 67, 1, "bf16", None, 1, (0, 0), True, True, True, True),
    "most_states": (1, 9, 10, 256, 1, "f32", None, 1, (0, 0), True, True, True, True),
    # 16-byte and narrower asynchronous copies of every shape: aligned rows, full tiles
    "most_states_bf16": (1, 150, 10, 256, 1, "bf16", None, 1, (0, 0), True, True, True, True),
    "states_128_bf16": (1, 150, 12, 128, 1, "bf16", None, 1, (0, 0), True, True, True, True),
    "states_128_f32": (1, 150, 12, 128, 1, "f32", [[70, 80]], 2, (0, 0), True, True, True, True),
    "states_64_bf16": (1, 150, 20, 64, 1, "bf16", [[70, 80]], 2, (0, 0), True, True, True, True),
    "states_32_bf16": (1, 150, 20, 32, 1, "bf16", None, 1, (0, 0), True, True, True, True),
    "states_8_f32": (1, 300, 64, 8, 1, "f32", None, 1, (0, 0), True, True, True, True),
    "packed": (2, 100, 48, 16, 1, "bf16", [[40, 60], [1, 99]], 2, (16, 0), True, True, True, True),
    "packed_short": (2, 40, 34, 16, 2, "f32", [[1, 1, 1, 2, 3, 32], [8, 8, 8, 7, 1, 8]], 6, (0, 0), True, True, True,
                     True),
    "packed_absent": (2, 34, 32, 24, 1, "bf16", [[0, 10, 0, 0, 24, 0], [34, 0, 0, 0, 0, 0]], 6, (0, 0), True, False,
                      True, True),
    "packed_cut_at_tiles": (1, 97, 9, 3, 1, "f32", [[32, 32, 1, 31, 1]], 7, (0, 0), False, True, True, True),
    "long": (1, 1500, 24, 16, 1, "f32", None, 1, (0, 0), True, True, True, True),
    "long_packed": (1, 1500, 24, 16, 1, "bf16", [[700, 1, 299, 500]], 4, (0, 0), True, True, True, True),
}


def scan_inputs(rng, b, T, c, N, G, dt, has_D, has_z, has_bias, softplus):
    u, z = rand(rng, b, T, c, dtype=dt), rand(rng, b, T, c, dtype=dt) if has_z else None
    step = rand(rng, b, T, c, dtype=dt, scale=1.0, shift=-2.0)
    if not softplus:
        step = (step.float().abs() * 0.1).to(DT[dt])
    A = -torch.exp(torch.from_numpy(rng.uniform(-3.0, 2.8, (c, N)).astype(np.float32)))
    B, C = rand(rng, b, T, G, N, dtype=dt), rand(rng, b, T, G, N, dtype=dt, scale=N ** -0.5)
    return dict(u=u, dt=step, A=A, B=B, C=C, D=rand(rng, c) if has_D else None, z=z,
                dt_bias=rand(rng, c, scale=0.3, shift=-0.5 if softplus else 0.5) if has_bias else None,
                dt_softplus=softplus)


def on_gpu(i, pad):
    """The scan's inputs on the GPU, activations as slices, B and C side by side in one tensor."""
    low = torch.cat([i["B"].flatten(-2), i["C"].flatten(-2)], -1)
    low = sliced(low, *pad)
    n = low.shape[-1] // 2
    shape = i["B"].shape[-2:]
    g = {k: sliced(i[k], *pad) for k in ("u", "dt", "z") if i[k] is not None}
    g.update(B=low[..., :n].unflatten(-1, shape), C=low[..., n:].unflatten(-1, shape), A=cuda(i["A"]), D=cuda(i["D"]),
             dt_bias=cuda(i["dt_bias"]), dt_softplus=i["dt_softplus"])
    return g


def scan_reference(i, **kw):
    j = {k: num(v) if torch.is_tensor(v) else v for k, v in i.items()}
    return ref.selective_scan(j["u"], j["dt"], j["A"], j["B"], j["C"], D=j["D"], z=j["z"], dt_bias=j["dt_bias"],
                              dt_softplus=j["dt_softplus"], bounds=True, **kw)


def check_scan(y, final, want, i, dt, what=""):
    wy, wf, ybound, fbound = want
    gate = 1.0 if i["z"] is None else 1.0 + np.abs(num(i["z"]))
    close(y, wy, FP32 * ybound * gate, dt, what + "y")
    close(final, wf, FP32 * (fbound + np.abs(wf)), "f32", what + "final states")


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("name", sorted(SCAN))
def test_selective_scan(name, init):
    b, T, c, N, G, dt, lengths, nseq, pad, has_D, has_z, has_bias, softplus = SCAN[name]
    rng = np.random.default_rng(len(name) + 50 * init)
    i = scan_inputs(rng, b, T, c, N, G, dt, has_D, has_z, has_bias, softplus)
    h0 = rand(rng, b, nseq, N, c) if init else None
    ids = None if lengths is None else ids_of(lengths, T)
    want = scan_reference(i, init_states=num(h0), seq_idx=ids, nseq=nseq)
    y, final = ssd.selective_scan(**on_gpu(i, pad), init_states=cuda(h0), seq_idx=cuda(ids), nseq=nseq)
    check_scan(y, final, want, i, dt)


@pytest.mark.parametrize("b,c,N,G,dt,pad", [(2, 40, 16, 1, "bf16", (0, 8)), (1, 1, 1, 1, "f32", (0, 0)),
                                            (3, 130, 5, 2, "f32", (1, 0)), (2, 33, 67, 1, "bf16", (0, 0)),
                                            (1, 12, 256, 1, "f32", (0, 0))])
def test_selective_steps_continue_a_prompt(b, c, N, G, dt, pad):
    T, T0 = 14, 9
    rng = np.random.default_rng(c)
    i = scan_inputs(rng, b, T, c, N, G, dt, True, True, True, True)
    want = scan_reference(i)
    g = on_gpu(i, pad)
    part = lambda f: {k: f(v) if k in ("u", "dt", "z", "B", "C") else v for k, v in g.items()}  # noqa: E731
    y0, final = ssd.selective_scan(**part(lambda v: v[:, :T0]))
    state, ys = final[:, 0].contiguous(), [y0]
    for t in range(T0, T):
        ys.append(ssd.selective_step(state=state, **part(lambda v: v[:, t]))[:, None])
    check_scan(torch.cat(ys, 1), state[:, None], want, i, dt)


def test_selective_scan_far_step_sizes():
    """Step sizes at both ends: none (delta = 0: the state stays), and large ones
    (the state is forgotten, decays below the smallest number)."""
    rng = np.random.default_rng(8)
    i = scan_inputs(rng, 1, 48, 32, 16, 1, "f32", True, True, False, False)
    i["dt"][:, ::3] = 0.0
    i["dt"][:, 1::7] = 60.0
    i["dt"][:, 5::11] = 1e4
    want = scan_reference(i)
    check_scan(*ssd.selective_scan(**on_gpu(i, (0, 0))), want, i, "f32")
    i = scan_inputs(rng, 1, 48, 32, 16, 1, "f32", True, True, False, True)
    i["dt"][:, ::3] = -40.0  # softplus underflows to exp(-40)
    i["dt"][:, 1::7] = 50.0  # softplus is the identity
    want = scan_reference(i)
    check_scan(*ssd.selective_scan(**on_gpu(i, (0, 0))), want, i, "f32")


# --------------------------------------------------------------------------- #
# Norms
# --------------------------------------------------------------------------- #

NORM = [  # (leading sizes, channels, groups, dtype, (before, after) of the slices)
    ((1,), 1, 1, "f32", (0, 0)), ((3,), 7, 1, "bf16", (1, 0)), ((2, 5), 96, 4, "bf16", (8, 8)),
    ((2, 3), 90, 2, "f32", (0, 2)), ((4, 2), 768, 1, "bf16", (0, 0)), ((2, 2), 1536, 8, "f32", (4, 0)),
    ((1, 3), 5120, 1, "bf16", (0, 16)), ((2,), 4999, 1, "f32", (0, 0)), ((2,), 8191, 1, "bf16", (0, 1)),
    ((2,), 10240, 1, "f32", (0, 0)), ((1,), 32768, 1, "bf16", (0, 0)), ((2,), 32768, 1, "f32", (0, 0)),
    ((1,), 32767, 1, "bf16", (0, 0)), ((2,), 20480, 4, "bf16", (0, 0)),
]


def norm_bound(want, z):
    # the mean's sum is a tree over positive terms, its root and quotient a few roundings:
    # a relative error of the norm, 16 * 2^-24 in all; the gate's as above
    return FP32 * np.abs(want) * (1.0 if z is None else 2 + np.abs(num(z)))


@pytest.mark.parametrize("gate", ["first", "last", "none"])
@pytest.mark.parametrize("lead,c,G,dt,pad", NORM)
def test_gated_norm(lead, c, G, dt, pad, gate):
    rng = np.random.default_rng(c + G)
    x, w = rand(rng, *lead, c, dtype=dt), rand(rng, c, scale=0.3, shift=1.0)
    z = None if gate == "none" else rand(rng, *lead, c, dtype=dt, scale=2.0)
    want = ref.gated_norm(num(x), num(w), num(z), G, 1e-5, gate == "first")
    y = ssd.gated_norm(sliced(x, *pad), cuda(w), None if z is None else sliced(z, pad[1], pad[0]), ngroups=G,
                       gate_first=gate == "first")
    assert y.shape == x.shape and y.dtype == x.dtype
    zmax = None if z is None else torch.full_like(z, float(z.abs().max()))  # a group's errors share its norm
    close(y, want, norm_bound(want, zmax), dt, "out")


@pytest.mark.parametrize("res", ["f32", "same", "none", "in_place"])
@pytest.mark.parametrize("scale", ["one", "number", "channels"])
@pytest.mark.parametrize("lead,c,G,dt,pad", [n for n in NORM if n[2] == 1])
def test_add_norm(lead, c, G, dt, pad, res, scale):
    rng = np.random.default_rng(c)
    x, w = rand(rng, *lead, c, dtype=dt), rand(rng, c, scale=0.3, shift=1.0)
    rdt = dt if res == "same" else "f32"
    r = None if res == "none" else rand(rng, *lead, c, dtype=rdt, scale=3.0)
    s = {"one": 1.0, "number": 0.625, "channels": rand(rng, c)}[scale]
    sv = num(s) if torch.is_tensor(s) else s
    want, wr = ref.add_norm(num(x), num(w), num(r), sv)
    rg = None if r is None else cuda(r) if res == "in_place" else sliced(r, *pad)
    kw = dict(residual_out=rg) if res == "in_place" else {}
    y, ro = ssd.add_norm(sliced(x, *pad), cuda(w), rg, scale=cuda(s) if torch.is_tensor(s) else s, **kw)
    assert ro.dtype == DT[rdt] and (res != "in_place" or ro is rg)
    size = np.abs(num(x) * sv) + (0.0 if r is None else np.abs(num(r)))  # the sum may cancel
    close(ro, wr, FP32 * size, rdt, "residual")
    rms = np.sqrt((wr * wr).mean(-1, keepdims=True) + 1e-5)
    close(y, want, FP32 * (np.abs(want) + np.abs(num(w)) * size / rms), dt, "out")


def test_norm_of_zero_and_of_large_rows():
    """A row of zeros gives zeros; values near the end of what 32 bits can square stay exact."""
    x = torch.zeros(3, 64, device="cuda")
    x[1] = 1e18
    x[2] = 1e-18
    w = torch.ones(64, device="cuda")
    y = ssd.gated_norm(x, w)
    want = ref.gated_norm(num(x), num(w))
    close(y, want, FP32 * np.abs(want), "f32", "out")
    assert (y[0] == 0).all()


# --------------------------------------------------------------------------- #
# A run of them, streams, graphs
# --------------------------------------------------------------------------- #

def test_mixer_prompt_then_tokens():
    """The token mixing of a block as it is used: the convolution's split feeds
    discretize and ssd_fwd, the gate is a slice of the same projection, and single
    tokens continue from the prompt's windows and states."""
    b, T, T0, H, P, N, d = 2, 140, 132, 4, 64, 64, 128
    inner, conv = H * P, H * P + 2 * N
    rng = np.random.default_rng(21)
    proj = rand(rng, b, T, inner + conv + H, dtype="bf16")
    w, bias, nw = rand(rng, conv, 4, scale=0.5), rand(rng, conv, scale=0.1), rand(rng, inner, scale=0.1, shift=1.0)
    A, D, dtb = -torch.exp(rand(rng, H)), rand(rng, H), rand(rng, H, shift=-2.0)
    res, pw = rand(rng, b, T, inner, scale=2.0), rand(rng, inner, scale=0.1, shift=1.0)
    # the definitions, in 64 bits throughout
    z, xbc, dt = (num(v) for v in proj.split([inner, conv, H], -1))
    y, _ = ref.causal_conv(xbc, num(w), num(bias))
    X = y[..., :inner].reshape(b, T, H, P)
    B, C = (y[..., inner + k * N:inner + (k + 1) * N].reshape(b, T, 1, N) for k in (0, 1))
    log_a, Xd = oracle.discretize(dt, num(A), X, dt_bias=num(dtb))
    Y, _ = oracle.ssd_reference(Xd, log_a, B, C, num(D), None, None)
    out = ref.gated_norm(Y.reshape(b, T, inner), num(nw), z)
    want, wres = ref.add_norm(out, num(pw), num(res), 0.5)

    g = proj.cuda()
    gw, gb, gnw, gA, gD, gdtb, gpw = map(cuda, (w, bias, nw, A, D, dtb, pw))

    def tail(Y, z, r):
        o = ssd.gated_norm(Y.flatten(-2), gnw, z=z)
        return ssd.add_norm(o, gpw, r, scale=0.5, residual_out=r)

    p = g[:, :T0]
    (x, B, C), win = ssd.causal_conv(p[..., inner:inner + conv], gw, gb, splits=[inner, N, N])
    la, X = ssd.discretize(p[..., -H:].float().contiguous(), gA, x.unflatten(-1, (H, P)), dt_bias=gdtb)
    Y, F = ssd.ssd_fwd(X, la, B.unsqueeze(2), C.unsqueeze(2), 128, D=gD)
    r0 = res[:, :T0].contiguous().cuda()
    ys, rs = [tail(Y, p[..., :inner], r0)[0]], [r0]
    win, state = win[:, 0].contiguous(), F[:, 0].contiguous()
    for t in range(T0, T):
        p = g[:, t]
        x, B, C = ssd.conv_step(p[..., inner:inner + conv], win, gw, gb, splits=[inner, N, N])
        la, X = ssd.discretize(p[:, None, -H:].float().contiguous(), gA, x.view(b, 1, H, P), dt_bias=gdtb)
        Y = ssd.decode_step(X[:, 0], la[:, 0], B.unsqueeze(1), C.unsqueeze(1), state, D=gD)
        r = res[:, t].contiguous().cuda()
        ys.append(tail(Y, p[..., :inner], r)[0][:, None])
        rs.append(r[:, None])
    torch.cuda.synchronize()
    ssd.check_device_error()
    # bf16 between the operators: ssd_fwd's tolerance of 2e-2 of the largest value carries the chain
    assert_close(num(torch.cat(ys, 1)), want, 2e-2, "block output")
    assert_close(num(torch.cat(rs, 1)), wres, 2e-2, "residual stream")


def all_ops(rng):
    """One call of each operator on its own inputs: name -> function returning tensors."""
    c, N, b, T = 64, 16, 2, 50
    i = on_gpu(scan_inputs(rng, b, T, c, N, 1, "bf16", True, True, True, True), (0, 0))
    one = {k: v[:, 0].contiguous() if k in ("u", "dt", "z", "B", "C") else v for k, v in i.items()}
    x, w, bias = rand(rng, b, T, c, dtype="bf16").cuda(), rand(rng, c, 4).cuda(), rand(rng, c).cuda()
    h0, win0 = rand(rng, b, N, c).cuda(), rand(rng, b, 3, c, dtype="bf16").cuda()
    state, win = h0.clone(), win0.clone()
    res = rand(rng, b, T, c).cuda()

    def conv_step():
        win.copy_(win0)
        return ssd.conv_step(x[:, 1], win, w, bias), win

    def scan_step():
        state.copy_(h0)
        return ssd.selective_step(state=state, **one), state

    return dict(conv=lambda: ssd.causal_conv(x, w, bias), conv_step=conv_step,
                scan=lambda: ssd.selective_scan(**i), scan_step=scan_step,
                gated_norm=lambda: (ssd.gated_norm(x, bias, z=i["z"]),),
                add_norm=lambda: ssd.add_norm(x, bias, res, scale=0.5))


@pytest.mark.parametrize("name", ["conv", "conv_step", "scan", "scan_step", "gated_norm", "add_norm"])
def test_other_stream_and_graph_give_the_same(name):
    f = all_ops(np.random.default_rng(4))[name]
    want = [t.clone() for t in f()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = f()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan")) if name not in ("conv_step", "scan_step") else None
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_at_once_on_two_streams():
    """Two calls of the same operators that overlap share nothing."""
    rng = np.random.default_rng(9)
    sets = [all_ops(rng), all_ops(rng)]
    want = [{k: [t.clone() for t in f()] for k, f in s.items()} for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [{}, {}]
    for k in sets[0]:
        for s, st, g in zip(sets, streams, got):
            with torch.cuda.stream(st):
                g[k] = s[k]()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for k in w:
            assert all(torch.equal(a, b) for a, b in zip(g[k], w[k])), k


def test_stream_argument_and_given_outputs():
    rng = np.random.default_rng(2)
    x, w = rand(rng, 2, 20, 32, dtype="bf16").cuda(), rand(rng, 32, 4).cuda()
    y0, f0 = ssd.causal_conv(x, w, splits=[16, 16])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in y0]
    fin = torch.empty_like(f0)
    torch.cuda.synchronize()
    y, f = ssd.causal_conv(x, w, splits=[16, 16], out=out, final_out=fin, stream=st)
    st.synchronize()
    assert f is fin and all(a is b for a, b in zip(y, out))
    assert all(torch.equal(a, b) for a, b in zip(y, y0)) and torch.equal(f, f0)
    # every operator on a given stream, its inputs dropped right after the call
    i = on_gpu(scan_inputs(rng, 1, 40, 32, 16, 1, "bf16", True, True, True, True), (0, 0))
    res, z, g = rand(rng, 2, 20, 32).cuda(), rand(rng, 2, 20, 32, dtype="bf16").cuda(), rand(rng, 32).cuda()
    want = [*ssd.selective_scan(**i), ssd.gated_norm(x, g, z=z), *ssd.add_norm(x, g, res, scale=g)]
    torch.cuda.synchronize()
    got = [*ssd.selective_scan(**{k: v.clone() if torch.is_tensor(v) else v for k, v in i.items()}, stream=st)]
    got.append(ssd.gated_norm(x.clone(), g.clone(), z=z.clone(), stream=st))
    got += ssd.add_norm(x.clone(), g.clone(), res.clone(), scale=g.clone(), stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y, f = ssd.causal_conv(x, w, return_final_states=False)
    assert f is None and torch.equal(y, torch.cat(y0, -1))


def test_refusals_on_the_gpu():
    x = torch.zeros(2, 8, 32, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(32, 4, device="cuda")
    with pytest.raises(ssd.SSDError, match="unsupported"):
        ssd.causal_conv(x, torch.zeros(32, 5, device="cuda"))
    with pytest.raises(ssd.SSDError, match="invalid"):  # an output on the input
        ssd.causal_conv(x, w, out=x)
    with pytest.raises(TypeError):
        ssd.causal_conv(x, w.bfloat16())
    with pytest.raises(ValueError, match="last dimension"):
        ssd.causal_conv(torch.zeros(2, 8, 64, device="cuda")[..., ::2], w)
    with pytest.raises(ValueError):
        ssd.conv_step(x[:, 0], torch.zeros(2, 2, 32, device="cuda", dtype=torch.bfloat16), w)
    with pytest.raises(ValueError, match="is on"):
        ssd.gated_norm(x, torch.zeros(32))
    with pytest.raises(ssd.SSDError, match="invalid"):
        ssd.gated_norm(x, w[:, 0].contiguous(), ngroups=5)
    with pytest.raises(TypeError):
        ssd.add_norm(x.float(), w[:, 0].contiguous(), x)
    with pytest.raises(TypeError):
        ssd.gated_norm(x.half(), w[:, 0].contiguous())
