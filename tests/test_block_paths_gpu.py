"""The operators around the scan on the paths that their launch rules choose by
size and alignment, against the fp64 definitions (oracle.block_oracle).
Tolerances: those of test_block_gpu, whose derivation is at its head. The large
convolutions are compared on the device with a vectorised form of the definition
in 64 bits, which a CPU test holds to the oracle's."""
import numpy as np
import pytest
import torch

import mamba_ssd_layer_chunked_b200 as ssd
from oracle import block_oracle as ref
from tests.test_block_gpu import (DT, FP32, HALF, check_scan, close, cuda, ids_of, num, on_gpu, rand, scan_inputs,
                                  scan_reference, sliced)

# --------------------------------------------------------------------------- #
# The short convolution: tiles of several batches
# --------------------------------------------------------------------------- #

def conv_tile(b, T, vectors):
    """Tokens that a thread walks, in batches of 4: 32, or fewer while the threads would not fill the SMs."""
    tile = 32
    while tile > 4 and b * -(-T // tile) * vectors < 148 * 4 * 128:
        tile //= 2
    return tile


# Sequence lengths by where they end in a tile of 32 (batches of 4): inside a batch, at a batch's edge, at a
# tile's edge, one token apart, an absent id (0); the rest of the row is one long sequence.
CUTS = {
    "plain": None,
    "in_batch": [5, 9, 21, 1, 30, 6, 23, 33],
    "batch_edge": [4, 8, 12, 8, 16, 4, 44],
    "tile_edge": [32, 64, 1, 31, 32],
    "singles": [1, 1, 1, 1, 1, 1, 25, 2, 1, 30, 3, 1, 29, 1],
    "absent": [0, 6, 0, 0, 27, 31, 0],
    "mixed_then_whole": [2, 19, 18, 14, 12, 33, 11, 27],
}

# (channels, vectors of them per row, W, dtype, (before, after) of the slice, splits)
ROWS = {
    "bf16_16_bytes": (4096, 512, 4, "bf16", (8, 8), [3584, 256, 256]),
    "f32_16_bytes": (2048, 512, 4, "f32", (4, 0), None),
    "w3": (2048, 256, 3, "bf16", (0, 0), None),
    "w2": (1024, 256, 2, "f32", (0, 4), [1000, 24]),
    "bf16_pairs": (1026, 513, 4, "bf16", (2, 0), None),
    "bf16_single": (515, 515, 4, "bf16", (1, 0), None),
    "f32_single": (515, 515, 3, "f32", (0, 0), None),
}


def conv_64(x, weight, bias, init, ids, act):
    """The definition in 64 bits for all tokens at once: (y, final windows). init [b, nseq, W-1, C]; ids may be None."""
    x, init = x.double(), init.double()
    (b, T, C), (nseq, back) = x.shape, init.shape[1:3]
    t = torch.arange(T, device=x.device).expand(b, T)
    ids = torch.zeros_like(t) if ids is None else ids.long()
    first = torch.ones_like(ids, dtype=torch.bool)
    first[:, 1:] = ids[:, 1:] != ids[:, :-1]
    start = torch.where(first, t, 0).cummax(1).values
    source = torch.cat([init.reshape(b, nseq * back, C), x], 1)  # every input and initial window of a row
    row = torch.arange(b, device=x.device)[:, None]

    def entry(k):  # where the input k tokens back is
        return torch.where(t - k >= start, nseq * back + t - k, ids * back + back + (t - k - start))

    y = torch.zeros_like(x)
    for k in range(back + 1):
        y += source[row, entry(k)] * weight.double()[:, back - k]
    if bias is not None:
        y += bias.double()
    final = init.clone()
    end = torch.ones_like(first)
    end[:, :-1] = first[:, 1:]
    r, e = end.nonzero(as_tuple=True)
    for k in range(back):
        final[r, ids[r, e], back - 1 - k] = source[r, entry(k)[r, e]]
    return (y / (1 + torch.exp(-y)) if act else y), final


@pytest.mark.parametrize("lengths", [None, [[1, 1, 0, 2, 9, 3, 0, 7], [23, 0, 0, 0, 0, 0, 0, 0]]])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_64_is_the_oracle(W, lengths):
    rng = np.random.default_rng(W)
    nseq = 1 if lengths is None else 8
    x, w, bias, h0 = rand(rng, 2, 23, 5), rand(rng, 5, W), rand(rng, 5), rand(rng, 2, nseq, W - 1, 5)
    ids = None if lengths is None else ids_of(lengths, 23)
    for act in (False, True):
        y, final = conv_64(x, w, bias, h0, ids, act)
        wy, wfinal = ref.causal_conv(num(x), num(w), num(bias), num(h0), ids, nseq, act)
        assert np.allclose(num(y), wy, rtol=1e-13, atol=1e-13) and np.array_equal(num(final), wfinal)


@pytest.mark.gpu
@pytest.mark.parametrize("cuts", sorted(CUTS))
@pytest.mark.parametrize("tile", [8, 16, 32])
@pytest.mark.parametrize("name", sorted(ROWS))
def test_conv_walks_tiles_of_several_batches(name, tile, cuts):
    C, vectors, W, dt, pad, splits = ROWS[name]
    tiles = -(-148 * 4 * 128 // vectors)
    b, T = (1, (tiles + 2) * tile - 13) if cuts != "plain" else (2, (tiles // 2 + 2) * tile + 3)
    assert conv_tile(b, T, vectors) == tile
    ids, nseq = None, 1
    if CUTS[cuts] is not None:
        head = CUTS[cuts]
        lengths = head + [T - 37 - sum(head), 20, 17, 0]  # the last cuts lie in the row's last tiles; an absent id
        ids, nseq = ids_of([lengths], T).cuda(), len(lengths)
    g = torch.Generator(device="cuda").manual_seed(C + tile)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    x, w, bias = normal(b, T, C).to(DT[dt]), 0.7 * normal(C, W), normal(C)
    h0 = normal(b, nseq, W - 1, C).to(DT[dt])
    want, wfinal = conv_64(x, w, bias, h0, ids, True)
    size, _ = conv_64(x.abs(), w.abs(), bias.abs(), h0.abs(), ids, False)
    y, final = ssd.causal_conv(sliced(x, *pad), w, bias, init_states=h0, seq_idx=ids, nseq=nseq, splits=splits)
    y = torch.cat(y, -1) if splits else y
    lim = HALF[dt] * want.abs() * (1 + 2.0 ** -7) + FP32 * size * (1 + size) + 1e-37
    over = (y.double() - want).abs() - lim
    at = np.unravel_index(int(over.argmax()), over.shape)
    assert over[at] <= 0, (at, float(y[at]), float(want[at]), float(lim[at]))  # also fails on NaN
    assert torch.equal(final.double(), wfinal)  # windows are copies of inputs


# --------------------------------------------------------------------------- #
# The selective scan
# --------------------------------------------------------------------------- #

def run_scan(rng, b, T, c, N, G, dt, lengths=None, pad=(0, 0), init=True):
    """selective_scan with every optional input, against its definition."""
    nseq = 1 if lengths is None else len(lengths[0])
    i = scan_inputs(rng, b, T, c, N, G, dt, True, True, True, True)
    h0 = rand(rng, b, nseq, N, c) if init else None
    ids = None if lengths is None else ids_of(lengths, T)
    want = scan_reference(i, init_states=None if h0 is None else h0.double().numpy(), seq_idx=ids, nseq=nseq)
    y, final = ssd.selective_scan(**on_gpu(i, pad), init_states=cuda(h0), seq_idx=cuda(ids), nseq=nseq)
    check_scan(y, final, want, i, dt)


# Aligned rows (copied 16 bytes at a time) whose last unit of channels is partial: a warp takes 8 channels
# with 9 to 16 states, 16 with fewer, and one copy holds 4 (fp32) or 8 (bf16) of them.
@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("c,N,G,dt", [(12, 16, 1, "f32"), (4, 12, 1, "f32"), (1540, 16, 1, "f32"), (24, 16, 2, "f32"),
                                      (20, 8, 1, "f32"), (24, 8, 1, "f32"), (28, 4, 1, "f32"), (2436, 8, 1, "f32"),
                                      (24, 8, 1, "bf16"), (8, 8, 1, "bf16"), (48, 8, 2, "bf16"), (2440, 8, 1, "bf16")])
def test_scan_of_partial_units(c, N, G, dt, packed):
    T = 77
    run_scan(np.random.default_rng(c + N), 1, T, c, N, G, dt, [[30, 47]] if packed else None)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_size_keeps_its_relative_accuracy(dt):
    """u = B = C = 1 and A = 0: one token's state is delta = softplus(dt + dt_bias). Relative error, counted in 2^-24:
    exponential 2, reciprocal 2, the sum 2 + e, the product, the series (2) and its last multiply-add 1 each: below
    the 16 of FP32, from e near 1 to e near the smallest normal number."""
    c = 4096
    step = torch.linspace(-85.0, 30.0, c).to(DT[dt])
    bias = torch.linspace(0.0, 0.5, c)
    z = (step.float() + bias).double().numpy()  # the sum, rounded as the kernel rounds it
    one = lambda *shape: torch.ones(shape, dtype=DT[dt], device="cuda")  # noqa: E731
    A, zero = torch.zeros(c, 1, device="cuda"), torch.zeros(1, 1, c, device="cuda")
    want = ref.softplus(z)
    y, final = ssd.selective_scan(one(1, 1, c), step.cuda().view(1, 1, c), A, one(1, 1, 1, 1), one(1, 1, 1, 1),
                                  dt_bias=bias.cuda())
    ys = ssd.selective_step(one(1, c), step.cuda().view(1, c), A, one(1, 1, 1), one(1, 1, 1), zero, dt_bias=bias.cuda())
    for state in (final, zero):
        close(state.view(-1), want, FP32 * want, "f32", "delta")
    for out in (y, ys):
        close(out.view(-1), want, FP32 * want, dt, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T", [1, 13, 77, 300])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_decays_of_minus_infinity(dt, T, packed):
    """A state with A = -inf forgets all but the last token, whatever the row's length."""
    b, c, N = 1, 32, 16
    rng = np.random.default_rng(T)
    i = scan_inputs(rng, b, T, c, N, 1, dt, True, True, True, True)
    i["A"][:, ::3] = -np.inf
    lengths = [T // 3, T - T // 3, 0] if packed else None
    nseq = 3 if packed else 1
    ids, h0 = ids_of([lengths], T) if packed else None, rand(rng, b, nseq, N, c)
    want = scan_reference(i, init_states=num(h0), seq_idx=ids, nseq=nseq)
    y, final = ssd.selective_scan(**on_gpu(i, (0, 0)), init_states=cuda(h0), seq_idx=cuda(ids), nseq=nseq)
    check_scan(y, final, want, i, dt)


# --------------------------------------------------------------------------- #
# The scan's shapes: states per lane, warps per CTA, copied and plain loads
# --------------------------------------------------------------------------- #

# states -> (channels of a warp, CTAs up to which one has more warps, tokens that the CTA's warps take in turn
# then, and else)
SHAPES = {8: (16, 148, 128, 64), 16: (8, 148, 128, 64), 24: (4, 148, 128, 64), 32: (4, 148, 128, 64),
          64: (4, 296, 32, 16), 128: (2, 296, 32, 16), 200: (2, 0, 16, 16)}


@pytest.mark.gpu
@pytest.mark.parametrize("copied", [True, False])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("N", sorted(SHAPES))
def test_scan_shapes(N, many, dt, packed, copied):
    """Rows of six turns of a CTA's warps and a rest: the loop without guards runs, and its ends. Rows aligned to 16
    bytes are copied ahead, others (an odd offset and stride) loaded element by element."""
    warp, few, turn, turn_many = SHAPES[N]
    G = 2 if many and packed else 1
    c = (few // G + 2) * G * warp if many else 3 * warp
    T = 6 * (turn_many if many else turn) + 13
    assert not many or c // warp > few
    lengths = [[T // 3, 1, 1, 5, T - T // 3 - 7 - 9, 0, 9]] if packed else None
    run_scan(np.random.default_rng(N + T), 1, T, c, N, G, dt, lengths, (0, 0) if copied else (1, 0))


# --------------------------------------------------------------------------- #
# Values and ids at the edges of the contract
# --------------------------------------------------------------------------- #

def same(a, b):
    """Bitwise, whatever the values."""
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.view(kind) == b.view(kind)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N", [5, 16])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_non_finite_inputs_of_the_scan_stay_in_their_sequence(dt, N, bad):
    """A NaN or infinity of u or dt at one token: other channels, rows, sequences and earlier tokens keep every bit."""
    b, T, c, t0, c0 = 2, 90, 40, 40, 11
    rng = np.random.default_rng(N)
    i = scan_inputs(rng, b, T, c, N, 1, dt, True, True, True, True)
    ids = ids_of([[30, 35, 25]] * b, T).cuda()
    h0 = rand(rng, b, 3, N, c).cuda()
    y0, f0 = ssd.selective_scan(**on_gpu(i, (0, 0)), init_states=h0, seq_idx=ids, nseq=3)
    for name in ("u", "dt"):
        if name == "dt" and bad == -float("inf"):
            continue  # a step size of 0, an ordinary value
        j = dict(i, **{name: i[name].clone()})
        j[name][1, t0, c0] = bad
        y, f = ssd.selective_scan(**on_gpu(j, (0, 0)), init_states=h0, seq_idx=ids, nseq=3)
        touched = torch.zeros_like(y, dtype=torch.bool)
        touched[1, t0:65, c0] = True
        assert (same(y, y0) | touched).all() and not torch.isfinite(y[1, t0, c0])
        ftouched = torch.zeros_like(f, dtype=torch.bool)
        ftouched[1, 1, :, c0] = True
        assert (same(f, f0) | ftouched).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_non_finite_inputs_of_the_others_stay_where_they_belong(dt):
    b, T, c, W = 2, 50, 64, 4
    rng = np.random.default_rng(1)
    x, w, bias = rand(rng, b, T, c, dtype=dt).cuda(), rand(rng, c, W).cuda(), rand(rng, c).cuda()
    z, res = rand(rng, b, T, c, dtype=dt).cuda(), rand(rng, b, T, c).cuda()
    ids = ids_of([[22, 28]] * b, T).cuda()
    bad = x.clone()
    bad[1, 20, 7] = float("nan")  # two tokens before its sequence's end
    bad[0, 5, 3] = float("inf")
    run = lambda v: (*ssd.causal_conv(v, w, bias, seq_idx=ids, nseq=2), ssd.gated_norm(v, bias, z=z, ngroups=4),  # noqa: E731
                     *ssd.add_norm(v, bias, res))
    (y0, f0, g0, a0, r0), (y, f, g, a, r) = run(x), run(bad)
    touched = torch.zeros_like(y, dtype=torch.bool)
    touched[1, 20:22, 7] = touched[0, 5:9, 3] = True
    assert (same(y, y0) | touched).all() and torch.isnan(y[1, 20:22, 7]).all()
    ftouched = torch.zeros_like(f, dtype=torch.bool)
    ftouched[1, 0, 1, 7] = True  # the sequence's last three inputs: tokens 19 to 21
    assert (same(f, f0) | ftouched).all() and torch.isnan(f[1, 0, 1, 7])
    rows = torch.zeros_like(y, dtype=torch.bool)
    rows[1, 20] = rows[0, 5] = True
    assert (same(a, a0) | rows).all()
    element = torch.zeros_like(rows)
    element[1, 20, 7] = element[0, 5, 3] = True
    assert (same(r, r0) | element).all()
    groups = torch.zeros_like(rows)
    groups[1, 20, :16] = groups[0, 5, :16] = True  # 4 groups of 16 channels
    assert (same(g, g0) | groups).all()


@pytest.mark.gpu
def test_ids_out_of_range_count_as_the_nearest_one():
    b, T, c, N = 1, 75, 32, 16
    rng = np.random.default_rng(3)
    ids = ids_of([[10, 20, 45]], T)
    wild = ids.clone()
    wild[0, :10] = torch.tensor([-1, -2 ** 31, 0, -7, 0, -1, -1, 0, 0, -3])
    wild[0, 30:] = torch.where(torch.arange(45) % 3 == 0, 2, 2 ** 31 - 1 - torch.arange(45)).int()
    i = on_gpu(scan_inputs(rng, b, T, c, N, 1, "f32", True, True, True, True), (0, 0))
    x, w = rand(rng, b, T, c).cuda(), rand(rng, c, 4).cuda()
    for f in (lambda s: ssd.selective_scan(**i, seq_idx=s, nseq=3), lambda s: ssd.causal_conv(x, w, seq_idx=s, nseq=3)):
        for got, want in zip(f(wild.cuda()), f(ids.cuda())):
            assert torch.equal(got, want)
