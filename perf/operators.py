"""Cases for the operators of a state-space block around its scan: the short
causal convolution, the selective scan with a decay per channel and state (both
for prompts and for single tokens), the gated norm after the mixer and the norm
before a block with its residual. ``run`` is one pass through one of them: in
plain torch operations, or (``own``) through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- #
# Cases
# --------------------------------------------------------------------------- #

def listed():
    return [
        # prompt of the 2.7B-shaped layer: x, B and C channels (80 heads of 64, dstate 128)
        # as one slice of the input projection's output, split into the scan's operands
        dict(name="conv_prompt", op="conv", batch=4, seqlen=4096, channels=5376, split1=128, split2=128, width=4,
             nseq=0, dtype="bf16", ahead=5120, behind=80, bias=True, silu=True),
        # packed prompts of different lengths, some continuing from cached windows, in fp32
        # (24 heads of 64 and dstate 128, the 130M-shaped layer)
        dict(name="conv_packed_f32", op="conv", batch=1, seqlen=8191, channels=1792, split1=0, split2=0, width=4,
             nseq=7, dtype="f32", ahead=0, behind=0, bias=True, silu=True),
        # one token for each of 64 sequences of the 2.7B-shaped layer
        dict(name="conv_step_64", op="conv_step", batch=64, channels=5376, split1=128, split2=128, width=4,
             dtype="bf16", ahead=5120, behind=80, bias=True, silu=True),
        # one token of one sequence: the smallest call, all latency
        dict(name="conv_step_1_f32", op="conv_step", batch=1, channels=1792, split1=0, split2=0, width=4,
             dtype="f32", ahead=0, behind=0, bias=True, silu=True),
        # one prompt through the selective scan: 5120 channels, 16 states each, gate in the
        # second half of the input projection, B and C behind the step size's low-rank columns
        dict(name="scan_prompt", op="scan", batch=1, seqlen=4096, channels=5120, dstate=16, ngroups=1, nseq=0,
             dtype="bf16", ahead=160, gate=True, skip=True, bias=True, softplus=True),
        # packed prompts with cached states in fp32, an odd total length
        dict(name="scan_packed_f32", op="scan", batch=1, seqlen=5003, channels=1536, dstate=16, ngroups=1, nseq=7,
             dtype="f32", ahead=48, gate=True, skip=True, bias=True, softplus=True),
        # one token for each of 64 sequences
        dict(name="scan_step_64", op="scan_step", batch=64, channels=5120, dstate=16, ngroups=1, dtype="bf16",
             ahead=160, gate=True, skip=True, bias=True, softplus=True),
        # one token for three sequences, fp32
        dict(name="scan_step_3_f32", op="scan_step", batch=3, channels=1536, dstate=16, ngroups=1, dtype="f32",
             ahead=48, gate=True, skip=True, bias=True, softplus=True),
        # after the mixer of the 2.7B-shaped layer: the gate is the first slice of the input projection
        dict(name="gated_norm_prompt", op="gated_norm", batch=4, seqlen=4096, channels=5120, ngroups=1, dtype="bf16",
             behind=5456, gate=True, gate_first=True),
        # a few tokens, eight groups per row, the gate after the norm, fp32
        dict(name="gated_norm_grouped_f32", op="gated_norm", batch=5, seqlen=1, channels=1536, ngroups=8, dtype="f32",
             behind=0, gate=True, gate_first=False),
        # before the block, the residual stream of a prompt kept in fp32 (half of 5120 wide)
        dict(name="add_norm_prompt", op="add_norm", batch=4, seqlen=4096, channels=2560, dtype="bf16",
             residual="f32", scaled=False),
        # one token, residual in bf16 with a scale per channel
        dict(name="add_norm_1", op="add_norm", batch=1, seqlen=1, channels=768, dtype="bf16", residual="bf16",
             scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _channels(rng, lo, hi):
    """Half of them multiples of 64, as projections have them, the others any number."""
    c = _log(rng, lo, hi)
    return max(64, c // 64 * 64) if rng.random() < 0.5 else c


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan_step", "gated_norm", "add_norm"])
    dtype = rng.choice(["bf16", "f32"])
    flag = lambda p=0.5: rng.random() < p  # noqa: E731
    if op in ("conv", "conv_step"):
        c = dict(op=op, channels=_channels(rng, 16, 8192), split1=0, split2=0, width=rng.choice([2, 3, 4, 4]),
                 dtype=dtype, ahead=rng.choice([0, 0, 64, 5120]), behind=rng.choice([0, 24, 80]), bias=flag(0.8),
                 silu=flag(0.8))
        if flag():
            c["split1"] = c["split2"] = max(1, min(128, c["channels"] // 4))
        if op == "conv_step":
            return dict(c, batch=_log(rng, 1, 256))
        batch = rng.choice([1, 1, 2, 4, 8])
        seqlen = _log(rng, 1, 32768)
        while batch * seqlen * c["channels"] * (1 if dtype == "bf16" else 2) > 4 * 4096 * 5376:
            seqlen = (seqlen + 1) // 2
        return dict(c, batch=batch, seqlen=seqlen, nseq=rng.choice([0, 1, 0, min(seqlen, rng.randint(2, 24))]))
    if op in ("scan", "scan_step"):
        groups = rng.choice([1, 1, 1, 2, 4])
        c = dict(op=op, channels=max(1, _channels(rng, 32, 8192) // groups) * groups,
                 dstate=rng.choice([16, 16, 16, 8, 5, 24, 32, 64]), ngroups=groups, dtype=dtype,
                 ahead=rng.choice([0, 48, 160]), gate=flag(0.8), skip=flag(0.8), bias=flag(0.8), softplus=flag(0.9))
        if op == "scan_step":
            return dict(c, batch=max(1, min(_log(rng, 1, 256), 256 * 5120 * 16 // (c["channels"] * c["dstate"]))))
        batch = rng.choice([1, 1, 2, 4])
        seqlen = _log(rng, 1, 16384)
        while batch * seqlen * c["channels"] * max(16, c["dstate"]) > 4096 * 5120 * 16:
            seqlen = (seqlen + 1) // 2
        return dict(c, batch=batch, seqlen=seqlen, nseq=rng.choice([0, 1, 0, min(seqlen, rng.randint(2, 24))]))
    batch, seqlen = rng.choice([1, 2, 4, 8]), _log(rng, 1, 4096)
    if op == "gated_norm":
        groups = rng.choice([1, 1, 2, 8])
        channels = max(1, _channels(rng, 64, 8192) // groups) * groups
        while batch * seqlen * channels * (1 if dtype == "bf16" else 2) > 4 * 4096 * 5120:
            seqlen = (seqlen + 1) // 2
        return dict(op=op, batch=batch, seqlen=seqlen, channels=channels, ngroups=groups, dtype=dtype,
                    behind=rng.choice([0, 24, 2128]), gate=flag(0.85), gate_first=flag(0.7))
    channels = _channels(rng, 64, 8192)
    while batch * seqlen * channels * (1 if dtype == "bf16" else 2) > 4 * 4096 * 2560:
        seqlen = (seqlen + 1) // 2
    return dict(op=op, batch=batch, seqlen=seqlen, channels=channels, dtype=dtype,
                residual=rng.choice(["f32", dtype, "none"]), scaled=flag())


# --------------------------------------------------------------------------- #
# Inputs
# --------------------------------------------------------------------------- #

class _Draw:
    """Seeded normal and uniform values on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(self, *shape, scale=1.0, dtype=torch.float32, shift=0.0):
        v = torch.randn(shape, generator=self.g, device="cuda")
        return v.mul_(scale).add_(shift).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.g, device="cuda").mul_(hi - lo).add_(lo)


def _ids(c, d):
    """Sequence ids [batch, seqlen] of nseq packed sequences with random lengths, or None."""
    b, t, n = c["batch"], c["seqlen"], c["nseq"]
    if n < 1:
        return None
    rank = torch.rand((b, t), generator=d.g, device="cuda")
    rank[:, 0] = -1.0  # the first token starts the first sequence, n - 1 others start at random places
    starts = torch.zeros((b, t), dtype=torch.int32, device="cuda")
    starts.scatter_(1, rank.argsort(dim=1)[:, 1:n], 1)
    return starts.cumsum(1, dtype=torch.int32).contiguous()


def _splits(c):
    tail = [n for n in (c["split1"], c["split2"]) if n > 0]
    return [c["channels"] - sum(tail)] + tail if tail else None


def _decays(d, channels, dstate):
    """A < 0 per channel and state, spread as a trained layer's: from 1 to about 16."""
    return -torch.exp(d.uniform(channels, dstate, lo=0.0, hi=math.log(16.0)))


def prepare(case, seed):
    c, d = case, _Draw(seed)
    dt = DTYPES[c["dtype"]]
    s = dict(case=c)
    op = c["op"]
    if op in ("conv", "conv_step"):
        n, w = c["channels"], c["width"]
        lead = (c["batch"], c["seqlen"]) if op == "conv" else (c["batch"],)
        proj = d.normal(*lead, c["ahead"] + n + c["behind"], dtype=dt)
        s["x"] = proj[..., c["ahead"]:c["ahead"] + n]
        s["weight"] = d.normal(n, w, scale=w ** -0.5)
        s["bias"] = d.normal(n, scale=0.1) if c["bias"] else None
        s["activation"] = "silu" if c["silu"] else None
        s["splits"] = _splits(c)
        if op == "conv":
            s["ids"], s["nseq"] = _ids(c, d), max(1, c["nseq"])
            s["init"] = d.normal(c["batch"], s["nseq"], w - 1, n, dtype=dt) if c["nseq"] > 0 else None
        else:
            s["state"] = d.normal(c["batch"], w - 1, n, dtype=dt)
    elif op in ("scan", "scan_step"):
        n, N, G = c["channels"], c["dstate"], c["ngroups"]
        lead = (c["batch"], c["seqlen"]) if op == "scan" else (c["batch"],)
        s["u"] = d.normal(*lead, n, dtype=dt)
        s["dt"] = d.normal(*lead, n, scale=0.5, shift=-0.5 if c["softplus"] else 0.0, dtype=dt)
        if not c["softplus"]:
            s["dt"] = s["dt"].float().abs_().mul_(0.1).to(dt)  # step sizes themselves: positive and small
        s["A"] = _decays(d, n, N)
        low = d.normal(*lead, c["ahead"] + 2 * G * N, scale=N ** -0.5, dtype=dt)
        s["B"] = low[..., c["ahead"]:c["ahead"] + G * N].unflatten(-1, (G, N))
        s["C"] = low[..., c["ahead"] + G * N:].unflatten(-1, (G, N))
        s["D"] = d.normal(n) if c["skip"] else None
        s["z"] = d.normal(*lead, 2 * n, dtype=dt)[..., n:] if c["gate"] else None
        s["bias"] = d.normal(n, shift=-2.5 if c["softplus"] else 0.01, scale=0.5 if c["softplus"] else 0.0) if c["bias"] else None
        s["softplus"] = c["softplus"]
        if op == "scan":
            s["ids"], s["nseq"] = _ids(c, d), max(1, c["nseq"])
            s["init"] = d.normal(c["batch"], s["nseq"], N, n) if c["nseq"] > 0 else None
        else:
            s["state"] = d.normal(c["batch"], N, n)
    else:
        lead, n = (c["batch"], c["seqlen"]), c["channels"]
        s["x"] = d.normal(*lead, n, dtype=dt)
        s["weight"] = d.normal(n, scale=0.2, shift=1.0)
        s["eps"] = 1e-5
        if op == "gated_norm":
            s["z"] = d.normal(*lead, n + c["behind"], dtype=dt)[..., :n] if c["gate"] else None
        else:
            s["residual"] = None if c["residual"] == "none" else d.normal(*lead, n, scale=3.0, dtype=DTYPES[c["residual"]])
            s["scale"] = d.normal(n, scale=0.1, shift=0.5) if c["scaled"] else 0.7
    return s


# --------------------------------------------------------------------------- #
# Plain forms, in 32 bits, rounded once at the end
# --------------------------------------------------------------------------- #

def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _positions(ids, batch, seqlen):
    """Each token's sequence id, the index of that sequence's first token, and whether it is that token."""
    t = torch.arange(seqlen, device="cuda").expand(batch, seqlen)
    if ids is None:
        first = t == 0
        return torch.zeros_like(t), torch.zeros_like(t), first
    ids = ids.long()
    first = torch.ones_like(ids, dtype=torch.bool)
    first[:, 1:] = ids[:, 1:] != ids[:, :-1]
    return ids, torch.cummax(torch.where(first, t, 0), dim=1).values, first


def _last(ids, nseq):
    """For each (row, id): whether it occurs, and its last token."""
    batch, seqlen = ids.shape
    t = torch.arange(seqlen, device="cuda").expand(batch, seqlen)
    last = torch.full((batch, nseq), -1, dtype=torch.long, device="cuda")
    last = last.scatter_reduce(1, ids, t, "amax")
    return last >= 0, last.clamp(min=0)


def _windows(s):
    """Inputs under each token's taps [b, T, width, C]: of its own sequence, from the initial window before it."""
    x, c = s["x"], s["case"]
    b, t, n = x.shape
    w = c["width"]
    ids, start, _ = _positions(s["ids"], b, t)
    init = s["init"] if s["init"] is not None else x.new_zeros(b, s["nseq"], w - 1, n)
    source = torch.cat([init.reshape(b, -1, n), x], dim=1)
    back = torch.arange(w - 1, -1, -1, device="cuda")
    pos = torch.arange(t, device="cuda")[None, :, None] - back  # the tokens under the taps
    before = pos - start[..., None]  # negative: that many tokens before the sequence's first
    at = torch.where(before >= 0, pos + s["nseq"] * (w - 1), ids[..., None] * (w - 1) + (w - 1) + before)
    return source, at, ids, init


def _plain_conv(s):
    c, x = s["case"], s["x"]
    b, t, n = x.shape
    w = c["width"]
    source, at, ids, init = _windows(s)
    rows = torch.arange(b, device="cuda")[:, None, None]
    y = (source[rows, at].float() * s["weight"].t()).sum(2)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["activation"]:
        y = _silu(y)
    # the window after a token: the inputs under its taps but the oldest
    occurs, last = _last(ids, s["nseq"])
    after = source[rows, at.gather(1, last[..., None].expand(-1, -1, w))[..., 1:]]
    final = torch.where(occurs[..., None, None], after, init)
    return _parts(y.to(x.dtype), s["splits"]), final


def _parts(y, splits):
    return [v.contiguous() for v in y.split(splits, -1)] if splits else y


def _plain_conv_step(s):
    x = s["x"]
    window = torch.cat([s["state"], x[:, None]], dim=1)
    y = (window.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["activation"]:
        y = _silu(y)
    s["state"].copy_(window[:, 1:])
    return _parts(y.to(x.dtype), s["splits"]), s["state"]


def _steps(s):
    """The recurrence's coefficients h <- a h + v: both [..., N, channels]."""
    u, dt = s["u"].float(), s["dt"].float()
    if s["bias"] is not None:
        dt = dt + s["bias"]
    if s["softplus"]:
        dt = _softplus(dt)
    per = u.shape[-1] // s["B"].shape[-2]
    a = torch.exp(dt[..., None, :] * s["A"].t())
    B = s["B"].float().transpose(-1, -2).repeat_interleave(per, -1)
    return a, B * (dt * u)[..., None, :], u, per


def _read_out(s, h, u, per):
    y = (h * s["C"].float().transpose(-1, -2).repeat_interleave(per, -1)).sum(-2)
    if s["D"] is not None:
        y = y + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["u"].dtype)


def _plain_scan(s):
    u = s["u"]
    b, t, n = u.shape
    a, h, uf, per = _steps(s)
    ids, _, first = _positions(s["ids"], b, t)
    N = a.shape[2]
    init = s["init"] if s["init"] is not None else torch.zeros(b, s["nseq"], N, n, device="cuda")
    # a sequence's first token takes its initial state in, and nothing of the token before it
    rows = torch.arange(b, device="cuda")[:, None].expand(b, t)
    h[first] += a[first] * init[rows[first], ids[first]]
    a[first] = 0.0
    # all prefixes at once, by doubling the span that each token's (a, h) stands for
    k = 1
    while k < t:
        h[:, k:] += a[:, k:] * h[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    occurs, last = _last(ids, s["nseq"])
    final = torch.where(occurs[..., None, None], h[torch.arange(b, device="cuda")[:, None], last], init)
    return _read_out(s, h, uf, per), final


def _plain_scan_step(s):
    a, v, u, per = _steps(s)
    s["state"].mul_(a).add_(v)
    return _read_out(s, s["state"], u, per), s["state"]


def _plain_gated_norm(s):
    x, z, g = s["x"].float(), s["z"], s["case"]["ngroups"]
    if z is not None and s["case"]["gate_first"]:
        x = x * _silu(z.float())
    y = x.unflatten(-1, (g, -1))
    y = (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"])).flatten(-2) * s["weight"]
    if z is not None and not s["case"]["gate_first"]:
        y = y * _silu(z.float())
    return y.to(s["x"].dtype)


def _plain_add_norm(s):
    r = s["x"].float() * s["scale"]
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    return y.to(s["x"].dtype), r.to(torch.float32 if s["residual"] is None else s["residual"].dtype)


_PLAIN = dict(conv=_plain_conv, conv_step=_plain_conv_step, scan=_plain_scan, scan_step=_plain_scan_step,
              gated_norm=_plain_gated_norm, add_norm=_plain_add_norm)


# --------------------------------------------------------------------------- #
# One pass
# --------------------------------------------------------------------------- #

def _own_run(s):
    import mamba_ssd_layer_chunked_b200 as ssd
    op = s["case"]["op"]
    if op == "conv":
        return ssd.causal_conv(s["x"], s["weight"], s["bias"], init_states=s["init"], seq_idx=s["ids"],
                               nseq=s["nseq"], activation=s["activation"], splits=s["splits"])
    if op == "conv_step":
        return ssd.conv_step(s["x"], s["state"], s["weight"], s["bias"], activation=s["activation"],
                             splits=s["splits"]), s["state"]
    if op == "scan":
        return ssd.selective_scan(s["u"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["bias"],
                                  dt_softplus=s["softplus"], init_states=s["init"], seq_idx=s["ids"], nseq=s["nseq"])
    if op == "scan_step":
        return ssd.selective_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                                  dt_bias=s["bias"], dt_softplus=s["softplus"]), s["state"]
    if op == "gated_norm":
        return ssd.gated_norm(s["x"], s["weight"], z=s["z"], ngroups=s["case"]["ngroups"], eps=s["eps"],
                              gate_first=s["case"]["gate_first"])
    return ssd.add_norm(s["x"], s["weight"], residual=s["residual"], scale=s["scale"], eps=s["eps"])


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------- #
# What a pass cannot do without
# --------------------------------------------------------------------------- #

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    op, n = c["op"], c["channels"]
    rows = c["batch"] * c.get("seqlen", 1)
    if op in ("conv", "conv_step"):
        w, per = c["width"], 2 * c["width"] + (5 if c["silu"] else 0)
        params = 4 * n * (w + c["bias"])
        window = c["batch"] * (w - 1) * n * e
        if op == "conv_step":
            return dict(bytes=2 * rows * n * e + 2 * window + params, flops=rows * n * per)
        windows = window * max(1, c["nseq"]) * (2 if c["nseq"] else 1) + (4 * rows if c["nseq"] else 0)
        return dict(bytes=2 * rows * n * e + windows + params, flops=rows * n * per)
    if op in ("scan", "scan_step"):
        N = c["dstate"]
        # per channel and state: dt A, its exp, v B, the recurrence's and the read-out's multiply-adds
        flops = rows * n * (7 * N + 1 + 5 * c["softplus"] + c["bias"] + 2 * c["skip"] + 6 * c["gate"])
        params = 4 * n * (N + c["skip"] + c["bias"])
        state = 4 * c["batch"] * N * n
        if op == "scan":
            state *= max(1, c["nseq"]) * (2 if c["nseq"] else 1)
        else:
            state *= 2
        ids = 4 * rows if c.get("nseq", 0) else 0
        return dict(bytes=rows * ((3 + c["gate"]) * n + 2 * c["ngroups"] * N) * e + params + state + ids, flops=flops)
    if op == "gated_norm":
        return dict(bytes=rows * n * e * (2 + c["gate"]) + 4 * n, flops=rows * n * (4 + 6 * c["gate"]))
    r = {"f32": 4, "bf16": 2, "none": 4}[c["residual"]]
    moved = rows * n * (2 * e + (1 if c["residual"] == "none" else 2) * r)
    return dict(bytes=moved + 4 * n * (1 + c["scaled"]), flops=rows * n * 6)


# --------------------------------------------------------------------------- #
# The definitions in 64 bits
# --------------------------------------------------------------------------- #

def _spans(s, row, seqlen):
    """(id, first token, end) of a row's sequences, in order."""
    if s["ids"] is None:
        return [(0, 0, seqlen)]
    ids = s["ids"][row].tolist()
    cuts = [0] + [t for t in range(1, seqlen) if ids[t] != ids[t - 1]] + [seqlen]
    return [(ids[a], a, e) for a, e in zip(cuts[:-1], cuts[1:])]


def _gate64(z):
    return z * torch.sigmoid(z)


def _exact_conv(s):
    x, weight = s["x"].double(), s["weight"].double()
    b, t, n = x.shape
    w = weight.shape[1]
    y = torch.empty_like(x)
    final = torch.zeros(b, s["nseq"], w - 1, n, dtype=torch.float64, device="cuda")
    if s["init"] is not None:
        final.copy_(s["init"])
    for row in range(b):
        for k, first, end in _spans(s, row, t):
            seen = torch.cat([final[row, k], x[row, first:end]])
            acc = seen[w - 1:] * weight[:, w - 1]
            for tap in range(w - 1):
                acc += seen[tap:tap + end - first] * weight[:, tap]
            y[row, first:end] = acc
            final[row, k] = seen[end - first:]
    if s["bias"] is not None:
        y += s["bias"].double()
    return _parts(_gate64(y) if s["activation"] else y, s["splits"]), final


def _exact_conv_step(s):
    x, state, weight = s["x"].double(), s["state"].double(), s["weight"].double()
    w = weight.shape[1]
    y = x * weight[:, w - 1] + torch.einsum("bwc,cw->bc", state, weight[:, :w - 1])
    if s["bias"] is not None:
        y += s["bias"].double()
    return _parts(_gate64(y) if s["activation"] else y, s["splits"]), torch.cat([state, x[:, None]], 1)[:, 1:]


def _recur64(s, t, h):
    """One token of the definition on h [..., channels, N]; returns the token's output."""
    at = (lambda v: v[:, t]) if t is not None else (lambda v: v)
    u, dt = at(s["u"]).double(), at(s["dt"]).double()
    if s["bias"] is not None:
        dt = dt + s["bias"].double()
    if s["softplus"]:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    per = u.shape[-1] // s["B"].shape[-2]
    B = at(s["B"]).double().repeat_interleave(per, 1)
    C = at(s["C"]).double().repeat_interleave(per, 1)
    h *= torch.exp(dt[..., None] * s["A"].double())
    h += (dt * u)[..., None] * B
    y = torch.einsum("bcn,bcn->bc", h, C)
    if s["D"] is not None:
        y += s["D"].double() * u
    if s["z"] is not None:
        y *= _gate64(at(s["z"]).double())
    return y


def _exact_scan(s):
    b, t, n = s["u"].shape
    y = torch.empty(b, t, n, dtype=torch.float64, device="cuda")
    N = s["A"].shape[1]
    final = torch.zeros(b, s["nseq"], N, n, dtype=torch.float64, device="cuda")
    if s["init"] is not None:
        final.copy_(s["init"])
    starts, ends = {}, {}
    for row in range(b):
        for k, first, end in _spans(s, row, t):
            starts.setdefault(first, []).append((row, k))
            ends.setdefault(end - 1, []).append((row, k))
    h = torch.zeros(b, n, N, dtype=torch.float64, device="cuda")
    for token in range(t):
        for row, k in starts.get(token, ()):
            h[row] = final[row, k].t()
        y[:, token] = _recur64(s, token, h)
        for row, k in ends.get(token, ()):
            final[row, k] = h[row].t()
    return y, final


def _exact_scan_step(s):
    h = s["state"].double().transpose(1, 2).contiguous()
    y = _recur64(s, None, h)
    return y, h.transpose(1, 2).contiguous()


def _rms64(v, eps):
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)


def _exact_gated_norm(s):
    c, x = s["case"], s["x"].double()
    gate = 1.0 if s["z"] is None else _gate64(s["z"].double())
    if c["gate_first"]:
        x = x * gate
    y = torch.cat([_rms64(v, s["eps"]) for v in x.chunk(c["ngroups"], -1)], -1) * s["weight"].double()
    return y if c["gate_first"] else y * gate


def _exact_add_norm(s):
    scale = s["scale"].double() if torch.is_tensor(s["scale"]) else s["scale"]
    r = s["x"].double() * scale + (0.0 if s["residual"] is None else s["residual"].double())
    return _rms64(r, s["eps"]) * s["weight"].double(), r


_EXACT = dict(conv=_exact_conv, conv_step=_exact_conv_step, scan=_exact_scan, scan_step=_exact_scan_step,
              gated_norm=_exact_gated_norm, add_norm=_exact_add_norm)


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
