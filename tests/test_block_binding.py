"""The binding of the operators around the scan: which tensors a call on a given
stream keeps, and what importing it needs."""
import os
import subprocess
import sys

import pytest
import torch

import mamba_ssd_layer_chunked_b200 as ssd
from mamba_ssd_layer_chunked_b200 import block


def calls(device):
    """name -> (function, arguments, keyword arguments): every tensor argument given, outputs too."""
    def t(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device=device)

    b, T, c, N, W = 2, 6, 32, 4, 4
    ids = t(b, T, dtype=torch.int32)
    scan = dict(D=t(c), dt_bias=t(c))
    return {
        "causal_conv": (ssd.causal_conv, (t(b, T, c), t(c, W), t(c)),
                        dict(init_states=t(b, 1, W - 1, c), seq_idx=ids, nseq=1, splits=[20, 8, 4],
                             out=(t(b, T, 20), t(b, T, 8), t(b, T, 4)), final_out=t(b, 1, W - 1, c))),
        "causal_conv_whole": (ssd.causal_conv, (t(b, T, c), t(c, W)), dict(out=t(b, T, c))),
        "conv_step": (ssd.conv_step, (t(b, c), t(b, W - 1, c), t(c, W), t(c)),
                      dict(splits=[20, 12], out=[t(b, 20), t(b, 12)])),
        "selective_scan": (ssd.selective_scan, (t(b, T, c), t(b, T, c), t(c, N), t(b, T, 1, N), t(b, T, 1, N)),
                           dict(scan, z=t(b, T, c), init_states=t(b, 1, N, c), seq_idx=ids, nseq=1, out=t(b, T, c),
                                final_out=t(b, 1, N, c))),
        "selective_step": (ssd.selective_step, (t(b, c), t(b, c), t(c, N), t(b, 1, N), t(b, 1, N), t(b, N, c)),
                           dict(scan, z=t(b, c), out=t(b, c))),
        "gated_norm": (ssd.gated_norm, (t(b, T, c), t(c)), dict(z=t(b, T, c), out=t(b, T, c))),
        "add_norm": (ssd.add_norm, (t(b, T, c), t(c)),
                     dict(residual=t(b, T, c), scale=t(c), out=t(b, T, c), residual_out=t(b, T, c))),
    }


def tensors(values):
    for v in values:
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, (tuple, list)):
            yield from tensors(v)


NAMES = sorted(calls("cpu"))


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_of_a_call_is_recorded(name, monkeypatch):
    """Given outputs too: their memory must not be reused while the stream still writes them."""
    f, args, kw = calls("cpu")[name]
    seen = []

    class Stop(Exception):
        pass

    def record(stream, *others):
        seen.extend(tensors(others))
        raise Stop

    monkeypatch.setattr(block, "_run_on", record)
    with pytest.raises(Stop):
        f(*args, **kw)
    missing = [list(t.shape) for t in tensors((*args, *kw.values())) if not any(t is s for s in seen)]
    assert not missing


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_dropped_outputs_waits_for_the_stream(name):
    """Outputs given to a call on another stream and dropped before it runs are not handed out again."""
    f, args, kw = calls("cuda")[name]
    f(*args, **kw)  # loads the kernel, which would outlast the sleep
    given = [t for k in ("out", "final_out", "residual_out") for t in tensors([kw.get(k)])]
    # memory of its own for every given output: a block larger than any other free one
    size = 24 << 20
    big = [torch.empty(size // t.element_size() * (i + 1), dtype=t.dtype, device="cuda") for i, t in enumerate(given)]
    views = iter([m[:t.numel()].view(t.shape) for m, t in zip(big, given)])
    kw = dict(kw)
    for k in ("out", "final_out", "residual_out"):
        if k in kw:
            kw[k] = next(views) if isinstance(kw[k], torch.Tensor) else [next(views) for _ in kw[k]]
    where = {m.data_ptr() for m in big}
    sizes = [m.numel() for m in big]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    f(*args, **kw, stream=side)
    assert not side.query()  # still asleep: the call has not run yet
    del big, given, kw, views
    again = [torch.empty(n, dtype=torch.float32, device="cuda") for n in sizes]
    assert not side.query()
    assert not where & {m.data_ptr() for m in again}
    side.synchronize()
    later = [torch.empty(n, dtype=torch.float32, device="cuda") for n in sizes]
    assert where & {m.data_ptr() for m in later}  # they had been dropped: now they are handed out


def test_import_and_refusals_need_no_cuda_build_of_torch():
    """Without the functions that only a CUDA build of torch has, the package imports and refuses CPU tensors."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import mamba_ssd_layer_chunked_b200 as ssd
try:
    ssd.gated_norm(torch.zeros(2, 8), torch.zeros(8))
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("not refused")
print("refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
