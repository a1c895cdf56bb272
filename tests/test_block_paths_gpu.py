"""The operators around the scan on the paths that their launch rules choose by
size and alignment, against the fp64 definitions (oracle.block_oracle).
Tolerances: those of test_block_gpu, whose derivation is at its head."""
import numpy as np
import pytest

import mamba_ssd_layer_chunked_b200 as ssd
from tests.test_block_gpu import check_scan, cuda, ids_of, on_gpu, rand, scan_inputs, scan_reference

pytestmark = pytest.mark.gpu


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
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("c,N,G,dt", [(12, 16, 1, "f32"), (4, 12, 1, "f32"), (1540, 16, 1, "f32"), (24, 16, 2, "f32"),
                                      (20, 8, 1, "f32"), (24, 8, 1, "f32"), (28, 4, 1, "f32"), (2436, 8, 1, "f32"),
                                      (24, 8, 1, "bf16"), (8, 8, 1, "bf16"), (48, 8, 2, "bf16"), (2440, 8, 1, "bf16")])
def test_scan_of_partial_units(c, N, G, dt, packed):
    T = 77
    run_scan(np.random.default_rng(c + N), 1, T, c, N, G, dt, [[30, 47]] if packed else None)
