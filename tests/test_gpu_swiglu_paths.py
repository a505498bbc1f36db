"""SwiGLU over sorted rows on its two kernels."""
import numpy as np
import pytest
import torch

from packed_bit_weight_b200 import qmm, synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def test_both_kernels_give_the_same_bits_for_the_same_sums():
    """One nonzero value of x per row, so both sums are exact whatever their
    order; k = 128 takes the tcgen05 kernel, k = 160 the generic one, and the
    values past 128 are zeros."""
    rng = np.random.default_rng(2)
    E, n, rows = 2, 512, 512
    out = {}
    mats = [synth.gen_iq4nl(rng, n, 128, E) for _ in range(2)]
    x = np.zeros((rows, 128), np.float16)
    x[np.arange(rows), rng.integers(0, 128, rows)] = (rng.standard_normal(rows) * 8).astype(np.float16)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    for k in (128, 160):
        ws = []
        for p in mats:
            w = dev(p)
            if k == 160:                  # (a fifth block of every row, its scale 0)
                d = torch.zeros(E * n, 5 * 18, dtype=torch.uint8, device="cuda")
                d[:, :4 * 18] = w.data.view(E * n, 4 * 18)
                w = qmm.PackedWeights(p.fmt, n, k, d.reshape(-1), None, 1.0, E)
            ws.append(w)
        xk = torch.zeros(rows, k, dtype=torch.float16, device="cuda")
        xk[:, :128] = torch.from_numpy(x).cuda()
        h = torch.empty(rows, n, dtype=torch.float16, device="cuda")
        qmm.qmm_grouped_swiglu(ws[0], ws[1], xk, off, h)
        assert ("tc" if k == 128 else "generic") in qmm.qmm_last_variant()
        out[k] = h
    assert qmm.qmm_sync_check() == 0
    assert bool(out[128].isfinite().all()) and float(out[128].abs().max()) > 0
    assert torch.equal(out[128], out[160])
