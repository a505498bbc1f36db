"""IQ4_NL products at and just past the longest k of the tile kernel."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import check_tol, dev, run_gemv
from packed_bit_weight_b200 import qmm, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k,tile", [(4864, True), (5120, True), (5376, False), (5632, False)])
@pytest.mark.parametrize("m", [1, 5])
def test_plain(k, tile, m):
    rng = np.random.default_rng(k + m)
    p, x = synth.gen_iq4nl(rng, 72, k), synth.gen_x(rng, m, k)
    y = run_gemv(dev(p), x)
    assert qmm.qmm_last_variant().startswith("iq4_tile") == tile, qmm.qmm_last_variant()
    check_tol(y, *oracle.matmul(synth.FMT_IQ4_NL, 72, k, p.data, None, 1.0, x), qmm.qmm_last_variant())


@pytest.mark.parametrize("k", [5120, 5376])
def test_routed(k):
    rng = np.random.default_rng(k)
    E, n, t, topk = 3, 48, 4, 2
    p, x = synth.gen_iq4nl(rng, n, k, E), synth.gen_x(rng, t, k)
    ids = torch.tensor([[0, 2], [2, 1], [1, 0], [2, 0]], dtype=torch.int32, device="cuda")
    y = torch.empty((t * topk, n), dtype=torch.int16, device="cuda")
    w = dev(p)
    ws = torch.empty(qmm.qmm_workspace_bytes(qmm.OP_GROUPED, w, 0, t, topk), dtype=torch.uint8, device="cuda")
    qmm.qmm_grouped_gemv(w, torch.from_numpy(x.view(np.int16)).cuda(), ids, y, ws=ws)
    assert qmm.qmm_sync_check() == 0
    for j, e in enumerate(ids.reshape(-1).tolist()):
        de = p.data[e * p.data_stride:(e + 1) * p.data_stride]
        ref = oracle.matmul(synth.FMT_IQ4_NL, n, k, de, None, 1.0, x[j // topk:j // topk + 1])
        check_tol(y[j:j + 1].cpu().numpy().view(np.uint16), *ref, "expert %d" % e)
