"""Calls from two host threads at once (each with its own stream and buffers)."""
import threading

import numpy as np
import pytest
import torch

from gpu_util import dev
from packed_bit_weight_b200 import qmm, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ks", [(256, 5120), (128, 1920)])
def test_iq4_products_of_different_length(ks):
    """One kernel instantiation with little and with much shared memory."""
    rng = np.random.default_rng(ks[1])
    jobs, errors = [], []
    for k in ks:
        w = dev(synth.gen_iq4nl(rng, 64, k))
        x = torch.from_numpy(synth.gen_x(rng, 1, k).view(np.int16)).cuda()
        want, y = (torch.zeros((1, 64), dtype=torch.int16, device="cuda") for _ in range(2))
        qmm.qmm_gemv(w, x, want)
        jobs.append((w, x, y, want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(w, x, y, want, stream):
        try:
            torch.cuda.set_device(0)
            for _ in range(3000):
                qmm.qmm_gemv(w, x, y, stream=stream)
        except Exception as e:                                 # noqa: BLE001 (shown below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for j in jobs:
        assert torch.equal(j[2], j[3])
    assert qmm.qmm_sync_check() == 0
