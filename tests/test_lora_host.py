"""Host side of the adapters, without a GPU: workspace sizes and the binding's
checks."""
import ctypes

import pytest

from packed_bit_weight_b200 import qmm

FAKE = 1 << 40


def _pool(L, rank, n=18560, k=4096):
    d = qmm.qmm_adapters()
    d.num_adapters, d.n, d.k, d.rank = L, n, k, rank
    d.a, d.b, d.scales, d.ranks = FAKE, FAKE, FAKE, None
    d.a_stride, d.b_stride = 2 * rank * k, 2 * rank * n
    return d


@pytest.mark.parametrize("rank", [8, 16, 32, 40, 64, 128, 136, 256])
@pytest.mark.parametrize("L", [1, 3, 130, 1024])
def test_a_workspace_serves_every_smaller_call(L, rank):
    for n, k in ((18560, 4096), (64, 64)):
        d = _pool(L, rank, n, k)
        sizes = [qmm._lib().qmm_lora_workspace_bytes(ctypes.byref(d), m) for m in range(1, 1200)]
        assert sizes == sorted(sizes) and sizes[-1] > 0
