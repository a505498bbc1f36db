"""Host side of the adapters, without a GPU: workspace sizes and the binding's
checks."""
import ctypes

import pytest
import torch

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


def test_bfloat16_is_refused_where_values_are_calculated_with():
    """Its bits would be taken for fp16.  (Refused before the device is looked
    at; 16-bit integers hold fp16 bits and get further.)"""
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)
    bf = lambda *s: z(*s, dt=torch.bfloat16)
    rows, off = z(8, 2, dt=torch.int32), z(5, dt=torch.int32)
    db = qmm.qmm_data_bytes(1, 64, 256)
    w = qmm.PackedWeights(1, 64, 256, torch.zeros(4 * db, dtype=torch.uint8), None, 1.0, 4)
    g = z(8, 2, dt=torch.float32)

    def refused(what, fn, *args):
        with pytest.raises(ValueError, match="%s is bfloat16" % what):
            fn(*args)

    refused("dxs", qmm.qmm_permute_backward, bf(16, 64), rows, z(8, 64))
    refused("ys", qmm.qmm_unpermute, bf(16, 64), rows, g, z(8, 64))
    refused("dout", qmm.qmm_unpermute_backward, bf(8, 64), z(16, 64), rows, g, z(16, 64), g)
    refused("a", qmm.Adapters(bf(4, 16, 256), z(4, 64, 16), z(4, dt=torch.float32)).desc)
    for dt in (torch.float16, torch.int16):
        with pytest.raises(ValueError, match="CUDA"):
            qmm.qmm_permute_backward(z(16, 64, dt=dt), rows, z(8, 64))
        with pytest.raises(ValueError, match="CUDA"):
            qmm.Adapters(z(4, 16, 256, dt=dt), z(4, 64, 16), z(4, dt=torch.float32)).desc()
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_permute(bf(8, 64), rows, bf(16, 64))       # copied: any 2-byte type


def test_packed_weights_of_another_size_at_the_same_address_are_checked_again():
    """As many scales, at the same address, in half the bytes."""
    n, k, E = 64, 256, 2
    fmt = qmm.FMT_FP4G16_F16
    data = torch.zeros(E * qmm.qmm_data_bytes(fmt, n, k), dtype=torch.uint8)
    scales = torch.zeros(E * n * k // 16, dtype=torch.float16)
    w = qmm.PackedWeights(fmt, n, k, data, scales, 1.0, E)
    assert w.desc().expert_scale_stride == scales.nbytes // E
    w.scales = scales.view(torch.uint8)[:scales.numel()]
    assert w.scales.data_ptr() == scales.data_ptr() and w.scales.numel() == scales.numel()
    with pytest.raises(ValueError, match="scales holds"):
        w.desc()
    w.scales = scales
    assert w.desc().expert_scale_stride == scales.nbytes // E
