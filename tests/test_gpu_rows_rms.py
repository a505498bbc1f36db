"""A second bound on the products over grouped rows: the root mean square of
the error over all outputs.

The bounds of the other tests are worst cases over the sum's terms, so a middle
product or a weight rounded once more could hide in them.  An output that is
rounded once to fp16 is off by an error spread evenly over +- half a step, a
mean square of 1/12 step^2.  The fp32 sums add at most 2^-23 sum |terms| a term
in the worst case and about sqrt(terms) 2^-24 of the result's own size as a rule,
less than 2^-18 of it for the sizes here where half a step is 2^-12 to 2^-11: a
mean square below 1 % of the rounding's.  Taken over N = 10^5 outputs the mean
itself scatters by 0.9 / sqrt(N) = 0.3 %.  So the mean square lies within 5 % of
1/12 step^2.  A second rounding to fp16, of the middle products or of the
weights, adds a mean square of the same size: a factor of 2.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev
from packed_bit_weight_b200 import qmm, synth
from rows_util import expert_products, lora

pytestmark = pytest.mark.gpu


def _one_rounding(got, ref):
    """Mean square error over the mean of step^2 / 12 (normal fp16 values)."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(ref), 2.0 ** -14))), -14) - 10)
    assert ref.size >= 50_000
    return float(((got - ref) ** 2).mean() / (step ** 2 / 12).mean())


@pytest.mark.parametrize("m,n,k,R,path", [(12, 8192, 512, 64, "lora_token"), (300, 1024, 1024, 32, "lora_tiled"),
                                          (300, 1024, 512, 64, "lora_tiled"), (400, 520, 512, 128, "lora_tiled"),
                                          (100, 1024, 512, 256, "lora_tiled"), (600, 264, 512, 48, "lora_tc"),
                                          (600, 520, 1024, 128, "lora_tc")])
def test_adapters_round_once(m, n, k, R, path):
    rng = np.random.default_rng(m + n + k + R)
    L = 3
    A = (rng.standard_normal((L, R, k)) / np.sqrt(k)).astype(np.float16)
    B = rng.standard_normal((L, n, R)).astype(np.float16)
    sc = np.ones(L, np.float32)
    x, base = rng.standard_normal((m, k)).astype(np.float16), np.zeros((m, n), np.float16)
    ids = (np.arange(m) % L).astype(np.int32)
    c = lambda a: torch.from_numpy(a).cuda()
    ad = qmm.Adapters(c(A), c(B), c(sc))
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(ad, m), dtype=torch.uint8, device="cuda")
    y = torch.empty((m, n), dtype=torch.float16, device="cuda")
    qmm.qmm_lora(ad, c(x), c(ids), c(base), y, ws=ws)
    assert qmm.qmm_last_variant().startswith(path) and qmm.qmm_sync_check() == 0
    d = lambda a: a.astype(np.float64)
    ref, _ = lora(d(x), d(base), ids, d(A), d(B), sc, None)
    ratio = _one_rounding(y.cpu().numpy(), ref)
    assert 0.95 < ratio < 1.05, ratio


@pytest.mark.parametrize("k", [896, 160])
@pytest.mark.parametrize("fmt", [synth.FMT_IQ4_NL, synth.FMT_FP4G16_F16, synth.FMT_FP4G16_E4M3, synth.FMT_MXFP4])
def test_experts_products_round_once(fmt, k):
    rng = np.random.default_rng(fmt + k)
    off = np.array([0, 100, 100, 300, 420], np.int32)
    p = synth.gen_weights(rng, fmt, 264, k, experts=4)
    x = synth.gen_x(rng, 420, k)
    y = torch.empty((420, 264), dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_gemm(dev(p), torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(off).cuda(), y)
    assert qmm.qmm_sync_check() == 0
    ref, _ = expert_products(p, x, off)
    ratio = _one_rounding(y.cpu().numpy(), ref)
    assert 0.95 < ratio < 1.05, ratio
