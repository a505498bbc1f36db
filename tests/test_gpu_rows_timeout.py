"""The bounded waits of the grouped expert product and of the adapters'
tensor-core product, made to run out without faulting anything (their TMA
loads withheld by the library's test switch): QMM_ERR_TIMEOUT once, and the
next normal call gives the right result."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from packed_bit_weight_b200 import qmm, synth
from rows_util import expert_products, lora, product_bound, within

pytestmark = pytest.mark.gpu

QMM_ERR_TIMEOUT = 6


@pytest.fixture
def debug_reset():
    yield
    qmm.qmm_debug_set(qmm.DEBUG_WITHHOLD_X_TILES, 0)
    qmm.qmm_debug_set(qmm.DEBUG_WAIT_LIMIT_NS, 2_000_000_000)


def _run_out(call, variant):
    assert qmm.qmm_sync_check() == 0
    qmm.qmm_debug_set(qmm.DEBUG_WAIT_LIMIT_NS, 1_000_000)
    qmm.qmm_debug_set(qmm.DEBUG_WITHHOLD_X_TILES, 1)
    call()
    assert qmm.qmm_last_variant().startswith(variant), qmm.qmm_last_variant()
    assert qmm.qmm_sync_check() == QMM_ERR_TIMEOUT
    assert qmm.qmm_sync_check() == 0                      # reported once, then cleared
    qmm.qmm_debug_set(qmm.DEBUG_WITHHOLD_X_TILES, 0)
    qmm.qmm_debug_set(qmm.DEBUG_WAIT_LIMIT_NS, 2_000_000_000)
    for _ in range(2):                                     # tensor memory is allocated again and again
        call()
        assert qmm.qmm_sync_check() == 0


@pytest.mark.parametrize("fmt", [synth.FMT_IQ4_NL, synth.FMT_FP4G16_F16])
def test_grouped_product(fmt, debug_reset):
    rng = np.random.default_rng(fmt)
    off = np.array([0, 300, 300, 340], np.int32)
    p = synth.gen_weights(rng, fmt, 200, 384, experts=3)
    x = synth.gen_x(rng, 340, 384)
    w, dx, do = dev(p), torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(off).cuda()
    y = torch.zeros((340, 200), dtype=torch.float16, device="cuda")
    _run_out(lambda: qmm.qmm_grouped_gemm(w, dx, do, y), "grouped_gemm_tc")
    ref, a = expert_products(p, x, off)
    within(y.cpu().numpy(), ref, product_bound(ref, a, 384))


def test_adapters(debug_reset):
    rng = np.random.default_rng(3)
    m, n, k, L, R = 530, 264, 128, 3, 48
    A, B = (rng.standard_normal((L, R, k)) * 0.1).astype(np.float16), rng.standard_normal((L, n, R)).astype(np.float16)
    sc = np.ones(L, np.float32)
    x, base = rng.standard_normal((m, k)).astype(np.float16), rng.standard_normal((m, n)).astype(np.float16)
    ids = rng.integers(-1, L, m).astype(np.int32)
    c = lambda v: torch.from_numpy(v).cuda()
    ad = qmm.Adapters(c(A), c(B), c(sc))
    dx, di, db, y = c(x), c(ids), c(base), torch.zeros((m, n), dtype=torch.float16, device="cuda")
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(ad, m), dtype=torch.uint8, device="cuda")
    _run_out(lambda: qmm.qmm_lora(ad, dx, di, db, y, ws=ws), "lora_tc")
    d = lambda v: v.astype(np.float64)
    within(y.cpu().numpy(), *lora(d(x), d(base), ids, d(A), d(B), sc, None))
