"""Buffers of more than 2^31 values: the row operators' and the adapters'
offsets pass 32 bits.  Rows from all over are compared with the definition."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from packed_bit_weight_b200 import qmm, synth
from rows_util import expert_products, lora, product_bound, within

pytestmark = pytest.mark.gpu


def _rows(g, m):
    """A few rows of all parts of [0, m), the ends among them."""
    r = torch.randint(0, m, (40,), generator=g).tolist() + [0, 1, m - 2, m - 1]
    return sorted(set(r))


def _values(m, n, seed):
    """[m][n] fp16 values on the GPU, made row block by row block."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty((m, n), dtype=torch.float16, device="cuda")
    for i in range(0, m, 16384):
        out[i:i + 16384].normal_(generator=g)
    return out


@pytest.mark.parametrize("R", [8, 40, 136])
def test_adapters(R):
    g = torch.Generator().manual_seed(R)
    rng = np.random.default_rng(R)
    m, n, k, L = 117_000, 18_560, 64, 3
    assert m * n > 2 ** 31
    A, B = rng.standard_normal((L, R, k)).astype(np.float16), rng.standard_normal((L, n, R)).astype(np.float16)
    sc = np.full(L, 0.25, np.float32)
    c = lambda a: torch.from_numpy(a).cuda()
    ad = qmm.Adapters(c(A), c(B), c(sc))
    x = rng.standard_normal((m, k)).astype(np.float16)
    ids = rng.integers(-1, L, m).astype(np.int32)
    y = _values(m, n, R)
    at = _rows(g, m)
    base = y[at].cpu().numpy()
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(ad, m), dtype=torch.uint8, device="cuda")
    qmm.qmm_lora(ad, c(x), c(ids), y, y, ws=ws)
    assert qmm.qmm_sync_check() == 0
    d = lambda a: a.astype(np.float64)
    within(y[at].cpu().numpy(), *lora(d(x[at]), d(base), ids[at], d(A), d(B), sc, None), qmm.qmm_last_variant())


def test_sort_and_back_with_gradients():
    g = torch.Generator().manual_seed(1)
    t, topk, E, d = 66_000, 8, 64, 4096
    P = t * topk
    assert P * d > 2 ** 31
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(200)]).to(torch.int32)
    ids = ids.repeat(t // 200, 1).contiguous().cuda()
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm, rows = torch.empty(P, dtype=torch.int32, device="cuda"), torch.empty((t, topk), dtype=torch.int32, device="cuda")
    qmm.qmm_route_rows(ids, E, off, perm, rows)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    assert torch.equal(perm.long(), order)
    x = _values(t, d, 2)
    xs = torch.empty((P, d), dtype=torch.float16, device="cuda")
    qmm.qmm_permute(x, rows, xs)
    for r in _rows(g, P):
        assert torch.equal(xs[r], x[int(perm[r]) // topk])
    w = torch.rand((t, topk), generator=g).cuda()
    out, dx = torch.empty_like(x), torch.empty_like(x)
    qmm.qmm_unpermute(xs, rows, w, out)
    qmm.qmm_permute_backward(xs, rows, dx)
    for i in _rows(g, t):                                  # every slot holds x[i]
        want = x[i].double() * w[i].double().sum()
        assert bool(((out[i].double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -20 * x[i].double().abs()
                     + 2.0 ** -25).all())
        assert torch.equal(dx[i], (x[i].double() * topk).half())
    del out, dx
    dys, dw = torch.empty_like(xs), torch.empty((t, topk), device="cuda")
    qmm.qmm_unpermute_backward(x, xs, rows, w, dys, dw)
    for r in _rows(g, P):
        p = int(perm[r])
        i = p // topk
        assert torch.equal(dys[r], (x[i].float() * w.reshape(-1)[p]).half())
        sq = float((x[i].double() ** 2).sum())
        assert abs(float(dw.reshape(-1)[p]) - sq) <= d * 2.0 ** -24 * sq
    assert qmm.qmm_sync_check() == 0


def test_experts_products():
    rng = np.random.default_rng(5)
    g = torch.Generator().manual_seed(5)
    rows, n, k, E = 850_000, 2_560, 2_560, 2
    assert rows * k > 2 ** 31 and rows * n > 2 ** 31
    p = synth.gen_iq4nl(rng, n, k, E)
    x = _values(rows, k, 6)
    off = np.array([0, 400_123, rows], np.int32)
    y = torch.empty((rows, n), dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_gemm(dev(p), x, torch.from_numpy(off).cuda(), y)
    assert qmm.qmm_sync_check() == 0
    at = _rows(g, rows)
    few = np.searchsorted(np.asarray(at), off).astype(np.int32)
    ref, a = expert_products(p, x[at].cpu().numpy().view(np.uint16), few)
    within(y[at].cpu().numpy(), ref, product_bound(ref, a, k), qmm.qmm_last_variant())
