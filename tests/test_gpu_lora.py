"""GPU parity of the low-rank adapters against the definition in double."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from packed_bit_weight_b200 import qmm, synth
from rows_util import lora, within

pytestmark = pytest.mark.gpu


def _pool(rng, L, R, n, k, ranks=False):
    A = (rng.standard_normal((L, R, k)) / np.sqrt(max(k, 1))).astype(np.float16)
    B = (rng.standard_normal((L, n, R)) * 0.2).astype(np.float16)
    scales = rng.uniform(0.1, 2.0, L).astype(np.float32)
    rk = rng.integers(0, R + 1, L).astype(np.int32) if ranks else None
    if ranks:
        rk[0] = R
        for a in range(L):             # what a rank leaves out is never used
            A[a, rk[a]:] = np.nan
            B[a][:, rk[a]:] = np.inf
    return A, B, scales, rk


def _adapters(A, B, scales, rk):
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()
    return qmm.Adapters(c(A), c(B), c(scales), c(rk))


def _run(ad, x, ids, base, inplace=False):
    c = lambda a: torch.from_numpy(a).cuda()
    b = c(base)
    y = b if inplace else torch.full_like(b, 7.0)
    nb = qmm.qmm_lora_workspace_bytes(ad, ids.size)
    ws = torch.full((nb + 256,), 0x7F, dtype=torch.uint8, device="cuda")   # NaN patterns: nothing stale is used
    qmm.qmm_lora(ad, c(x), c(ids), b, y, ws=ws[:nb])
    assert (ws[nb:] == 0x7F).all()
    return y


def _d(a):
    return a.astype(np.float64)


CASES = [  # m, n, k, R, L, how ids are drawn
    (1, 16, 64, 8, 1, "one"), (1, 18560, 4096, 16, 8, "any"), (1, 40, 8, 256, 2, "any"), (2, 1001, 128, 16, 4, "any"),
    (3, 7, 520, 24, 4, "any"), (5, 264, 4096, 64, 3, "none"), (8, 512, 1024, 32, 8, "distinct"),
    (16, 4096, 2048, 64, 16, "distinct"), (16, 999, 136, 40, 2, "any"), (17, 130, 896, 128, 5, "any"),
    (33, 520, 264, 8, 40, "any"), (64, 777, 512, 96, 1, "one"), (70, 264, 2560, 256, 3, "runs"),
    (128, 1024, 256, 16, 130, "distinct"), (300, 1096, 904, 64, 7, "runs"), (513, 260, 1024, 48, 9, "any"),
    (1100, 333, 384, 128, 2, "runs"), (600, 1000, 256, 8, 3, "any"), (1500, 640, 128, 40, 30, "runs"),
    (777, 129, 64, 72, 300, "any"), (520, 4104, 128, 120, 1, "one"), (640, 256, 64, 136, 3, "any")]


def _ids(rng, m, L, how):
    if how == "one":
        return np.zeros(m, np.int32)
    if how == "none":
        return np.full(m, -1, np.int32)
    if how == "distinct":
        return rng.permutation(L)[:m].astype(np.int32)
    ids = rng.integers(-1, L, m).astype(np.int32)
    return np.sort(ids) if how == "runs" else ids


@pytest.mark.parametrize("ranks", [False, True])
@pytest.mark.parametrize("m,n,k,R,L,how", CASES)
def test_lora(m, n, k, R, L, how, ranks):
    rng = np.random.default_rng(m + n + R)
    A, B, sc, rk = _pool(rng, L, R, n, k, ranks)
    x, base = rng.standard_normal((m, k)).astype(np.float16), rng.standard_normal((m, n)).astype(np.float16)
    ids = _ids(rng, m, L, how)
    x[ids < 0] = np.nan                        # rows without an adapter are not multiplied
    y = _run(_adapters(A, B, sc, rk), x, ids, base)
    assert qmm.qmm_sync_check() == 0
    ref, bound = lora(_d(x), _d(base), ids, _d(A), _d(B), sc, rk)
    within(y.cpu().numpy(), ref, bound, qmm.qmm_last_variant())
    y2 = _run(_adapters(A, B, sc, rk), x, ids, base, inplace=True)
    assert torch.equal(y2, y)                  # in place, and the same bits again


@pytest.mark.parametrize("m", [1, 9, 100, 300, 700])
def test_bad_ids_and_ranks_are_reported(m):
    rng = np.random.default_rng(m)
    R = 48 if m >= 512 else 16                  # (on the tensor-core product from 512 rows)
    A, B, sc, _ = _pool(rng, 3, R, 72, 64)
    rk = np.array([R, 99, -3], np.int32)        # clamped: all of it, all of it, none
    x, base = rng.standard_normal((m, 64)).astype(np.float16), rng.standard_normal((m, 72)).astype(np.float16)
    ids = np.array([[3, -2, 0][i % 3] for i in range(m)], np.int32)
    ad = _adapters(A, B, sc, None)
    y = _run(ad, x, ids, base)
    assert qmm.qmm_sync_check() == 7
    within(y.cpu().numpy(), *lora(_d(x), _d(base), ids, _d(A), _d(B), sc, None))
    ids = np.array([[1, 2, 0][i % 3] for i in range(m)], np.int32)
    y = _run(_adapters(A, B, sc, rk), x, ids, base)
    assert qmm.qmm_sync_check() == 7
    within(y.cpu().numpy(), *lora(_d(x), _d(base), ids, _d(A), _d(B), sc, rk))


@pytest.mark.parametrize("m", [2, 70, 600])
def test_values_outside_fp16_between_the_products(m):
    """A x beyond fp16's range and below its smallest step, brought back by B
    and the scale: the middle product is held in fp32."""
    rng = np.random.default_rng(3)
    L, R, n, k = 2, 48 if m >= 512 else 16, 64, 512
    A = np.ones((L, R, k), np.float16) * np.float16(400.0)
    A[1] = np.float16(2.0 ** -20)
    x = np.abs(rng.standard_normal((m, k)) + 2).astype(np.float16)
    x[1::2] = x[1::2] * np.float16(2.0 ** -8)
    B = (rng.standard_normal((L, n, R))).astype(np.float16)
    sc = np.array([2.0 ** -16, 2.0 ** 14], np.float32)
    base = np.zeros((m, n), np.float16)
    ids = (np.arange(m) % 2).astype(np.int32)
    y = _run(_adapters(A, B, sc, None), x, ids, base)
    within(y.cpu().numpy(), *lora(_d(x), _d(base), ids, _d(A), _d(B), sc, None))


@pytest.mark.parametrize("m", [2, 40, 300, 700])
def test_infinities_and_nan_stay_in_their_row(m):
    rng = np.random.default_rng(4)
    A, B, sc, _ = _pool(rng, 2, 48 if m >= 512 else 32, 136, 256)
    x, base = rng.standard_normal((m, 256)).astype(np.float16), rng.standard_normal((m, 136)).astype(np.float16)
    ids = (np.arange(m) % 2).astype(np.int32)
    x[0, 5] = np.nan
    base[1, 7] = np.inf
    y = _run(_adapters(A, B, sc, None), x, ids, base).cpu().numpy()
    assert np.isnan(y[0]).all() and y[1, 7] == np.inf
    x[0], base[1, 7] = 0, 0
    ref, bound = lora(_d(x), _d(base), ids, _d(A), _d(B), sc, None)
    ref[1, 7], bound[1, 7] = np.inf, 0
    within(y[1:], ref[1:], bound[1:])


def test_an_infinite_middle_product_gives_what_fp32_gives():
    """An infinity in x: A x is +-inf, and the outputs are +-inf or NaN where
    infinities of both signs (or 0 * inf) meet."""
    for m in (1, 70, 600):
        L, R, n, k = 1, 40 if m >= 512 else 8, 16, 64
        A, B = np.ones((L, R, k), np.float16), np.ones((L, n, R), np.float16)
        B[0, 1] = -1
        B[0, 2, :4] = -1
        B[0, 3, 0] = 0
        x = np.ones((m, k), np.float16)
        x[0, 0] = np.inf
        y = _run(_adapters(A, B, np.ones(1, np.float32), None), x, np.zeros(m, np.int32),
                 np.zeros((m, n), np.float16)).cpu().numpy()
        assert y[0, 0] == np.inf and y[0, 1] == -np.inf and np.isnan(y[0, 2:4]).all() and (y[0, 4:] == np.inf).all()
        assert np.isfinite(y[1:]).all()


@pytest.mark.parametrize("m,R", [(3, 16), (70, 16), (600, 16), (600, 72)])
def test_strided_pool_and_shifted_buffers(m, R):
    """Adapters further apart than their size; base and y 16 bytes into an
    allocation (aligned to 16, not to 32)."""
    rng = np.random.default_rng(6)
    n = 80
    A, B, sc, _ = _pool(rng, 4, R, n, 64)
    big_a, big_b = np.full((4, R + 8, 64), np.nan, np.float16), np.full((4, n + 8, R), np.nan, np.float16)
    big_a[:, :R], big_b[:, :n] = A, B
    ad = qmm.Adapters(torch.from_numpy(big_a).cuda()[:, :R], torch.from_numpy(big_b).cuda()[:, :n],
                      torch.from_numpy(sc).cuda())
    x, base = rng.standard_normal((m, 64)).astype(np.float16), rng.standard_normal((m, n)).astype(np.float16)
    ids = _ids(rng, m, 4, "any")
    ref, bound = lora(_d(x), _d(base), ids, _d(A), _d(B), sc, None)
    y = _run(ad, x, ids, base)
    within(y.cpu().numpy(), ref, bound)
    buf = torch.full((m * n + 24,), 7.0, dtype=torch.float16, device="cuda")
    shifted = buf[8:8 + m * n].view(m, n)
    shifted.copy_(torch.from_numpy(base))
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(ad, m), dtype=torch.uint8, device="cuda")
    qmm.qmm_lora(ad, torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), shifted, shifted, ws=ws)
    assert torch.equal(shifted, y)
    assert bool((buf[:8] == 7).all()) and bool((buf[8 + m * n:] == 7).all())


@pytest.mark.parametrize("m", [40, 600])
def test_every_rank_of_a_pool(m):
    """Ranks 0 .. R one adapter each, what they leave out not a number."""
    rng = np.random.default_rng(m)
    R, n, k = 64, 136, 72
    A, B, sc, _ = _pool(rng, R + 1, R, n, k)
    rk = np.arange(R + 1, dtype=np.int32)
    for a in range(R + 1):
        A[a, a:], B[a][:, a:] = np.nan, np.nan
    x, base = rng.standard_normal((m, k)).astype(np.float16), rng.standard_normal((m, n)).astype(np.float16)
    ids = (np.arange(m) % (R + 1)).astype(np.int32)
    y = _run(_adapters(A, B, sc, rk), x, ids, base)
    assert qmm.qmm_sync_check() == 0
    within(y.cpu().numpy(), *lora(_d(x), _d(base), ids, _d(A), _d(B), sc, rk), qmm.qmm_last_variant())


def test_zero_sizes():
    rng = np.random.default_rng(7)
    A, B, sc, _ = _pool(rng, 2, 16, 72, 64)
    ad = _adapters(A, B, sc, None)
    e = torch.empty((0, 72), dtype=torch.float16, device="cuda")
    qmm.qmm_lora(ad, torch.empty((0, 64), dtype=torch.float16, device="cuda"),
                 torch.empty(0, dtype=torch.int32, device="cuda"), e, e)
    for R, k in ((0, 64), (16, 0)):            # an empty sum: y = base
        A, B, sc, _ = _pool(rng, 2, R, 72, k)
        for m in (3, 70, 600):
            base = rng.standard_normal((m, 72)).astype(np.float16)
            y = _run(_adapters(A, B, sc, None), np.zeros((m, k), np.float16), _ids(rng, m, 2, "any"), base)
            assert np.array_equal(y.cpu().numpy(), base)
    assert qmm.qmm_sync_check() == 0


@pytest.mark.parametrize("m", [4, 200, 530])
def test_beside_a_packed_projection_on_two_streams_and_in_a_graph(m):
    """The projection and its adapters in place, as a server runs them: on two
    streams at once with a workspace each, and captured and replayed."""
    rng = np.random.default_rng(11)
    n, k, L, R = 520, 512, 5, 32
    p = synth.gen_weights(rng, synth.FMT_FP4G16_F16, n, k)
    w = dev(p)
    A, B, sc, rk = _pool(rng, L, R, n, k, True)
    ad = _adapters(A, B, sc, rk)
    xs = [torch.from_numpy(rng.standard_normal((m, k)).astype(np.float16)).cuda() for _ in range(4)]
    idss = [torch.from_numpy(_ids(rng, m, L, "any")).cuda() for _ in range(4)]

    def step(x, ids, y, ws):
        (qmm.qmm_gemv if m <= 16 else qmm.qmm_gemm)(w, x, y)
        qmm.qmm_lora(ad, x, ids, y, y, ws=ws)

    new_ws = lambda: torch.empty(qmm.qmm_lora_workspace_bytes(ad, m), dtype=torch.uint8, device="cuda")
    want = []
    for x, ids in zip(xs, idss):
        base = torch.empty((m, n), dtype=torch.float16, device="cuda")
        (qmm.qmm_gemv if m <= 16 else qmm.qmm_gemm)(w, x, base)
        ref, bound = lora(_d(x.cpu().numpy()), _d(base.cpu().numpy()), ids.cpu().numpy(), _d(A), _d(B), sc, rk)
        y = torch.empty_like(base)
        step(x, ids, y, new_ws())
        within(y.cpu().numpy(), ref, bound)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    ys, wss = [torch.empty_like(want[0]) for _ in range(4)], [new_ws() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, ids, y, ws in zip(streams, xs, idss, ys, wss):
            with torch.cuda.stream(s):
                step(x, ids, y, ws)
    torch.cuda.synchronize()
    for y, v in zip(ys, want):
        assert torch.equal(y, v)
    x, ids, y, ws = xs[0].clone(), idss[0].clone(), torch.empty_like(want[0]), new_ws()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, ids, y, ws)
    for i in (2, 0, 3, 1):
        x.copy_(xs[i])
        ids.copy_(idss[i])
        graph.replay()
        assert torch.equal(y, want[i])
    assert qmm.qmm_sync_check() == 0
