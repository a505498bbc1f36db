"""Adapters whose values or ranks are out of the ordinary, on each of their
paths (a cluster per row, sorted tiles, sorted tiles on tcgen05)."""
import threading

import numpy as np
import pytest
import torch

from packed_bit_weight_b200 import qmm
from rows_util import lora, within

pytestmark = pytest.mark.gpu

# rows, rank of the pool and the kernel that they take
PATHS = [(1, 64, "lora_token"), (70, 32, "lora_tiled"), (300, 64, "lora_tiled"), (300, 128, "lora_tiled"),
         (80, 256, "lora_tiled"), (600, 48, "lora_tc"), (600, 128, "lora_tc")]


def _c(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _run(A, B, sc, rk, x, ids, base, path):
    ad = qmm.Adapters(_c(A), _c(B), _c(sc), _c(rk))
    ws = torch.full((qmm.qmm_lora_workspace_bytes(ad, ids.size),), 0x7F, dtype=torch.uint8, device="cuda")
    y = torch.full(base.shape, 7.0, dtype=torch.float16, device="cuda")
    qmm.qmm_lora(ad, _c(x), _c(ids), _c(base), y, ws=ws)
    assert qmm.qmm_last_variant().startswith(path), qmm.qmm_last_variant()
    y2 = _c(base)
    qmm.qmm_lora(ad, _c(x), _c(ids), y2, y2, ws=ws)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))   # in place
    assert qmm.qmm_sync_check() == 0
    return y.cpu().numpy()


def _definition(x, base, ids, A, B, sc, rk):
    """(y, bound) in double; infinities and NaN have to be met exactly."""
    d = lambda v: v.astype(np.float64)
    with np.errstate(invalid="ignore"):
        y, bound = lora(d(x), d(base), ids, d(A), d(B), sc, rk)
    return y, np.where(np.isfinite(y), bound, 0.0)


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("m,R,path", PATHS)
def test_ranks_in_use_with_an_infinity_or_nan_in_x(m, R, path, value):
    """What a rank leaves out adds nothing, whatever x holds: with positive
    values an infinity in x gives +inf in every column of its row (base for a
    rank of 0), and NaN gives NaN there (base for a rank of 0)."""
    rng = np.random.default_rng(m + R)
    ranks = np.unique([0, 1, 7, 8, 17, 24, R // 2 + 1, R - 8, R - 1, R]).astype(np.int32)
    for shift in range(len(ranks) if m == 1 else 1):
        rk = np.roll(ranks, -shift).copy()
        L, n, k = rk.size, 136, 72
        A, B = np.abs(rng.standard_normal((2, L, max(R, n), max(R, k)))).astype(np.float16) + np.float16(0.25)
        A, B = np.ascontiguousarray(A[:, :R, :k]), np.ascontiguousarray(B[:, :n, :R])
        sc = np.full(L, 0.5, np.float32)
        x = (np.abs(rng.standard_normal((m, k))) + 0.25).astype(np.float16)
        base = rng.standard_normal((m, n)).astype(np.float16)
        ids = (np.arange(m) % L).astype(np.int32)
        x[:: 2 if m > 1 else 1, 5] = value
        y = _run(A, B, sc, rk, x, ids, base, path)
        within(y, *_definition(x, base, ids, A, B, sc, rk), path)
        hit = np.flatnonzero(~np.isfinite(x).all(axis=1))
        none = rk[ids[hit]] == 0
        assert np.array_equal(y[hit[none]], base[hit[none]])
        assert (np.isnan(y[hit[~none]]) if np.isnan(value) else y[hit[~none]] == np.inf).all()


@pytest.mark.parametrize("n", [401, 408, 416])
@pytest.mark.parametrize("m,R,path", PATHS)
def test_infinities_and_nan_in_b(m, R, path, n):
    """An infinity in B gives an infinity of h's sign in its column (NaN where
    two of opposite sign or 0 * inf meet), NaN gives NaN, and the other columns
    are what they were."""
    rng = np.random.default_rng(2 * m + R)
    L, k = 2, 72
    A = (rng.standard_normal((L, R, k)) * 0.1).astype(np.float16)
    B = rng.standard_normal((L, n, R)).astype(np.float16)
    cols = []
    for c in (3, 395):
        B[:, c, 1], B[:, c + 1, R - 1], B[:, c + 2, 3] = np.inf, -np.inf, np.nan
        B[:, c + 3, 0], B[:, c + 3, 1] = np.inf, np.inf
        cols += range(c, c + 4)
    sc = np.array([0.5, 2.0], np.float32)
    x, base = rng.standard_normal((m, k)).astype(np.float16), rng.standard_normal((m, n)).astype(np.float16)
    ids = (np.arange(m) % L).astype(np.int32)
    if m > 1:
        x[m - 1] = 0                       # h = 0: 0 * inf
    y = _run(A, B, sc, None, x, ids, base, path)
    ref, bound = _definition(x, base, ids, A, B, sc, None)
    within(y, ref, bound, path)
    assert np.isinf(y[0, [3, 4, 395, 396]]).all() and np.isnan(y[:, [5, 397]]).all()
    assert np.isfinite(np.delete(y, cols, 1)).all()


@pytest.mark.parametrize("ratio", [20, 30, 40, 43])
@pytest.mark.parametrize("m,R,path", PATHS)
def test_middle_products_of_very_different_sizes(m, R, path, ratio):
    """A x of one rank 2^ratio times that of the others, and a B that leaves
    the large one out: every value of A x is held as fp32 holds it, to 2^-21
    of itself and not of the row's largest."""
    rng = np.random.default_rng(m + R + ratio)
    L, n, k = 1, 136, 64
    A = np.zeros((L, R, k), np.float16)
    A[0, :, : k // 2] = np.float16(2.0 ** -max(ratio - 29, 0)) * (1 + rng.random((R, k // 2))).astype(np.float16)
    A[0, 0] = 0
    A[0, 0, k // 2:] = 2.0 ** 8
    x = (1 + rng.random((m, k))).astype(np.float16)
    x[:, : k // 2] *= np.float16(2.0 ** -8)
    x[:, k // 2:] = x[:, k // 2:] * np.float16(2.0 ** (min(ratio, 29) - 16))
    B = rng.standard_normal((L, n, R)).astype(np.float16)
    B[:, :, 0] = 0
    sc = np.array([2.0 ** max(ratio - 29, 0)], np.float32)
    base = np.zeros((m, n), np.float16)
    ids = np.zeros(m, np.int32)
    h = A[0].astype(np.float64) @ x[0].astype(np.float64)
    assert 2.0 ** (ratio - 3) < h[0] / h[1:].max() < 2.0 ** (ratio + 3)
    y = _run(A, B, sc, None, x, ids, base, path)
    within(y, *_definition(x, base, ids, A, B, sc, None), path)


def test_two_host_threads_with_tiles_of_different_heights():
    """Calls of one kernel instantiation with different amounts of shared
    memory, from two host threads at once."""
    rng = np.random.default_rng(1)
    L, R, n, k = 2, 256, 264, 64
    A, B = rng.standard_normal((L, R, k)).astype(np.float16), rng.standard_normal((L, n, R)).astype(np.float16)
    ad = qmm.Adapters(_c(A), _c(B), _c(np.full(L, 0.05, np.float32)))
    errors, jobs = [], []
    for m in (300, 600):
        x, base = _c(rng.standard_normal((m, k)).astype(np.float16)), _c(rng.standard_normal((m, n)).astype(np.float16))
        ids = _c((np.arange(m) % L).astype(np.int32))
        ws = torch.empty(qmm.qmm_lora_workspace_bytes(ad, m), dtype=torch.uint8, device="cuda")
        want, y = torch.empty_like(base), torch.empty_like(base)
        qmm.qmm_lora(ad, x, ids, base, want, ws=ws)
        jobs.append((x, ids, base, y, ws, want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(x, ids, base, y, ws, want, stream):
        try:
            torch.cuda.set_device(0)
            for _ in range(3000):
                qmm.qmm_lora(ad, x, ids, base, y, ws=ws, stream=stream)
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
        assert torch.equal(j[3], j[5])
    assert qmm.qmm_sync_check() == 0


def test_a_replaced_tensor_at_the_same_address_is_checked_again():
    """Only descriptors are built here: nothing is launched."""
    L, R, n, k = 4, 16, 64, 128
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt, device="cuda")
    ad = qmm.Adapters(z(L, R, k), z(L, n, R), z(L, dt=torch.float32), z(L, dt=torch.int32))
    good = ad.desc()
    for name, other in (("ranks", ad.ranks[:L - 1]), ("ranks", ad.ranks.view(torch.int64)),
                        ("ranks", ad.ranks.view(torch.int16).view(2, L)[:1].expand(2, L)),
                        ("scales", ad.scales[:L - 1]), ("scales", ad.scales.view(torch.float64)),
                        ("scales", ad.scales[:1].expand(L)), ("ranks", ad.ranks[:1].expand(L)),
                        ("a", ad.a.view(torch.int8)[..., :k]), ("b", ad.b.view(torch.int8)[..., :R])):
        kept = getattr(ad, name)
        assert other.data_ptr() == kept.data_ptr()
        setattr(ad, name, other)
        with pytest.raises(ValueError):
            ad.desc()
        setattr(ad, name, kept)
        d = ad.desc()
        assert (d.a, d.b, d.scales, d.ranks) == (good.a, good.b, good.scales, good.ranks)
    short = ad.ranks
    ad.desc()
    short.resize_(L - 1)                       # (in place: the same object)
    with pytest.raises(ValueError):
        ad.desc()


def test_bfloat16_is_refused_in_every_place():
    """With everything else on the GPU and right, one bfloat16 tensor at a time."""
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt, device="cuda")
    rows, off, g = z(8, 2, dt=torch.int32), z(3, dt=torch.int32), z(8, 2, dt=torch.float32)
    db = qmm.qmm_data_bytes(1, 64, 256)
    w = qmm.PackedWeights(1, 64, 256, torch.zeros(2 * db, dtype=torch.uint8, device="cuda"), None, 1.0, 2)
    ad = qmm.Adapters(z(2, 16, 64), z(2, 64, 16), z(2, dt=torch.float32))
    ids = z(8, dt=torch.int32)
    calls = [
        (lambda a, b: qmm.qmm_permute_backward(a, rows, b), [(16, 64), (8, 64)]),
        (lambda a, b: qmm.qmm_unpermute(a, rows, g, b), [(16, 64), (8, 64)]),
        (lambda a, b, c: qmm.qmm_unpermute_backward(a, b, rows, g, c, g.clone()), [(8, 64), (16, 64), (16, 64)]),
        (lambda a, b: qmm.qmm_grouped_gemm(w, a, off, b), [(8, 256), (8, 64)]),
        (lambda a, b: qmm.qmm_grouped_swiglu(w, w, a, off, b), [(8, 256), (8, 64)]),
        (lambda a, b, c: qmm.qmm_lora(ad, a, ids, b, c), [(8, 64), (8, 64), (8, 64)]),
        (lambda a, b: qmm.Adapters(a, b, ad.scales).desc(), [(2, 16, 64), (2, 64, 16)]),
    ]
    for fn, shapes in calls:
        for dt in (torch.float16, torch.int16):
            fn(*[z(*s, dt=dt) for s in shapes])
        for i in range(len(shapes)):
            with pytest.raises(ValueError, match="bfloat16"):
                fn(*[z(*s, dt=torch.bfloat16 if j == i else torch.float16) for j, s in enumerate(shapes)])
    qmm.qmm_permute(z(8, 64, dt=torch.bfloat16), rows, z(16, 64, dt=torch.bfloat16))   # copied
    assert qmm.qmm_sync_check() == 0


@pytest.mark.parametrize("m", [3, 70, 600])
@pytest.mark.parametrize("R,k", [(0, 64), (16, 0)])
def test_bad_ids_and_ranks_are_reported_without_a_product(R, k, m):
    """A pool of rank 0, or k = 0: y = base, and bad ids are still reported."""
    n, L = 72, 3
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    base = torch.randn(m, n, device="cuda").to(torch.float16)
    for inplace in (False, True):
        for bad_id, bad_rank in ((-1, False), (L, False), (-2, False), (0, True)):
            ranks = torch.zeros(L, dtype=torch.int32, device="cuda")
            if bad_rank:
                ranks[0] = R + 1
            ad = qmm.Adapters(z(L, R, k), z(L, n, R), torch.ones(L, device="cuda"), ranks)
            ids = (torch.arange(m, device="cuda") % (L - 1) + 1).to(torch.int32)
            ids[m - 1] = bad_id
            y = base.clone() if inplace else torch.empty_like(base)
            qmm.qmm_lora(ad, z(m, k), ids, y if inplace else base, y)
            assert qmm.qmm_sync_check() == (0 if bad_id == -1 else 7)
            assert torch.equal(y, base)
