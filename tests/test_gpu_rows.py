"""GPU parity of the sort of pairs by expert, the row movement both ways and
the gradients, against the definitions in double."""
import numpy as np
import pytest
import torch

from packed_bit_weight_b200 import qmm, synth
from rows_util import T16, U16, U32, sort_rows, unpermute, within

pytestmark = pytest.mark.gpu


def _ids(rng, t, topk, E, padded=0, repeat=False):
    ids = rng.integers(0, E, (t, topk)).astype(np.int32) if repeat or topk > E else synth.gen_topk(rng, t, topk, E)
    if padded:
        ids[rng.permutation(t)[:padded]] = -1
    return ids


def _route(ids, E):
    d = torch.from_numpy(ids).cuda()
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    perm = torch.full((max(ids.size, 1),), -7, dtype=torch.int32, device="cuda")
    rows = torch.full(ids.shape if ids.size else (1, 1), -7, dtype=torch.int32, device="cuda")
    qmm.qmm_route_rows(d, E, off, perm, rows)
    return off, perm, rows


@pytest.mark.parametrize("t,topk,E,padded,repeat", [
    (1, 1, 1, 0, False), (1, 4, 32, 0, False), (7, 3, 5, 2, False), (64, 4, 32, 0, False), (333, 1, 1024, 40, True),
    (257, 4, 8, 257, False), (1024, 1, 3, 0, True), (1025, 1, 3, 1, True), (2048, 4, 32, 0, False),
    (5000, 8, 256, 77, False), (40001, 3, 61, 0, True)])
def test_route_rows(t, topk, E, padded, repeat):
    rng = np.random.default_rng(t + E)
    ids = _ids(rng, t, topk, E, padded, repeat)
    off, perm, rows = _route(ids, E)
    assert qmm.qmm_sync_check() == 0            # -1 is no fault
    eo, ep, er = sort_rows(ids, E)
    assert np.array_equal(off.cpu().numpy(), eo)
    assert np.array_equal(perm.cpu().numpy()[:ep.size], ep)
    assert (perm.cpu().numpy()[ep.size:] == -7).all()      # behind the last row: as it was
    assert np.array_equal(rows.cpu().numpy(), er)


def test_route_rows_reports_ids_out_of_range():
    ids = np.array([[0, 8], [-2, 3], [1, 1]], dtype=np.int32)
    off, perm, rows = _route(ids, 8)
    assert qmm.qmm_sync_check() == 7
    assert qmm.qmm_sync_check() == 0
    assert rows.cpu().tolist() == [[0, -1], [-1, 3], [1, 2]]
    assert off.cpu().tolist() == [0, 1, 3, 3, 4, 4, 4, 4, 4]


def test_no_pairs():
    """No tokens, and tokens without slots: the offsets are zeros, an output
    row without slots is zero."""
    off = torch.full((6,), -7, dtype=torch.int32, device="cuda")
    for t, topk in ((0, 4), (3, 0)):
        e = torch.empty((t, topk), dtype=torch.int32, device="cuda")
        qmm.qmm_route_rows(e, 5, off, e, e)
        assert off.tolist() == [0] * 6
        x = torch.ones((t, 16), dtype=torch.float16, device="cuda")
        xs = torch.empty((0, 16), dtype=torch.float16, device="cuda")
        qmm.qmm_permute(x, e, xs)
        out = torch.full_like(x, 7.0)
        qmm.qmm_unpermute(xs, e, None, out)
        assert bool((out == 0).all())
        qmm.qmm_unpermute_backward(x, xs, e, None, xs, torch.empty((t, topk), device="cuda"))
    assert qmm.qmm_sync_check() == 0


SHAPES = [(1, 1, 4, 8, 0), (4, 4, 32, 2560, 0), (17, 6, 64, 896, 3), (33, 3, 8, 1032, 0), (300, 2, 13, 4096, 300),
          (515, 8, 128, 264, 50), (2100, 4, 32, 2560, 0)]


def _case(t, topk, E, d, padded, seed):
    rng = np.random.default_rng(seed)
    ids = _ids(rng, t, topk, E, padded, repeat=topk > E)
    off, perm, rows = _route(ids, E)
    return rng, sort_rows(ids, E), rows


def _h(rng, *shape):
    return rng.standard_normal(shape).astype(np.float16)


@pytest.mark.parametrize("t,topk,E,d,padded", SHAPES)
def test_permute(t, topk, E, d, padded):
    rng, (_, ep, er), rows = _case(t, topk, E, d, padded, d + t)
    x = _h(rng, t, d)
    x[0, :2] = [np.nan, np.inf]                          # copied, whatever they are
    xs = torch.full((t * topk, d), 7.0, dtype=torch.float16, device="cuda")
    qmm.qmm_permute(torch.from_numpy(x).cuda(), rows, xs)
    want = np.full((t * topk, d), 7.0, dtype=np.float16)  # rows behind the last: as they were
    want[:ep.size] = x[ep // topk]
    assert np.array_equal(xs.cpu().numpy().view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("t,topk,E,d,padded", SHAPES)
def test_unpermute(t, topk, E, d, padded, weighted):
    rng, (_, ep, er), rows = _case(t, topk, E, d, padded, d + t + 1)
    ys = _h(rng, t * topk, d)
    ys[ep.size:] = np.nan                                 # rows of no pair are not read
    g = rng.standard_normal((t, topk)).astype(np.float32) if weighted else np.ones((t, topk), np.float32)
    gw = g.copy()
    gw[er < 0] = np.nan                                   # nor are their weights used
    out = torch.full((t, d), 7.0, dtype=torch.float16, device="cuda")
    qmm.qmm_unpermute(torch.from_numpy(ys).cuda(), rows, torch.from_numpy(gw).cuda() if weighted else None, out)
    ref, mag = unpermute(ys.astype(np.float64), er, g.astype(np.float64))
    err = 2 * U32 * topk * mag
    within(out.cpu().numpy(), ref, err + U16 * (np.abs(ref) + err) + T16, "unpermute")
    if not weighted:                                      # the gradient of permute is the same sum
        dx = torch.empty_like(out)
        qmm.qmm_permute_backward(torch.from_numpy(ys).cuda(), rows, dx)
        assert torch.equal(dx, out)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("t,topk,E,d,padded", SHAPES)
def test_unpermute_backward(t, topk, E, d, padded, weighted):
    rng, (_, ep, er), rows = _case(t, topk, E, d, padded, d + t + 2)
    ys, dout = _h(rng, t * topk, d), _h(rng, t, d)
    ys[ep.size:] = np.nan
    g = rng.standard_normal((t, topk)).astype(np.float32) if weighted else np.ones((t, topk), np.float32)
    dys = torch.full((t * topk, d), 7.0, dtype=torch.float16, device="cuda")
    dw = torch.full((t, topk), 7.0, dtype=torch.float32, device="cuda")
    args = (torch.from_numpy(dout).cuda(), torch.from_numpy(ys).cuda(), rows,
            torch.from_numpy(g).cuda() if weighted else None)
    qmm.qmm_unpermute_backward(*args, dys, dw)
    tok = ep // topk
    v = g.reshape(-1)[ep].astype(np.float64)[:, None] * dout.astype(np.float64)[tok]
    got = dys.cpu().numpy()
    within(got[:ep.size], v, (U16 + 2 * U32) * np.abs(v) + T16, "dys")
    assert (got[ep.size:] == 7.0).all()
    prod = ys[:ep.size].astype(np.float64) * dout.astype(np.float64)[tok]
    want, bound = np.zeros(t * topk), np.zeros(t * topk)
    want[ep] = prod.sum(1)
    bound[ep] = 2 * U32 * (d / 32 + 8) * np.abs(prod).sum(1)   # a lane adds d/32 terms, then five joins
    within(dw.cpu().numpy().reshape(-1), want, bound, "dweights")
    dw2 = torch.empty_like(dw)
    qmm.qmm_unpermute_backward(*args, dys, dw2)
    assert torch.equal(dw, dw2)                            # the same bits every call


def test_gradients_against_differences():
    """<dout, U(ys + a, g) - U(ys, g)> = <dys, a> and the same for g: the
    operator is linear in each, so the difference may be of any size."""
    t, topk, E, d = 37, 4, 8, 520
    rng, (_, ep, er), rows = _case(t, topk, E, d, 5, 99)
    dev = lambda a: torch.from_numpy(a).cuda()
    ys, dout = _h(rng, t * topk, d), _h(rng, t, d)
    g = rng.uniform(0.5, 1.5, (t, topk)).astype(np.float32)

    def fwd(y, w):
        out = torch.empty((t, d), dtype=torch.float16, device="cuda")
        return qmm.qmm_unpermute(dev(y), rows, dev(w), out).cpu().numpy().astype(np.float64)

    dys = torch.zeros((t * topk, d), dtype=torch.float16, device="cuda")
    dw = torch.zeros((t, topk), dtype=torch.float32, device="cuda")
    qmm.qmm_unpermute_backward(dev(dout), dev(ys), rows, dev(g), dys, dw)
    dys, dw = dys.cpu().numpy().astype(np.float64), dw.cpu().numpy().astype(np.float64)
    base, D = fwd(ys, g), dout.astype(np.float64)
    # in the direction of the gradient itself, so that the difference is large
    y2 = ys.copy()
    y2[:ep.size] = (ys[:ep.size].astype(np.float32) + dys[:ep.size].astype(np.float32)).astype(np.float16)
    a = y2.astype(np.float64) - ys.astype(np.float64)
    out = fwd(y2, g)
    tol = (2 * U16 * np.abs(D) * (np.abs(base) + np.abs(out) + 1e-6)).sum() + 2 * U16 * np.abs(dys * a).sum()
    assert abs((D * (out - base)).sum() - (dys * a).sum()) <= tol < 0.1 * abs((dys * a).sum())
    g2 = (g + 0.05 * dw).astype(np.float32)
    out = fwd(ys, g2)
    b = g2.astype(np.float64) - g.astype(np.float64)
    tol = (2 * U16 * np.abs(D) * (np.abs(base) + np.abs(out) + 1e-6)).sum() + 1e-5 * np.abs(dw * b).sum()
    assert abs((D * (out - base)).sum() - (dw * b).sum()) <= tol < 0.1 * abs((dw * b).sum())


def test_bad_row_numbers_are_skipped():
    """Row numbers outside [0, t*topk) move nothing."""
    rows = torch.tensor([[0, 5], [-9, 1], [2 ** 30, 3]], dtype=torch.int32, device="cuda")
    x = torch.arange(24, dtype=torch.float16, device="cuda").reshape(3, 8)
    xs = torch.full((6, 8), -1.0, dtype=torch.float16, device="cuda")
    qmm.qmm_permute(x, rows, xs)
    want = torch.full_like(xs, -1.0)
    want[0], want[5], want[1], want[3] = x[0], x[0], x[1], x[2]
    assert torch.equal(xs, want)
    out = torch.empty_like(x)
    qmm.qmm_permute_backward(xs, rows, out)
    assert torch.equal(out, torch.stack([x[0] * 2, x[1], x[2]]))


def test_large_offsets():
    """Row offsets past 2^31 bytes: one expert holds every row."""
    t, topk, d = 70000, 4, 8192                   # 280,000 rows of 16 KB: 4.6 GB
    ids = torch.zeros((t, topk), dtype=torch.int32, device="cuda")
    off = torch.empty(2, dtype=torch.int32, device="cuda")
    perm = torch.empty(t * topk, dtype=torch.int32, device="cuda")
    rows = torch.empty((t, topk), dtype=torch.int32, device="cuda")
    qmm.qmm_route_rows(ids, 1, off, perm, rows)
    x = torch.randint(-100, 100, (t, 1), device="cuda", dtype=torch.int16).half().expand(t, d).contiguous()
    xs = torch.zeros((t * topk, d), dtype=torch.float16, device="cuda")
    qmm.qmm_permute(x, rows, xs)
    assert torch.equal(xs[:, ::1024], x[:, ::1024].repeat_interleave(topk, 0))
    out = torch.empty_like(x)
    qmm.qmm_permute_backward(xs, rows, out)
    assert torch.equal(out, x * topk)
