"""GPU parity of the experts' products over sorted rows against the decoded
weights in double."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from packed_bit_weight_b200 import qmm, synth
from rows_util import expert_products, product_bound, swiglu_bound, within

pytestmark = pytest.mark.gpu

FMTS = [synth.FMT_IQ4_NL, synth.FMT_FP4G16_F16, synth.FMT_FP4G16_E4M3, synth.FMT_MXFP4]


def _f(t):
    return t.cpu().numpy().astype(np.float64)


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _x(rng, rows, k, offsets):
    x = synth.gen_x(rng, rows, k)
    x[offsets[-1]:] = 0x7E00          # NaN: rows of no expert are not read
    return x


def _gemm(p, x, offsets):
    y = torch.full((x.shape[0], p.n), 7.0, dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_gemm(dev(p), torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(offsets).cuda(), y)
    assert qmm.qmm_sync_check() == 0, qmm.qmm_last_variant()
    return _f(y)


CASES = [  # rows per expert, rows behind the last, n, k
    ([1], 0, 16, 32), ([0, 0, 1, 0], 0, 40, 64), ([3, 0, 5], 2, 33, 96), ([17, 1, 0, 30], 1, 130, 256),
    ([0, 0], 4, 64, 128), ([129, 0, 1, 127, 128], 0, 200, 384), ([5, 300, 0, 256, 257], 3, 264, 512),
    ([0, 700], 5, 96, 896), ([2, 2, 2, 2, 2, 2, 2, 2], 0, 2560, 896), ([40] * 6, 0, 320, 2560),
    ([1000, 3], 0, 1, 256), ([60, 70], 0, 72, 160)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,behind,n,k", CASES)
def test_grouped_gemm(fmt, counts, behind, n, k):
    rng = np.random.default_rng(n + k + fmt)
    off = _offsets(counts)
    p = synth.gen_weights(rng, fmt, n, k, experts=len(counts))
    x = _x(rng, off[-1] + behind, k, off)
    y = _gemm(p, x, off)
    ref, a = expert_products(p, x, off)
    within(y[:off[-1]], ref[:off[-1]], product_bound(ref, a, k)[:off[-1]], qmm.qmm_last_variant())
    assert (y[off[-1]:] == 7.0).all()                  # rows behind: as they were


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,behind,n,k", CASES)
def test_grouped_swiglu(fmt, counts, behind, n, k):
    rng = np.random.default_rng(n + k + fmt + 50)
    off = _offsets(counts)
    pg = synth.gen_weights(rng, fmt, n, k, experts=len(counts))
    pu = synth.gen_weights(rng, fmt, n, k, experts=len(counts))
    x = _x(rng, off[-1] + behind, k, off)
    h = torch.full((x.shape[0], n), 7.0, dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_swiglu(dev(pg), dev(pu), torch.from_numpy(x.view(np.int16)).cuda(),
                           torch.from_numpy(off).cuda(), h)
    assert qmm.qmm_sync_check() == 0
    zg, ag = expert_products(pg, x, off)
    zu, au = expert_products(pu, x, off)
    ref, bound = swiglu_bound(zg, ag, zu, au, k)
    h = _f(h)
    within(h[:off[-1]], ref[:off[-1]], bound[:off[-1]], qmm.qmm_last_variant())
    assert (h[off[-1]:] == 7.0).all()


def test_gate_and_up_views_of_one_stack():
    """Gate and up as row views of one [E][2f][k] stack (expert strides above
    one matrix, the second half 16-byte aligned)."""
    rng = np.random.default_rng(5)
    E, f, k, counts = 3, 96, 256, [70, 0, 200]
    off = _offsets(counts)
    p = synth.gen_iq4nl(rng, 2 * f, k, E)
    x = _x(rng, off[-1], k, off)
    w = dev(p)
    h = torch.empty((off[-1], f), dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_swiglu(w.rows(0, f), w.rows(f, 2 * f), torch.from_numpy(x.view(np.int16)).cuda(),
                           torch.from_numpy(off).cuda(), h)
    assert qmm.qmm_sync_check() == 0
    z, a = expert_products(p, x, off)
    ref, bound = swiglu_bound(z[:, :f], a[:, :f], z[:, f:], a[:, f:], k)
    within(_f(h), ref, bound)


@pytest.mark.parametrize("rows", [6, 700])
def test_a_row_of_infinities_and_nan_stays_in_its_row(rows):
    rng = np.random.default_rng(8)
    off = _offsets([rows // 2, rows - rows // 2])
    p = synth.gen_iq4nl(rng, 64, 256, 2)
    x = _x(rng, rows, 256, off)
    x[1, 3], x[rows - 2, :2] = 0x7E00, [0x7C00, 0xFC00]
    y = _gemm(p, x, off)
    keep = np.ones(rows, bool)
    keep[[1, rows - 2]] = False
    ref, a = expert_products(p, np.where(keep[:, None], x, np.uint16(0)).astype(np.uint16), off)
    within(y[keep], ref[keep], product_bound(ref, a, 256)[keep])
    assert np.isnan(y[1]).all() and not np.isfinite(y[rows - 2]).any()


@pytest.mark.parametrize("rows", [9, 600])
def test_bad_offsets_are_reported_and_clamped(rows):
    rng = np.random.default_rng(9)
    p = synth.gen_iq4nl(rng, 64, 256, 3)
    x = _x(rng, rows, 256, np.array([0, rows]))
    off = np.array([-5, rows // 3, rows // 3, rows + 1000], dtype=np.int32)
    y = torch.full((rows, 64), 7.0, dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_gemm(dev(p), torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(off).cuda(), y)
    assert qmm.qmm_sync_check() == 7
    good = np.array([0, rows // 3, rows // 3, rows], dtype=np.int32)
    ref, a = expert_products(p, x, good)
    within(_f(y), ref, product_bound(ref, a, 256))


def test_no_rows():
    p = dev(synth.gen_iq4nl(np.random.default_rng(1), 64, 256, 3))
    x = torch.empty((0, 256), dtype=torch.float16, device="cuda")
    y = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    qmm.qmm_grouped_gemm(p, x, torch.zeros(4, dtype=torch.int32, device="cuda"), y)
    assert qmm.qmm_sync_check() == 0


def _moe_inputs(t, seed=3):
    E, f, d, topk = 32, 896, 2560, 4
    wgu, wdn, x, wr, br = synth.make_moe(E, f, d, t, topk, seed)
    g = {"gate_up": dev(wgu), "down": dev(wdn), "E": E, "f": f, "d": d, "topk": topk, "t": t,
         "x": torch.from_numpy(x.view(np.int16)).cuda(), "wr": torch.from_numpy(wr.view(np.int16)).cuda(),
         "br": torch.from_numpy(br).cuda()}
    i32, i16, P = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int16, device="cuda"), t * topk
    g.update(ids=torch.empty((t, topk), **i32), w=torch.empty((t, topk), dtype=torch.float32, device="cuda"),
             off=torch.empty(E + 1, **i32), perm=torch.empty(P, **i32), rows=torch.empty((t, topk), **i32),
             xs=torch.empty((P, d), **i16), h=torch.empty((P, f), **i16), ys=torch.empty((P, d), **i16),
             out=torch.empty((t, d), **i16))
    return g


def _moe_prefill(g):
    gate, up = g["gate_up"].rows(0, g["f"]), g["gate_up"].rows(g["f"], 2 * g["f"])
    qmm.qmm_router_topk(g["x"], g["wr"], g["br"], g["topk"], g["ids"], g["w"])
    qmm.qmm_route_rows(g["ids"], g["E"], g["off"], g["perm"], g["rows"])
    qmm.qmm_permute(g["x"], g["rows"], g["xs"])
    qmm.qmm_grouped_swiglu(gate, up, g["xs"], g["off"], g["h"])
    qmm.qmm_grouped_gemm(g["down"], g["h"], g["off"], g["ys"])
    return qmm.qmm_unpermute(g["ys"], g["rows"], g["w"], g["out"])


@pytest.mark.parametrize("t", [1, 3, 61, 517])
def test_prefill_layer_matches_the_decode_block(t):
    """Router, sort, permute, SwiGLU, down and back together against
    qmm_moe_routed.  They differ by their sums' orders (each within
    product_bound of the same h), and by fp16 of the down outputs: U16 of
    sum |g y| and of the result, on top of the block's own rounding.  h itself
    may differ by one fp16 step, which the down product carries to at most
    2 * U16 * sum |w h|."""
    g = _moe_inputs(t)
    out = _f(_moe_prefill(g).view(torch.float16))
    ref = torch.empty_like(g["out"])
    gate, up = g["gate_up"].rows(0, g["f"]), g["gate_up"].rows(g["f"], 2 * g["f"])
    ws = torch.empty(qmm.qmm_workspace_bytes(qmm.OP_MOE, gate, 0, t, g["topk"]), dtype=torch.uint8, device="cuda")
    qmm.qmm_moe_routed(gate, up, g["down"], g["x"], g["ids"], g["w"], ref, ws=ws)
    assert qmm.qmm_sync_check() == 0
    # magnitudes sum_s g sum_f |w h| of the down products, on the GPU in fp32
    mag = torch.zeros((t, g["d"]), dtype=torch.float32, device="cuda")
    off, perm = g["off"].tolist(), g["perm"].long()
    wd = torch.empty((g["d"], g["f"]), dtype=torch.float16, device="cuda")
    for e in range(g["E"]):
        if off[e + 1] > off[e]:
            p = g["down"]
            one = qmm.PackedWeights(p.fmt, p.n, p.k, p.data[e * p.desc().expert_data_stride:], None)
            qmm.qmm_dequant(one, wd)
            m = g["h"].view(torch.float16)[off[e]:off[e + 1]].float().abs() @ wd.float().abs().t()
            pr = perm[off[e]:off[e + 1]]
            mag.index_add_(0, pr // g["topk"], m * g["w"].reshape(-1)[pr, None])
    from rows_util import T16, U16, U32
    ref, mag = _f(ref.view(torch.float16)), mag.cpu().numpy().astype(np.float64)
    bound = 2 * U16 * mag + 4 * U32 * (g["f"] + 8) * mag + 2 * U16 * mag + 2 * U16 * np.abs(ref) + 8 * T16
    within(out, ref, bound, "prefill layer")


def test_prefill_layer_captured_and_replayed():
    """The whole layer in one CUDA graph, replayed on new inputs, gives what
    the same calls give outside it."""
    g = _moe_inputs(130, seed=4)
    want = []
    xs = [g["x"].clone(), torch.roll(g["x"], 1, 0).contiguous(), g["x"].flip(0).contiguous()]
    for x in xs:
        g["x"].copy_(x)
        want.append(_moe_prefill(g).clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _moe_prefill(g)
    for x, w in zip(xs, want):
        g["x"].copy_(x)
        g["out"].fill_(-1)
        graph.replay()
        assert torch.equal(g["out"], w)
    assert qmm.qmm_sync_check() == 0
