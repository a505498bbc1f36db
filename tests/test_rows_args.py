"""Host-side refusals of the grouped-row operators and the adapters, without a
GPU: the C checks (fake addresses that are never dereferenced) and the
binding's checks."""
import ctypes

import pytest
import torch

from packed_bit_weight_b200 import qmm

OK, INVALID, UNSUPPORTED, MISALIGNED, NOT_SM100, CUDA, WORKSPACE = 0, 1, 2, 3, 4, 5, 8
FAKE = 1 << 40


def _vp(a):
    return ctypes.c_void_p(a) if a else None


def _no_device(status):
    """Passed every check that comes before the device is looked at."""
    return status in (OK, NOT_SM100, CUDA)


def test_route_rows():
    L = qmm._lib()

    def call(t=8, k=2, E=4, ids=FAKE, off=FAKE, perm=FAKE, rows=FAKE):
        return L.qmm_route_rows(_vp(ids), t, k, E, _vp(off), _vp(perm), _vp(rows), None)

    assert call(t=-1) == INVALID and call(k=-1) == INVALID and call(E=0) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(t=1 << 30) == UNSUPPORTED and call(t=1 << 62, k=1 << 40) == UNSUPPORTED
    for name in ("ids", "off", "perm", "rows"):
        assert call(**{name: 0}) == INVALID
        assert call(**{name: FAKE + 4}) == MISALIGNED


def test_row_movers():
    L = qmm._lib()

    def permute(x=FAKE, r=FAKE, t=8, k=2, d=64, xs=FAKE):
        return L.qmm_permute(_vp(x), _vp(r), t, k, d, _vp(xs), None)

    def back(ys=FAKE, r=FAKE, g=FAKE, t=8, k=2, d=64, out=FAKE):
        return L.qmm_unpermute(_vp(ys), _vp(r), _vp(g), t, k, d, _vp(out), None)

    def bwd(do=FAKE, ys=FAKE, r=FAKE, g=FAKE, t=8, k=2, d=64, dys=FAKE, dg=FAKE):
        return L.qmm_unpermute_backward(_vp(do), _vp(ys), _vp(r), _vp(g), t, k, d, _vp(dys), _vp(dg), None)

    for f in (permute, back, bwd):
        assert f(t=-1) == INVALID and f(k=-1) == INVALID and f(d=-8) == INVALID
        assert f(d=60) == UNSUPPORTED and f(t=1 << 30) == UNSUPPORTED and f(t=1 << 62, k=1 << 40) == UNSUPPORTED
        assert f(r=0) == INVALID and f(r=FAKE + 4) == MISALIGNED
    assert permute(x=0) == INVALID and permute(xs=0) == INVALID and permute(xs=FAKE + 8) == MISALIGNED
    assert back(ys=0) == INVALID and back(out=0) == INVALID and back(g=FAKE + 4) == MISALIGNED
    assert bwd(do=0) == INVALID and bwd(dys=0) == INVALID and bwd(dg=0) == INVALID and bwd(ys=FAKE + 2) == MISALIGNED


def _stack(fmt=1, n=64, k=256, experts=4, data_stride=None):
    d = qmm.qmm_weights()
    d.fmt, d.reserved, d.n, d.k = fmt, 0, n, k
    d.data = ctypes.c_void_p(FAKE)
    d.scales = None if fmt == 1 else ctypes.c_void_p(FAKE)
    d.global_scale, d.reserved2, d.num_experts = 1.0, 0, experts
    d.expert_data_stride = qmm.qmm_data_bytes(fmt, n, k) if data_stride is None else data_stride
    d.expert_scale_stride = qmm.qmm_scale_bytes(fmt, n, k)
    return d


def test_grouped_products():
    L = qmm._lib()

    def gemm(w=None, x=FAKE, off=FAKE, rows=8, y=FAKE):
        return L.qmm_grouped_gemm(ctypes.byref(w or _stack()), _vp(x), _vp(off), rows, _vp(y), None)

    assert L.qmm_grouped_gemm(None, _vp(FAKE), _vp(FAKE), 8, _vp(FAKE), None) == INVALID
    assert gemm(_stack(fmt=7)) == INVALID and gemm(_stack(k=250)) == UNSUPPORTED
    assert gemm(_stack(data_stride=16)) == INVALID
    assert gemm(_stack(experts=257)) == UNSUPPORTED
    assert gemm(rows=-1) == INVALID and gemm(rows=1 << 31) == UNSUPPORTED
    for name in ("x", "off", "y"):
        assert gemm(**{name: 0}) == INVALID and gemm(**{name: FAKE + 8}) == MISALIGNED

    def swiglu(g, u):
        return L.qmm_grouped_swiglu(ctypes.byref(g), ctypes.byref(u), _vp(FAKE), _vp(FAKE), 8, _vp(FAKE), None)

    assert swiglu(_stack(), _stack(n=80)) == INVALID and swiglu(_stack(), _stack(k=512)) == INVALID
    assert swiglu(_stack(), _stack(fmt=4)) == INVALID and swiglu(_stack(), _stack(experts=5)) == INVALID


def _adapters(**kw):
    d = qmm.qmm_adapters()
    v = dict(num_adapters=4, n=64, k=256, rank=16, a=FAKE, b=FAKE, scales=FAKE, ranks=0)
    v.update(kw)
    v.setdefault("a_stride", 2 * v["rank"] * v["k"])
    v.setdefault("b_stride", 2 * v["rank"] * v["n"])
    for key, val in v.items():
        setattr(d, key, _vp(val) if key in ("a", "b", "scales", "ranks") else val)
    return d


def test_lora():
    L = qmm._lib()

    def call(ad=None, x=FAKE, ids=FAKE, m=8, base=FAKE, y=FAKE, ws=FAKE, wb=1 << 30):
        return L.qmm_lora(ctypes.byref(ad or _adapters()), _vp(x), _vp(ids), m, _vp(base), _vp(y), _vp(ws), wb, None)

    assert L.qmm_lora(None, _vp(FAKE), _vp(FAKE), 8, _vp(FAKE), _vp(FAKE), None, 0, None) == INVALID
    assert call(_adapters(num_adapters=0)) == INVALID and call(_adapters(num_adapters=1025)) == UNSUPPORTED
    assert call(_adapters(rank=12)) == UNSUPPORTED and call(_adapters(rank=264)) == UNSUPPORTED
    assert call(_adapters(k=252)) == UNSUPPORTED and call(_adapters(n=-1)) == INVALID
    assert call(_adapters(a=0)) == INVALID and call(_adapters(b=0)) == INVALID and call(_adapters(scales=0)) == INVALID
    assert call(_adapters(a=FAKE + 8)) == MISALIGNED and call(_adapters(ranks=FAKE + 4)) == MISALIGNED
    assert call(_adapters(a_stride=64)) == INVALID and call(_adapters(b_stride=2 * 16 * 64 + 8)) == MISALIGNED
    assert call(m=-1) == INVALID and call(m=1 << 31) == UNSUPPORTED
    for name in ("x", "ids", "base", "y"):
        assert call(**{name: 0}) == INVALID and call(**{name: FAKE + 8}) == MISALIGNED
    assert call(ws=FAKE + 4) == MISALIGNED
    assert L.qmm_lora_workspace_bytes(ctypes.byref(_adapters()), -1) == 0
    assert L.qmm_lora_workspace_bytes(ctypes.byref(_adapters(rank=12)), 8) == 0
    assert L.qmm_lora_workspace_bytes(ctypes.byref(_adapters()), 65) > 0


def _short(fn, *a, **kw):
    with pytest.raises(ValueError, match="holds"):
        fn(*a, **kw)


def test_binding_refuses_undersized_or_host_tensors():
    i16, i32, f32 = torch.int16, torch.int32, torch.float32
    z = lambda *s, dt=i16: torch.zeros(*s, dtype=dt)
    ids = z(8, 2, dt=i32)
    _short(qmm.qmm_route_rows, ids, 4, z(4, dt=i32), z(16, dt=i32), z(8, 2, dt=i32))
    _short(qmm.qmm_route_rows, ids, 4, z(5, dt=i32), z(15, dt=i32), z(8, 2, dt=i32))
    _short(qmm.qmm_route_rows, ids, 4, z(5, dt=i32), z(16, dt=i32), z(8, 1, dt=i32))
    _short(qmm.qmm_permute, z(8, 64), ids, z(15, 64))
    _short(qmm.qmm_permute_backward, z(15, 64), ids, z(8, 64))
    _short(qmm.qmm_unpermute, z(15, 64), ids, None, z(8, 64))
    _short(qmm.qmm_unpermute, z(16, 64), ids, z(8, 1, dt=f32), z(8, 64))
    _short(qmm.qmm_unpermute_backward, z(8, 64), z(16, 64), ids, None, z(15, 64), z(8, 2, dt=f32))
    _short(qmm.qmm_unpermute_backward, z(8, 64), z(16, 64), ids, None, z(16, 64), z(8, 1, dt=f32))
    with pytest.raises(ValueError, match=r"\[t\]\[d\]"):
        qmm.qmm_permute(z(7, 64), ids, z(16, 64))
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_permute(z(8, 64), ids, z(16, 64))
    db = qmm.qmm_data_bytes(1, 64, 256)
    w = qmm.PackedWeights(1, 64, 256, torch.zeros(4 * db, dtype=torch.uint8), None, 1.0, 4)
    _short(qmm.qmm_grouped_gemm, w, z(8, 255), z(5, dt=i32), z(8, 64))
    _short(qmm.qmm_grouped_gemm, w, z(8, 256), z(4, dt=i32), z(8, 64))
    _short(qmm.qmm_grouped_gemm, w, z(8, 256), z(5, dt=i32), z(8, 63))
    _short(qmm.qmm_grouped_swiglu, w, w, z(8, 256), z(5, dt=i32), z(7, 64))
    ad = qmm.Adapters(z(4, 16, 256), z(4, 64, 16), z(4, dt=f32))
    _short(qmm.qmm_lora, ad, z(7, 256), z(8, dt=i32), z(8, 64), z(8, 64))
    _short(qmm.qmm_lora, ad, z(8, 256), z(8, dt=i32), z(8, 64), z(7, 64))
    _short(qmm.Adapters(z(4, 16, 256), z(4, 64, 16), z(3, dt=f32)).desc)
    with pytest.raises(ValueError, match="rank"):
        qmm.Adapters(z(4, 16, 256), z(4, 64, 8), z(4, dt=f32)).desc()
    with pytest.raises(ValueError, match="contiguous"):
        qmm.Adapters(z(4, 256, 16).transpose(1, 2), z(4, 64, 16), z(4, dt=f32)).desc()
    with pytest.raises(ValueError, match="CUDA"):
        ad.desc()
