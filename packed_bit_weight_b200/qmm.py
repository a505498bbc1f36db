"""ctypes binding of libqmm.so (include/qmm.h).

Argument marshalling only: every function here takes torch tensors, checks
that they are CUDA tensors of the right element size and that each holds at
least the bytes the call will read or write (the C ABI takes bare pointers
and cannot see a buffer's extent), passes raw device pointers and the current
CUDA stream to the C ABI, and raises ``QmmError`` on a non-OK status.  No arithmetic of the path happens in Python, and there is
no fallback: if the library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

from . import _build

FMT_IQ4_NL = 1
FMT_FP4G16_F16 = 2
FMT_FP4G16_E4M3 = 3
FMT_MXFP4 = 4

OP_DEQUANT, OP_GEMV, OP_GEMM, OP_ROUTE, OP_GROUPED, OP_MOE = 0, 1, 2, 3, 4, 5

STATUS = {0: "QMM_OK", 1: "QMM_ERR_INVALID_ARG", 2: "QMM_ERR_UNSUPPORTED_SHAPE", 3: "QMM_ERR_MISALIGNED",
          4: "QMM_ERR_NOT_SM100", 5: "QMM_ERR_CUDA", 6: "QMM_ERR_TIMEOUT", 7: "QMM_ERR_DEVICE_FAULT",
          8: "QMM_ERR_WORKSPACE"}


class QmmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), _lib().qmm_status_string(status).decode()))


class qmm_weights(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_scale", ctypes.c_float),
                ("reserved2", ctypes.c_int32), ("num_experts", ctypes.c_int64),
                ("expert_data_stride", ctypes.c_int64), ("expert_scale_stride", ctypes.c_int64)]


class qmm_adapters(ctypes.Structure):
    _fields_ = [("num_adapters", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("rank", ctypes.c_int64), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("ranks", ctypes.c_void_p), ("a_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64)]


_L = None
LIB_PATH = _build.LIB


def _lib():
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libqmm.so is not built (expected at %s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        W = ctypes.POINTER(qmm_weights)
        A = ctypes.POINTER(qmm_adapters)
        sigs = {
            "qmm_data_bytes": (sz, [i32, i64, i64]),
            "qmm_scale_bytes": (sz, [i32, i64, i64]),
            "qmm_packed_bytes": (sz, [i32, i64, i64]),
            "qmm_dequant": (i32, [W, vp, vp]),
            "qmm_quantize": (i32, [i32, vp, i64, i64, vp, vp, vp]),
            "qmm_gemv": (i32, [W, vp, i64, vp, vp, sz, vp]),
            "qmm_gemv_host": (i32, [W, vp, i64, vp, vp, vp, vp]),
            "qmm_gemm": (i32, [W, vp, i64, vp, vp, sz, vp]),
            "qmm_route": (i32, [vp, i64, i64, i64, vp, vp, vp, sz, vp]),
            "qmm_grouped_gemv": (i32, [W, vp, i32, vp, i64, i64, vp, vp, sz, vp]),
            "qmm_grouped_gemv_noalloc": (i32, [W, vp, i32, vp, i64, i64, vp, vp]),
            "qmm_router_topk": (i32, [vp, vp, vp, i64, i64, i64, i64, vp, vp, vp, vp]),
            "qmm_moe_routed": (i32, [W, W, W, vp, vp, vp, i64, i64, vp, vp, sz, vp]),
            "qmm_route_rows": (i32, [vp, i64, i64, i64, vp, vp, vp, vp]),
            "qmm_permute": (i32, [vp, vp, i64, i64, i64, vp, vp]),
            "qmm_permute_backward": (i32, [vp, vp, i64, i64, i64, vp, vp]),
            "qmm_unpermute": (i32, [vp, vp, vp, i64, i64, i64, vp, vp]),
            "qmm_unpermute_backward": (i32, [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp]),
            "qmm_grouped_gemm": (i32, [W, vp, vp, i64, vp, vp]),
            "qmm_grouped_swiglu": (i32, [W, W, vp, vp, i64, vp, vp]),
            "qmm_lora": (i32, [A, vp, vp, i64, vp, vp, vp, sz, vp]),
            "qmm_lora_workspace_bytes": (sz, [A, i64]),
            "qmm_workspace_bytes": (sz, [i32, W, i64, i64, i64]),
            "qmm_sync_check": (i32, [vp]),
            "qmm_debug_set": (i32, [i32, i64]),
            "qmm_status_string": (ctypes.c_char_p, [i32]),
            "qmm_last_variant": (ctypes.c_char_p, []),
            "qmm_version": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sigs.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _L = L
    return _L


def lib():
    return _lib()


def _check(status: int, where: str):
    if status != 0:
        raise QmmError(status, where)


def _stream(stream=None):
    if stream is None and torch.cuda.is_initialized():
        # the raw handle: building a Stream object costs more than the launch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _need(t: torch.Tensor | None, nbytes: int, name: str) -> None:
    """Refuse a tensor smaller than the bytes the C call touches through its
    pointer: an undersized buffer would otherwise be an out-of-bounds access
    on the device instead of an error here.  None is left to the C checks."""
    if t is not None and t.nbytes < nbytes:
        raise ValueError("%s holds %d bytes; the call reads or writes %d" % (name, t.nbytes, nbytes))


def _ptr(t: torch.Tensor | None, esize: int | None = None, name: str = "tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if esize is not None and t.element_size() != esize:
        raise ValueError("%s must have %d-byte elements" % (name, esize))
    return ctypes.c_void_p(t.data_ptr())


@dataclass
class PackedWeights:
    """Device tensors of one packed matrix (or expert stack) plus its C descriptor."""
    fmt: int
    n: int
    k: int
    data: torch.Tensor
    scales: torch.Tensor | None
    global_scale: float = 1.0
    experts: int = 1
    data_stride: int | None = None    # bytes between experts (default: data split evenly)
    scale_stride: int | None = None

    def desc(self) -> qmm_weights:
        """The C descriptor, rebuilt only when a field or a buffer changed."""
        key = (self.fmt, self.n, self.k, None if self.data is None else (self.data.data_ptr(), self.data.nbytes),
               None if self.scales is None else (self.scales.data_ptr(), self.scales.nbytes), self.global_scale,
               self.experts, self.data_stride, self.scale_stride)
        cached = self.__dict__.get("_desc")
        if cached is not None and cached[0] == key:
            return cached[1]
        d = self._build_desc()
        self.__dict__["_desc"] = (key, d)
        return d

    def _build_desc(self) -> qmm_weights:
        d = qmm_weights()
        d.fmt, d.reserved, d.n, d.k = self.fmt, 0, self.n, self.k
        d.data = ctypes.c_void_p(self.data.data_ptr()) if self.data is not None else None
        d.scales = ctypes.c_void_p(self.scales.data_ptr()) if self.scales is not None else None
        d.global_scale, d.reserved2, d.num_experts = float(self.global_scale), 0, self.experts
        if self.data_stride is not None:
            d.expert_data_stride = self.data_stride
        else:
            d.expert_data_stride = self.data.numel() // self.experts if self.data is not None else 0
        if self.scale_stride is not None:
            d.expert_scale_stride = self.scale_stride
        else:
            d.expert_scale_stride = (self.scales.numel() * self.scales.element_size() // self.experts
                                     if self.scales is not None else 0)
        # every expert's codes and scales must lie inside the tensors (the
        # sizes are 0 for a shape the C checks reject anyway)
        last = max(int(self.experts), 1) - 1
        db, sb = qmm_data_bytes(self.fmt, self.n, self.k), qmm_scale_bytes(self.fmt, self.n, self.k)
        _need(self.data, last * d.expert_data_stride + db if db else 0, "data")
        _need(self.scales, last * d.expert_scale_stride + sb if sb else 0, "scales")
        return d

    def rows(self, r0: int, r1: int) -> "PackedWeights":
        """View of rows [r0, r1) of every matrix of the stack (no copy): e.g.
        the gate and up halves of an expert stack stored as [E][2f][k]."""
        db, sb = qmm_data_bytes(self.fmt, 1, self.k), qmm_scale_bytes(self.fmt, 1, self.k)
        d = self.desc()
        data = self.data.view(torch.uint8).reshape(-1)[r0 * db:]
        scales = None if self.scales is None else self.scales.view(torch.uint8).reshape(-1)[r0 * sb:]
        return PackedWeights(self.fmt, r1 - r0, self.k, data, scales, self.global_scale, self.experts,
                             d.expert_data_stride, d.expert_scale_stride)

    @property
    def nbytes(self) -> int:
        return self.data.numel() + (0 if self.scales is None else self.scales.numel() * self.scales.element_size())

    @staticmethod
    def from_host(p, device="cuda") -> "PackedWeights":
        """From a ``synth.Packed`` (numpy bytes) to device tensors.  An expert
        stack whose per-expert byte counts are not multiples of 16 (e.g.
        MXFP4 scales of an odd row count) is copied with each expert padded
        to 16 bytes, as the expert strides of the C ABI require."""
        ds, ss = p.data_stride, p.scale_stride
        if p.experts > 1 and (ds % 16 or ss % 16):
            pd, ps = -(-ds // 16) * 16, -(-ss // 16) * 16
            d = np.zeros((p.experts, pd), dtype=np.uint8)
            d[:, :ds] = p.data.reshape(p.experts, ds)
            sc = None
            if p.scales is not None:
                sc = np.zeros((p.experts, ps), dtype=np.uint8)
                sc[:, :ss] = p.scales.reshape(p.experts, ss)
                sc = torch.from_numpy(sc.reshape(-1)).to(device)
            return PackedWeights(p.fmt, p.n, p.k, torch.from_numpy(d.reshape(-1)).to(device), sc, p.global_scale,
                                 p.experts, pd, ps if p.scales is not None else None)
        data = torch.from_numpy(p.data).to(device)
        scales = None if p.scales is None else torch.from_numpy(p.scales).to(device)
        return PackedWeights(p.fmt, p.n, p.k, data, scales, p.global_scale, p.experts)


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def qmm_data_bytes(fmt: int, n: int, k: int) -> int:
    return _lib().qmm_data_bytes(fmt, n, k)


def qmm_scale_bytes(fmt: int, n: int, k: int) -> int:
    return _lib().qmm_scale_bytes(fmt, n, k)


def qmm_packed_bytes(fmt: int, n: int, k: int) -> int:
    return _lib().qmm_packed_bytes(fmt, n, k)


def qmm_workspace_bytes(op: int, w: PackedWeights | None, m: int = 0, t: int = 0, topk: int = 0) -> int:
    d = w.desc() if w is not None else None
    return _lib().qmm_workspace_bytes(op, ctypes.byref(d) if d is not None else None, m, t, topk)


def qmm_dequant(w: PackedWeights, out: torch.Tensor, stream=None) -> torch.Tensor:
    d = w.desc()
    _need(out, 2 * w.n * w.k, "out")
    _check(_lib().qmm_dequant(ctypes.byref(d), _ptr(out, 2, "out"), _stream(stream)), "qmm_dequant")
    return out


def qmm_quantize(fmt: int, w: torch.Tensor, data: torch.Tensor, scales: torch.Tensor | None = None,
                 stream=None) -> None:
    """fp16 weights w [n][k] (2-byte elements) -> packed data / scales."""
    n, k = w.shape
    _need(data, qmm_data_bytes(fmt, n, k), "data")
    _need(scales, qmm_scale_bytes(fmt, n, k), "scales")
    _check(_lib().qmm_quantize(fmt, _ptr(w, 2, "w"), n, k, _ptr(data, None, "data"), _ptr(scales, None, "scales"),
                               _stream(stream)), "qmm_quantize")


def _ws(ws):
    return (_ptr(ws, None, "ws"), 0 if ws is None else ws.numel() * ws.element_size())


def qmm_gemv(w: PackedWeights, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    d = w.desc()
    wp, wb = _ws(ws)
    m = x.shape[0] if x.dim() == 2 else 1
    _need(x, 2 * m * w.k, "x")
    _need(y, 2 * m * w.n, "y")
    _check(_lib().qmm_gemv(ctypes.byref(d), _ptr(x, 2, "x"), m, _ptr(y, 2, "y"), wp, wb, _stream(stream)), "qmm_gemv")
    return y


def _host_ptr(t: torch.Tensor, esize: int, name: str):
    if t.is_cuda:
        raise ValueError("%s must be a host tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.element_size() != esize:
        raise ValueError("%s must have %d-byte elements" % (name, esize))
    return ctypes.c_void_p(t.data_ptr())


def qmm_gemv_host(w: PackedWeights, x_host: torch.Tensor, y_host: torch.Tensor, x_dev: torch.Tensor,
                  y_dev: torch.Tensor, stream=None) -> torch.Tensor:
    """qmm_gemv on host tensors in one library call: x_host -> x_dev, the
    product into y_dev, y_dev -> y_host, enqueued on the stream (asynchronous
    when the host tensors are pinned)."""
    d = w.desc()
    m = x_host.shape[0] if x_host.dim() == 2 else 1
    xb, yb = 2 * m * w.k, 2 * m * w.n
    _need(x_host, xb, "x_host")
    _need(x_dev, xb, "x_dev")
    _need(y_host, yb, "y_host")
    _need(y_dev, yb, "y_dev")
    _check(_lib().qmm_gemv_host(ctypes.byref(d), _host_ptr(x_host, 2, "x_host"), m, _host_ptr(y_host, 2, "y_host"),
                                _ptr(x_dev, 2, "x_dev"), _ptr(y_dev, 2, "y_dev"), _stream(stream)), "qmm_gemv_host")
    return y_host


def qmm_gemm(w: PackedWeights, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    d = w.desc()
    wp, wb = _ws(ws)
    _need(x, 2 * x.shape[0] * w.k, "x")
    _need(y, 2 * x.shape[0] * w.n, "y")
    _check(_lib().qmm_gemm(ctypes.byref(d), _ptr(x, 2, "x"), x.shape[0], _ptr(y, 2, "y"), wp, wb, _stream(stream)),
           "qmm_gemm")
    return y


def qmm_route(topk_ids: torch.Tensor, num_experts: int, offsets: torch.Tensor, perm: torch.Tensor,
              ws: torch.Tensor | None = None, stream=None):
    t, topk = topk_ids.shape
    wp, wb = _ws(ws)
    _need(offsets, 4 * (num_experts + 1), "offsets")
    _need(perm, 4 * t * topk, "perm")
    _check(_lib().qmm_route(_ptr(topk_ids, 4, "topk_ids"), t, topk, num_experts, _ptr(offsets, 4, "offsets"),
                            _ptr(perm, 4, "perm"), wp, wb, _stream(stream)), "qmm_route")
    return offsets, perm


def _need_grouped(w: PackedWeights, x, topk_ids, y, x_per_pair):
    t, topk = topk_ids.shape
    _need(x, 2 * w.k * (t * topk if x_per_pair else t), "x")
    _need(y, 2 * t * topk * w.n, "y")
    return t, topk


def qmm_grouped_gemv(w: PackedWeights, x: torch.Tensor, topk_ids: torch.Tensor, y: torch.Tensor,
                     x_per_pair: bool = False, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    d = w.desc()
    t, topk = _need_grouped(w, x, topk_ids, y, x_per_pair)
    wp, wb = _ws(ws)
    _check(_lib().qmm_grouped_gemv(ctypes.byref(d), _ptr(x, 2, "x"), int(bool(x_per_pair)),
                                   _ptr(topk_ids, 4, "topk_ids"), t, topk, _ptr(y, 2, "y"), wp, wb,
                                   _stream(stream)), "qmm_grouped_gemv")
    return y


def qmm_grouped_gemv_noalloc(w: PackedWeights, x: torch.Tensor, topk_ids: torch.Tensor, y: torch.Tensor,
                             x_per_pair: bool = False, stream=None) -> torch.Tensor:
    """qmm_grouped_gemv without a workspace: the routing scratch is the
    library's own fixed device array (at most 65536 pairs, 256 experts; calls
    that overlap on the GPU race on it)."""
    d = w.desc()
    t, topk = _need_grouped(w, x, topk_ids, y, x_per_pair)
    _check(_lib().qmm_grouped_gemv_noalloc(ctypes.byref(d), _ptr(x, 2, "x"), int(bool(x_per_pair)),
                                           _ptr(topk_ids, 4, "topk_ids"), t, topk, _ptr(y, 2, "y"),
                                           _stream(stream)), "qmm_grouped_gemv_noalloc")
    return y


def qmm_router_topk(x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor, topk: int,
                    topk_ids: torch.Tensor, topk_weights: torch.Tensor, logits: torch.Tensor | None = None,
                    stream=None):
    """Router logits (fp64 sums rounded once to fp32), fp32 softmax and the
    top-k experts with their softmax weights."""
    t, k = x.shape
    E = w_router.shape[0]
    for tt, nb, name in ((w_router, 2 * E * k, "w_router"), (bias, 4 * E, "bias"),
                         (topk_ids, 4 * t * topk, "topk_ids"), (topk_weights, 4 * t * topk, "topk_weights"),
                         (logits, 4 * t * E, "logits")):
        _need(tt, nb, name)
    _check(_lib().qmm_router_topk(_ptr(x, 2, "x"), _ptr(w_router, 2, "w_router"), _ptr(bias, 4, "bias"), t, k, E,
                                  topk, _ptr(topk_ids, 4, "topk_ids"), _ptr(topk_weights, 4, "topk_weights"),
                                  _ptr(logits, 4, "logits"), _stream(stream)), "qmm_router_topk")
    return topk_ids, topk_weights


def qmm_moe_routed(gate: PackedWeights, up: PackedWeights, down: PackedWeights, x: torch.Tensor,
                   topk_ids: torch.Tensor, topk_weights: torch.Tensor, out: torch.Tensor,
                   ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum_s g[t][s] * W_down,e (SiLU(W_gate,e x_t) * W_up,e x_t)."""
    dg, du, dd = gate.desc(), up.desc(), down.desc()
    t, topk = topk_ids.shape
    wp, wb = _ws(ws)
    _need(x, 2 * t * gate.k, "x")
    _need(topk_weights, 4 * t * topk, "topk_weights")
    _need(out, 2 * t * down.n, "out")
    _check(_lib().qmm_moe_routed(ctypes.byref(dg), ctypes.byref(du), ctypes.byref(dd), _ptr(x, 2, "x"),
                                 _ptr(topk_ids, 4, "topk_ids"), _ptr(topk_weights, 4, "topk_weights"), t, topk,
                                 _ptr(out, 2, "out"), wp, wb, _stream(stream)), "qmm_moe_routed")
    return out


# -- rows grouped by expert ------------------------------------------------------
def _dev() -> int:
    """The current device, -1 before CUDA is in use."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1


def _here(t: torch.Tensor | None, esize: int | None, name: str, dev: int):
    """The address of a tensor that must be on the current device `dev` (the C
    ABI launches there, whatever device the pointer is of)."""
    if t is None:
        return None
    if t.get_device() == dev >= 0 and t.is_contiguous() and (esize is None or t.element_size() == esize):
        return t.data_ptr()
    _ptr(t, esize, name)  # says what is wrong
    raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, dev))


def _half(t: torch.Tensor | None, name: str, dev: int):
    """The address of a tensor of fp16 values that are calculated with:
    torch.float16, or a 16-bit integer type that holds their bits."""
    if t is not None and t.dtype is torch.bfloat16:
        raise ValueError("%s is bfloat16; fp16 values (or their bits as int16) are expected" % name)
    return _here(t, 2, name, dev)


def _weights_here(w: PackedWeights, dev: int) -> None:
    _here(w.data, None, "data", dev)
    _here(w.scales, None, "scales", dev)


def _stream_on(stream, dev: int):
    """The raw handle of the stream (a Stream object costs more than a launch)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def qmm_route_rows(topk_ids: torch.Tensor, num_experts: int, offsets: torch.Tensor, perm: torch.Tensor,
                   rows: torch.Tensor, stream=None):
    """qmm_route with the row of every pair (the inverse of perm): topk_ids
    [t][topk] -> offsets [num_experts+1], perm [t*topk], rows [t][topk]."""
    t, topk = topk_ids.shape
    _need(offsets, 4 * (num_experts + 1), "offsets")
    _need(perm, 4 * t * topk, "perm")
    _need(rows, 4 * t * topk, "rows")
    dev = _dev()
    _check(_lib().qmm_route_rows(_here(topk_ids, 4, "topk_ids", dev), t, topk, num_experts,
                                 _here(offsets, 4, "offsets", dev), _here(perm, 4, "perm", dev),
                                 _here(rows, 4, "rows", dev), _stream_on(stream, dev)), "qmm_route_rows")
    return offsets, perm, rows


def _need_rows(rows: torch.Tensor, tok: torch.Tensor, tok_name: str, sorted_rows, weights=None):
    """(t, topk, d) of a row mover: tok is [t][d], every tensor of
    sorted_rows holds t*topk rows of d."""
    t, topk = rows.shape
    if tok.dim() != 2 or tok.shape[0] != t:
        raise ValueError("%s must be [t][d] for rows of %d tokens" % (tok_name, t))
    d = tok.shape[1]
    for s, name in sorted_rows:
        _need(s, 2 * t * topk * d, name)
    for w, name in weights or ():
        _need(w, 4 * t * topk, name)
    return t, topk, d


def qmm_permute(x: torch.Tensor, rows: torch.Tensor, xs: torch.Tensor, stream=None) -> torch.Tensor:
    """xs[rows[t][s]] = x[t]: x [t][d] -> xs [t*topk][d] (any 2-byte type: the
    values are copied)."""
    t, topk, d = _need_rows(rows, x, "x", ((xs, "xs"),))
    dev = _dev()
    _check(_lib().qmm_permute(_here(x, 2, "x", dev), _here(rows, 4, "rows", dev), t, topk, d, _here(xs, 2, "xs", dev),
                              _stream_on(stream, dev)), "qmm_permute")
    return xs


def qmm_permute_backward(dxs: torch.Tensor, rows: torch.Tensor, dx: torch.Tensor, stream=None) -> torch.Tensor:
    """dx[t] = sum_s dxs[rows[t][s]]: the gradient of qmm_permute."""
    t, topk, d = _need_rows(rows, dx, "dx", ((dxs, "dxs"),))
    dev = _dev()
    _check(_lib().qmm_permute_backward(_half(dxs, "dxs", dev), _here(rows, 4, "rows", dev), t, topk, d,
                                       _half(dx, "dx", dev), _stream_on(stream, dev)), "qmm_permute_backward")
    return dx


def qmm_unpermute(ys: torch.Tensor, rows: torch.Tensor, topk_weights: torch.Tensor | None, out: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """out[t] = sum_s topk_weights[t][s] * ys[rows[t][s]] (weights of 1 when
    None): ys [t*topk][d] -> out [t][d]."""
    t, topk, d = _need_rows(rows, out, "out", ((ys, "ys"),), ((topk_weights, "topk_weights"),))
    dev = _dev()
    _check(_lib().qmm_unpermute(_half(ys, "ys", dev), _here(rows, 4, "rows", dev),
                                _here(topk_weights, 4, "topk_weights", dev), t, topk, d, _half(out, "out", dev),
                                _stream_on(stream, dev)), "qmm_unpermute")
    return out


def qmm_unpermute_backward(dout: torch.Tensor, ys: torch.Tensor, rows: torch.Tensor,
                           topk_weights: torch.Tensor | None, dys: torch.Tensor, dweights: torch.Tensor,
                           stream=None):
    """The gradients of qmm_unpermute: dys [t*topk][d] and dweights [t][topk]."""
    t, topk, d = _need_rows(rows, dout, "dout", ((ys, "ys"), (dys, "dys")),
                            ((topk_weights, "topk_weights"), (dweights, "dweights")))
    dev = _dev()
    _check(_lib().qmm_unpermute_backward(_half(dout, "dout", dev), _half(ys, "ys", dev),
                                         _here(rows, 4, "rows", dev), _here(topk_weights, 4, "topk_weights", dev),
                                         t, topk, d, _half(dys, "dys", dev), _here(dweights, 4, "dweights", dev),
                                         _stream_on(stream, dev)), "qmm_unpermute_backward")
    return dys, dweights


def qmm_grouped_gemm(w: PackedWeights, xs: torch.Tensor, offsets: torch.Tensor, ys: torch.Tensor,
                     stream=None) -> torch.Tensor:
    """ys[r] = W_e xs[r] for the rows offsets[e] <= r < offsets[e+1]."""
    d = w.desc()
    _need(xs, 2 * xs.shape[0] * w.k, "xs")
    _need(ys, 2 * xs.shape[0] * w.n, "ys")
    _need(offsets, 4 * (w.experts + 1), "offsets")
    dev = _dev()
    _weights_here(w, dev)
    _check(_lib().qmm_grouped_gemm(ctypes.byref(d), _half(xs, "xs", dev), _here(offsets, 4, "offsets", dev),
                                   xs.shape[0], _half(ys, "ys", dev), _stream_on(stream, dev)), "qmm_grouped_gemm")
    return ys


def qmm_grouped_swiglu(gate: PackedWeights, up: PackedWeights, xs: torch.Tensor, offsets: torch.Tensor,
                       h: torch.Tensor, stream=None) -> torch.Tensor:
    """h[r] = SiLU(W_gate,e xs[r]) * (W_up,e xs[r]) over the sorted rows."""
    dg, du = gate.desc(), up.desc()
    _need(xs, 2 * xs.shape[0] * gate.k, "xs")
    _need(h, 2 * xs.shape[0] * gate.n, "h")
    _need(offsets, 4 * (gate.experts + 1), "offsets")
    dev = _dev()
    _weights_here(gate, dev)
    _weights_here(up, dev)
    _check(_lib().qmm_grouped_swiglu(ctypes.byref(dg), ctypes.byref(du), _half(xs, "xs", dev),
                                     _here(offsets, 4, "offsets", dev), xs.shape[0], _half(h, "h", dev),
                                     _stream_on(stream, dev)), "qmm_grouped_swiglu")
    return h


# -- low-rank adapters -------------------------------------------------------------
@dataclass
class Adapters:
    """Device tensors of a pool of low-rank adapters plus its C descriptor:
    a [L][rank][k] and b [L][n][rank] (fp16; adapters may be further apart
    than their size), scales [L] fp32, ranks [L] int32 or None."""
    a: torch.Tensor
    b: torch.Tensor
    scales: torch.Tensor
    ranks: torch.Tensor | None = None

    def __setattr__(self, name, value):
        # a new tensor is checked again, also where it lies at the old one's address
        self.__dict__.pop("_desc", None)
        self.__dict__[name] = value

    def desc(self) -> qmm_adapters:
        """The C descriptor, rebuilt only when a tensor was replaced, moved or
        reshaped or another device became current."""
        a, b, s, r = self.a, self.b, self.scales, self.ranks
        key = (a.data_ptr(), b.data_ptr(), s.data_ptr(), a.shape, b.shape, s.shape, a.stride(), b.stride(), s.stride(),
               None if r is None else (r.data_ptr(), r.shape, r.stride()), _dev())
        cached = self.__dict__.get("_desc")
        if cached is not None and cached[0] == key:
            return cached[1]
        d = self._build_desc()
        self.__dict__["_desc"] = (key, d, ctypes.byref(d))
        return d

    def _ref(self):
        self.desc()
        return self.__dict__["_desc"][2]

    def _build_desc(self) -> qmm_adapters:
        a, b = self.a, self.b
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("a must be [L][rank][k] and b [L][n][rank]")
        L, R, k = a.shape
        n = b.shape[1]
        for t, name in ((a, "a"), (b, "b")):
            if t.numel() and not t[0].is_contiguous():
                raise ValueError("%s must have contiguous adapters" % name)
        _need(self.scales, 4 * L, "scales")
        _need(self.ranks, 4 * L, "ranks")
        d = qmm_adapters()
        d.num_adapters, d.n, d.k, d.rank = L, n, k, R
        for t, name in ((a, "a"), (b, "b")):
            if t.dtype is torch.bfloat16:
                raise ValueError("%s is bfloat16; fp16 values (or their bits as int16) are expected" % name)
            if not t.is_cuda:
                raise ValueError("%s must be a CUDA tensor" % name)
            if t.element_size() != 2:
                raise ValueError("%s must have 2-byte elements" % name)
            if t.get_device() != _dev():
                raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, _dev()))
        d.a, d.b = ctypes.c_void_p(a.data_ptr()), ctypes.c_void_p(b.data_ptr())
        d.a_stride = 2 * (a.stride(0) if L > 1 else R * k)
        d.b_stride = 2 * (b.stride(0) if L > 1 else n * R)
        d.scales, d.ranks = _here(self.scales, 4, "scales", _dev()), _here(self.ranks, 4, "ranks", _dev())
        return d


def qmm_lora_workspace_bytes(adapters: Adapters, m: int) -> int:
    return _lib().qmm_lora_workspace_bytes(adapters._ref(), m)


def qmm_lora(adapters: Adapters, x: torch.Tensor, adapter_ids: torch.Tensor, base: torch.Tensor, y: torch.Tensor,
             ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[i] = base[i] + scale_a B_a (A_a x[i]) with a = adapter_ids[i]
    (y[i] = base[i] for -1); y may be base."""
    m, n, k = adapter_ids.numel(), adapters.b.shape[1], adapters.a.shape[2]
    _need(x, 2 * m * k, "x")
    _need(base, 2 * m * n, "base")
    _need(y, 2 * m * n, "y")
    dev = _dev()
    wb = 0 if ws is None else ws.nbytes
    _check(_lib().qmm_lora(adapters._ref(), _half(x, "x", dev), _here(adapter_ids, 4, "adapter_ids", dev), m,
                           _half(base, "base", dev), _half(y, "y", dev), _here(ws, None, "ws", dev), wb,
                           _stream_on(stream, dev)), "qmm_lora")
    return y


DEBUG_WAIT_LIMIT_NS = 1
DEBUG_WITHHOLD_X_TILES = 2
DEBUG_WITHHOLD_TILE_COPIES = 3


def qmm_debug_set(what: int, value: int) -> None:
    """Test hooks of the bounded pipeline waits (include/qmm.h)."""
    _check(_lib().qmm_debug_set(int(what), int(value)), "qmm_debug_set")


def qmm_sync_check(stream=None) -> int:
    return _lib().qmm_sync_check(_stream(stream))


def qmm_last_variant() -> str:
    return _lib().qmm_last_variant().decode()


def qmm_version() -> str:
    return _lib().qmm_version().decode()
