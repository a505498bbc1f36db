"""Double-precision definitions of the operators over grouped rows, and their
error bounds (test code).

U16 is half a step of fp16 relative to the value (the one rounding at the
end), T16 half its smallest spacing; U32 half a step of fp32.  A sum of c
terms held in fp32 is off by at most c steps (2 * U32) of sum |terms|,
whatever the order and even where an adder truncates instead of rounding.
"""
import numpy as np

import oracle

U16, T16, U32 = 2.0 ** -11, 2.0 ** -25, 2.0 ** -24


def sort_rows(ids, E):
    """(offsets, perm, rows) of the stable sort, rows -1 for pairs left out."""
    flat = np.asarray(ids).reshape(-1)
    offsets, perm = [0], []
    for e in range(E):
        perm += [p for p in np.flatnonzero(flat == e)]
        offsets.append(len(perm))
    rows = np.full(flat.size, -1, dtype=np.int32)
    rows[np.asarray(perm, dtype=np.int64)] = np.arange(len(perm), dtype=np.int32)
    return np.asarray(offsets, np.int32), np.asarray(perm, np.int32), rows.reshape(np.asarray(ids).shape)


def unpermute(ys, rows, g):
    """(out, sum |g y|) in double; ys [P][d] double, g [t][topk] double."""
    t, topk = rows.shape
    out, mag = np.zeros((t, ys.shape[1])), np.zeros((t, ys.shape[1]))
    for s in range(topk):
        has = rows[:, s] >= 0
        term = g[has, s, None] * ys[rows[has, s]]
        out[has] += term
        mag[has] += np.abs(term)
    return out, mag


def expert_products(p, xs, offsets):
    """(y, sum |w x|) in double of the sorted rows xs (fp16 bits [rows][k]);
    rows of no expert are NaN.  The E4M3 products follow the library's
    definition: exact code * e4m3 products, the global scale on the sum."""
    rows = xs.shape[0]
    y, a = np.full((rows, p.n), np.nan), np.full((rows, p.n), np.nan)
    x = xs.view(np.float16).astype(np.float64)
    for e in range(p.experts):
        r0, r1 = offsets[e], offsets[e + 1]
        if r1 <= r0:
            continue
        de = p.data[e * p.data_stride:(e + 1) * p.data_stride]
        se = None if p.scales is None else p.scales[e * p.scale_stride:(e + 1) * p.scale_stride]
        gs = 1.0 if p.fmt != 3 else float(p.global_scale)
        w = oracle.dequant(p.fmt, p.n, p.k, de, se, 1.0).view(np.float16).astype(np.float64)
        y[r0:r1] = gs * (x[r0:r1] @ w.T)
        a[r0:r1] = abs(gs) * (np.abs(x[r0:r1]) @ np.abs(w).T)
    return y, a


def product_bound(y, a, k):
    """Bound of an fp16 product of k terms summed in fp32 (and one fp32
    multiply by the global scale)."""
    return U16 * np.abs(y) + 2 * U32 * (k + 2) * a * (1 + U16) + T16


def swiglu_bound(zg, ag, zu, au, k):
    """(h, bound): h = SiLU(zg) zu.  Both sums are off by at most d =
    2 U32 (k + 2) sum |w x|, and |SiLU'| <= 1.1.  The fast exponential is off by
    2 + 1.173 |z| steps (2 U32 each), the fast division by 2, the sum and the
    product by half a step: (4 + 2.35 |z| + 4 + 2) U32 together."""
    dg, du = 2 * U32 * (k + 2) * ag, 2 * U32 * (k + 2) * au
    with np.errstate(over="ignore"):
        s = zg / (1.0 + np.exp(-zg))
    h = s * zu
    err = 1.1 * dg * np.abs(zu) + np.abs(s) * du + 1.1 * dg * du
    rel = (10 + 2.35 * np.abs(zg)) * U32
    err = err + rel * np.abs(h)
    return h, err + U16 * (np.abs(h) + err) + T16


def lora(x, base, ids, A, B, scales, ranks):
    """(y, bound) in double: x [m][k], base [m][n], A [L][R][k], B [L][n][R]."""
    m, k = x.shape
    L, R = A.shape[:2]
    y, err = base.copy(), np.zeros_like(base)
    for i in range(m):
        a = ids[i]
        if not 0 <= a < L:
            continue
        r = R if ranks is None else int(np.clip(ranks[a], 0, R))
        Ar, Br = A[a, :r], B[a][:, :r]
        h, ha = Ar @ x[i], np.abs(Ar) @ np.abs(x[i])
        dh = 2 * U32 * k * ha
        delta, da = Br @ h, np.abs(Br) @ np.abs(h)
        # fp32 sums over rank (two per term where h is held as two fp16 halves, 2^-21 off in all)
        dd = np.abs(Br) @ dh * (1 + U16) + (2 * U32 * (2 * r + 4) + 2.0 ** -21) * da
        s = abs(float(scales[a]))
        y[i] = base[i] + float(scales[a]) * delta
        err[i] = s * dd + 4 * U32 * (np.abs(base[i]) + s * np.abs(delta))
    none = ~((ids >= 0) & (ids < L))
    bound = err + U16 * (np.abs(y) + err) + T16
    bound[none] = 0.0   # rows without an adapter are copied
    return y, bound


def within(got, ref, bound, what=""):
    """|got - ref| <= bound, NaN where the reference is NaN, equal infinities;
    a value whose rounding leaves fp16's range counts as the infinity."""
    got = np.asarray(got, dtype=np.float64)
    over = np.abs(ref) >= 65520.0
    ref = np.where(over, np.sign(ref) * np.inf, ref)
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - ref) <= bound) | (got == ref) | (np.isnan(got) & np.isnan(ref))
        # at the edge of the range either side may round to the infinity
        edge = np.abs(np.abs(np.where(over, 65520.0, np.abs(ref))) - 65520.0) <= bound
        ok |= edge & (np.isinf(got) | (np.abs(got) >= 65472.0))
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError("%s: %d/%d outside; first %s: got %r ref %r bound %r" %
                             (what, (~ok).sum(), ok.size, i, got[i], ref[i], np.broadcast_to(bound, ok.shape)[i]))
