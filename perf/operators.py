"""Cases of the operators over rows that are grouped by an index.

Kinds of case:
  permute    (token, slot) pairs sorted by expert and the token rows laid out
             in that order
  unpermute  the rows brought back: a token's slots times their weights, added
  backward   the gradients of both (of the tokens, of the experts' outputs and
             of the weights)
  experts    the packed experts' products over the sorted rows (one product,
             or SiLU(gate) * up in one pass)
  lora       low-rank adapters of many requests beside a shared projection

With ``own`` false every operator is computed by elementary torch operations
in 32 bits, rounded once at the end; with ``own`` true by the library.
"""
import math

import torch

own = False

IQ4_NL, FP4G16_F16, FP4G16_E4M3, MXFP4 = 1, 2, 3, 4

# Printed tables of the formats.
IQ4_TABLE = (-127, -104, -83, -65, -49, -35, -22, -10, 1, 13, 25, 38, 53, 69, 89, 113)
E2M1_TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of four sequences through a 32-expert layer (hidden 2560, top-4): launch latency
        dict(name="permute_decode", kind="permute", t=4, topk=4, experts=32, d=2560, padded=0),
        # a 2,048-token prefill window of the same layer
        dict(name="permute_prefill", kind="permute", t=2048, topk=4, experts=32, d=2560, padded=0),
        # a small odd batch with padded tokens, more experts than pairs of any one of them
        dict(name="unpermute_decode", kind="unpermute", t=17, topk=6, experts=64, d=2560, padded=3),
        # several windows at once, many experts, an odd token count and padding at the end
        dict(name="unpermute_long", kind="unpermute", t=8191, topk=8, experts=128, d=4096, padded=37),
        # gradients of one window of the 32-expert layer
        dict(name="backward_window", kind="backward", t=2048, topk=4, experts=32, d=2560, padded=0),
        # gradients of a long training batch
        dict(name="backward_long", kind="backward", t=16384, topk=4, experts=64, d=2560, padded=101),
        # gate and up of the 32 IQ4_NL experts (896 x 2560 each) over a prefill window's pairs
        dict(name="experts_gate_up", kind="experts", swiglu=True, fmt=IQ4_NL, experts=32, n=896, k=2560, rows=8192,
             behind=0),
        # their down projection (2560 x 896), the same pairs
        dict(name="experts_down", kind="experts", swiglu=False, fmt=IQ4_NL, experts=32, n=2560, k=896, rows=8192,
             behind=0),
        # one token through an adapter beside the Mamba-2 8B input projection (4096 -> 18560): launch latency
        dict(name="lora_token", kind="lora", m=1, n=18560, k=4096, rank=16, adapters=8, used=1, bare=0, ragged=False),
        # a decode batch of 16 requests, each with its own adapter, beside the output projection (8192 -> 4096)
        dict(name="lora_decode16", kind="lora", m=16, n=4096, k=8192, rank=64, adapters=64, used=16, bare=0,
             ragged=False),
        # decode and prefill rows of many requests mixed, ragged ranks, some requests without an adapter
        dict(name="lora_mixed", kind="lora", m=333, n=18560, k=4096, rank=64, adapters=48, used=40, bare=21,
             ragged=True),
        # a 2,048-token window of four requests, rank 128
        dict(name="lora_prefill", kind="lora", m=2048, n=18560, k=4096, rank=128, adapters=4, used=4, bare=0,
             ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["permute", "unpermute", "backward", "experts", "experts", "lora", "lora"])
    if kind in ("permute", "unpermute", "backward"):
        topk = rng.choice([1, 2, 3, 4, 6, 8])
        experts = rng.choice([8, 13, 32, 64, 128, 256])
        d = rng.choice([8 * rng.randint(16, 512), 896, 2560, 4096])
        # no larger than 16384 tokens of four pairs of 2560
        t = _log_int(rng, 1, min(16384, 16384 * 4 * 2560 // (topk * d)))
        return dict(kind=kind, t=t, topk=topk, experts=experts, d=d, padded=rng.choice([0, 0, t // 7]))
    if kind == "experts":
        fmt = rng.choice([IQ4_NL, IQ4_NL, FP4G16_F16, FP4G16_E4M3, MXFP4])
        swiglu = rng.random() < 0.5
        n, k = (896, 2560) if swiglu else rng.choice([(2560, 896), (1792, 2560), (8 * rng.randint(60, 300), 1024)])
        experts = rng.choice([4, 8, 17, 32])
        rows = _log_int(rng, 1, 8192)
        return dict(kind=kind, swiglu=swiglu, fmt=fmt, experts=experts, n=n, k=k, rows=rows,
                    behind=rng.choice([0, 0, rows // 9]))
    m = _log_int(rng, 1, 2048)
    n, k = rng.choice([(18560, 4096), (4096, 8192), (2560, 896), (1792, 2560), (rng.randint(500, 6000), 2048)])
    adapters = rng.choice([1, 4, 16, 64, 130])
    rank = rng.choice([8, 16, 24, 32, 64, 64, 128])
    return dict(kind=kind, m=m, n=n, k=k, rank=rank, adapters=adapters, used=rng.randint(1, adapters),
                bare=rng.choice([0, 0, m // 5]), ragged=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 12345)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _topk_ids(g, t, topk, experts, padded):
    """Distinct experts per token, some more popular than others; the last
    `padded` tokens belong to no expert (-1)."""
    z = _randn(g, t, experts) + 0.5 * _randn(g, 1, experts)
    v, ids = z.topk(topk, dim=1)
    w = torch.softmax(v, dim=1)
    ids = ids.to(torch.int32)
    if padded:
        ids[t - padded:] = -1
    return ids.contiguous(), w.contiguous()


def _rows_of_pairs(ids, experts):
    """(offsets, perm, row of each pair) by a stable sort; int32, the part of
    perm behind the last routed pair -1."""
    flat = ids.reshape(-1).to(torch.int64)
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    sorted_key = key[order]
    bounds = torch.arange(experts + 1, device=flat.device)
    offsets = torch.searchsorted(sorted_key, bounds)
    routed = sorted_key < experts
    perm = torch.where(routed, order, torch.full_like(order, -1))
    position = torch.arange(flat.numel(), device=flat.device)
    row = torch.empty_like(position)
    row[order] = torch.where(routed, position, torch.full_like(position, -1))
    return offsets.to(torch.int32), perm.to(torch.int32), row.to(torch.int32).reshape(ids.shape)


def _packed(g, fmt, experts, n, k):
    """Packed weights of the format: (data bytes, scale tensor or None, global
    scale), experts one after another."""
    if fmt == IQ4_NL:
        data = torch.randint(0, 256, (experts, n, k // 32, 18), generator=g, device="cuda", dtype=torch.uint8)
        d = (_randn(g, experts, n, k // 32).abs() * 0.002).to(torch.float16)
        data[..., :2] = d.view(torch.uint8).reshape(experts, n, k // 32, 2)
        return data, None, 1.0
    data = torch.randint(0, 256, (experts, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == MXFP4:
        s = _randn(g, experts, n, k // 32).abs().clamp_min(1e-6) * 0.05
        return data, (127.0 + torch.floor(torch.log2(s))).to(torch.uint8), 1.0
    s = _randn(g, experts, n, k // 16).abs() * 0.05
    if fmt == FP4G16_F16:
        return data, s.to(torch.float16), 1.0
    gs = float(s.max() / 448.0)
    return data, (s / gs).to(torch.float8_e4m3fn), gs


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    kind = case["kind"]
    if kind in ("permute", "unpermute", "backward"):
        t, topk, E, d = case["t"], case["topk"], case["experts"], case["d"]
        ids, w = _topk_ids(g, t, topk, E, case["padded"])
        st.update(ids=ids, w=w)
        P = t * topk
        if kind == "permute":
            st["x"] = _randn(g, t, d).to(torch.float16)
            st["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            st["perm"] = torch.full((P,), -1, dtype=torch.int32, device="cuda")
            st["rows"] = torch.full((t, topk), -1, dtype=torch.int32, device="cuda")
            st["xs"] = torch.zeros(P, d, dtype=torch.float16, device="cuda")
        else:
            # the plan that the forward pass left behind
            st["offsets"], st["perm"], st["rows"] = _rows_of_pairs(ids, E)
            st["ys"] = _randn(g, P, d).to(torch.float16)
            if kind == "unpermute":
                st["out"] = torch.zeros(t, d, dtype=torch.float16, device="cuda")
            else:
                st["dout"] = (_randn(g, t, d) * 0.1).to(torch.float16)
                st["dxs"] = (_randn(g, P, d) * 0.1).to(torch.float16)
                st["dx"] = torch.zeros(t, d, dtype=torch.float16, device="cuda")
                st["dys"] = torch.zeros(P, d, dtype=torch.float16, device="cuda")
                st["dw"] = torch.zeros(t, topk, dtype=torch.float32, device="cuda")
    elif kind == "experts":
        E, n, k, rows, fmt = case["experts"], case["n"], case["k"], case["rows"], case["fmt"]
        pop = torch.softmax(0.3 * _randn(g, E), dim=0)
        owner = torch.sort(torch.multinomial(pop, rows, replacement=True, generator=g)).values
        owner = owner[:rows - case["behind"]]   # the rows behind belong to no expert
        st["offsets"] = torch.searchsorted(owner, torch.arange(E + 1, device="cuda")).to(torch.int32)
        st["host_offsets"] = st["offsets"].tolist()
        st["xs"] = _randn(g, rows, k).to(torch.float16)
        st["y"] = torch.zeros(rows, n, dtype=torch.float16, device="cuda")
        st["w"] = [_packed(g, fmt, E, n, k) for _ in range(2 if case["swiglu"] else 1)]
        if own:
            from packed_bit_weight_b200 import qmm
            st["pw"] = [qmm.PackedWeights(fmt, n, k, data.reshape(-1),
                                          None if s is None else s.view(torch.uint8).reshape(-1), gs, E)
                        for data, s, gs in st["w"]]
    else:
        m, n, k, R, L = case["m"], case["n"], case["k"], case["rank"], case["adapters"]
        st["x"] = _randn(g, m, k).to(torch.float16)
        st["base"] = _randn(g, m, n).to(torch.float16)
        st["a"] = (_randn(g, L, R, k) / math.sqrt(k)).to(torch.float16)
        st["b"] = (_randn(g, L, n, R) * 0.05).to(torch.float16)
        st["scales"] = (2.0 / R) * (4.0 + torch.rand(L, generator=g, device="cuda"))
        st["ranks"] = None
        if case["ragged"]:
            st["ranks"] = torch.randint(1, R + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
            st["ranks"][0] = R
        # requests are runs of rows (prefill pieces and single tokens); the last `bare` rows have no adapter
        chosen = torch.randperm(L, generator=g, device="cuda")[:case["used"]]
        if m <= 2 * case["used"]:
            pick = torch.arange(m, device="cuda") % case["used"]
        else:
            pick = torch.sort(torch.randint(0, case["used"], (m,), generator=g, device="cuda")).values
        ids = chosen[pick].to(torch.int32)
        if case["bare"]:
            ids[m - case["bare"]:] = -1
        st["ids"] = ids.contiguous()
        st["host_ids"] = sorted(set(i for i in st["ids"].tolist() if i >= 0))
        st["y"] = torch.zeros(m, n, dtype=torch.float16, device="cuda")
        if own:
            from packed_bit_weight_b200 import qmm
            st["adapters"] = qmm.Adapters(st["a"], st["b"], st["scales"], st["ranks"])
            st["ws"] = torch.empty(qmm.qmm_lora_workspace_bytes(st["adapters"], m), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _run_own(st):
    from packed_bit_weight_b200 import qmm
    case = st["case"]
    kind = case["kind"]
    if kind == "permute":
        qmm.qmm_route_rows(st["ids"], case["experts"], st["offsets"], st["perm"], st["rows"])
        qmm.qmm_permute(st["x"], st["rows"], st["xs"])
        return st["offsets"], st["perm"], st["rows"], st["xs"]
    if kind == "unpermute":
        return qmm.qmm_unpermute(st["ys"], st["rows"], st["w"], st["out"])
    if kind == "backward":
        qmm.qmm_unpermute_backward(st["dout"], st["ys"], st["rows"], st["w"], st["dys"], st["dw"])
        qmm.qmm_permute_backward(st["dxs"], st["rows"], st["dx"])
        return st["dx"], st["dys"], st["dw"]
    if kind == "experts":
        if case["swiglu"]:
            return qmm.qmm_grouped_swiglu(st["pw"][0], st["pw"][1], st["xs"], st["offsets"], st["y"])
        return qmm.qmm_grouped_gemm(st["pw"][0], st["xs"], st["offsets"], st["y"])
    return qmm.qmm_lora(st["adapters"], st["x"], st["ids"], st["base"], st["y"], ws=st["ws"])


def _nibbles(b):
    return b & 15, b >> 4


def _weights32(fmt, packed, e):
    """(decoded weights [n][k] in fp32, factor of the sum) of expert e."""
    data, scales, gs = packed
    if fmt == IQ4_NL:
        blocks = data[e]
        n, nb = blocks.shape[:2]
        d = blocks[..., :2].contiguous().view(torch.float16).float()
        lo, hi = _nibbles(blocks[..., 2:].long())
        table = torch.tensor(IQ4_TABLE, dtype=torch.float32, device=data.device)
        w = torch.cat([table[lo], table[hi]], dim=-1) * d
        return w.to(torch.float16).float().reshape(n, nb * 32), 1.0
    n, half = data[e].shape
    lo, hi = _nibbles(data[e].long())
    table = torch.tensor(E2M1_TABLE, dtype=torch.float32, device=data.device)
    codes = torch.stack([table[lo], table[hi]], dim=-1).reshape(n, half * 2)
    if fmt == MXFP4:
        s = torch.exp2(scales[e].float() - 127.0).repeat_interleave(32, dim=1)
        return (codes * s).to(torch.float16).float(), 1.0
    s = scales[e].float().repeat_interleave(16, dim=1)
    return (codes * s).to(torch.float16).float(), gs


def _run_plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "permute":
        offsets, perm, rows = _rows_of_pairs(st["ids"], case["experts"])
        has = perm >= 0
        token = torch.where(has, perm, torch.zeros_like(perm)).long() // case["topk"]
        xs = torch.where(has[:, None], st["x"][token], torch.zeros((), dtype=torch.float16, device="cuda"))
        return offsets, perm, rows, xs
    if kind in ("unpermute", "backward"):
        rows = st["rows"].long()
        has = rows >= 0
        at = torch.where(has, rows, torch.zeros_like(rows))
        if kind == "unpermute":
            acc = torch.zeros(st["out"].shape, dtype=torch.float32, device="cuda")
            for s in range(case["topk"]):
                g = torch.where(has[:, s], st["w"][:, s], torch.zeros_like(st["w"][:, s]))
                acc += g[:, None] * st["ys"][at[:, s]].float() * has[:, s, None]
            return acc.to(torch.float16)
        dx = torch.zeros(st["dx"].shape, dtype=torch.float32, device="cuda")
        dys = torch.zeros_like(st["dys"])
        dw = torch.zeros_like(st["dw"])
        dout = st["dout"].float()
        for s in range(case["topk"]):
            h = has[:, s]
            dx += st["dxs"][at[:, s]].float() * h[:, None]
            dw[:, s] = (st["ys"][at[:, s]].float() * dout).sum(1) * h
            dys[at[h, s]] = (st["w"][h, s, None] * dout[h]).to(torch.float16)
        return dx.to(torch.float16), dys, dw
    if kind == "experts":
        y = torch.zeros_like(st["y"])
        for e in range(case["experts"]):
            r0, r1 = st["host_offsets"][e], st["host_offsets"][e + 1]
            if r1 == r0:
                continue
            x = st["xs"][r0:r1].float()
            out = []
            for packed in st["w"]:
                w, gs = _weights32(case["fmt"], packed, e)
                out.append((x @ w.t()) * gs)
            if case["swiglu"]:
                out = [out[0] / (1.0 + torch.exp(-out[0])) * out[1]]
            y[r0:r1] = out[0].to(torch.float16)
        return y
    y = st["base"].clone()
    for a in st["host_ids"]:
        at = (st["ids"] == a).nonzero().squeeze(1)
        A, B = st["a"][a].float(), st["b"][a].float()
        if st["ranks"] is not None:
            keep = torch.arange(case["rank"], device="cuda") < st["ranks"][a]
            A, B = A * keep[:, None], B * keep[None, :]
        h = st["x"][at].float() @ A.t()
        y[at] = (st["base"][at].float() + st["scales"][a] * (h @ B.t())).to(torch.float16)
    return y


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _packed_bytes(fmt, n, k):
    return n * k * {IQ4_NL: 18 / 32, FP4G16_F16: 0.625, FP4G16_E4M3: 0.5625, MXFP4: 17 / 32}[fmt]


def work(case):
    kind = case["kind"]
    if kind in ("permute", "unpermute", "backward"):
        t, d = case["t"], case["d"]
        P = t * case["topk"]
        live = (t - case["padded"]) * case["topk"]
        if kind == "permute":
            return dict(bytes=12 * P + 4 * case["experts"] + 2 * (t - case["padded"]) * d + 2 * live * d, flops=0)
        if kind == "unpermute":
            return dict(bytes=8 * P + 2 * live * d + 2 * t * d, flops=2 * live * d)
        return dict(bytes=12 * P + 2 * t * d + 6 * live * d + 2 * t * d, flops=4 * live * d)
    if kind == "experts":
        E, n, k, rows = case["experts"], case["n"], case["k"], case["rows"] - case["behind"]
        mats = 2 if case["swiglu"] else 1
        hit = E * (1.0 - (1.0 - 1.0 / E) ** rows)   # experts that have a row, for even routing
        return dict(bytes=int(mats * hit * _packed_bytes(case["fmt"], n, k) + 2 * rows * (n + k)),
                    flops=2 * mats * rows * n * k)
    m, n, k, R = case["m"], case["n"], case["k"], case["rank"]
    live = m - case["bare"]
    used = min(case["used"], live)
    mean = 0.5 if case["ragged"] else 1.0
    return dict(bytes=int(2 * used * mean * R * (n + k) + 2 * live * k + 4 * m * n + 4 * m),
                flops=int(2 * live * mean * R * (n + k)))


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _decode64(fmt, packed, e):
    """Weights of expert e in double, element by element from the bytes."""
    data, scales, _ = packed
    raw = data[e].cpu()
    if fmt == IQ4_NL:
        n, nb = raw.shape[:2]
        d = raw[:, :, 0:2].contiguous().view(torch.float16).double()
        q = raw[:, :, 2:].int()
        table = torch.tensor(IQ4_TABLE, dtype=torch.float64)
        w = torch.empty(n, nb, 32, dtype=torch.float64)
        w[:, :, :16] = table[(q % 16).long()]
        w[:, :, 16:] = table[(q // 16).long()]
        return (w * d).half().double().reshape(n, nb * 32).cuda()
    n, half = raw.shape
    table = torch.tensor(E2M1_TABLE, dtype=torch.float64)
    w = torch.empty(n, 2 * half, dtype=torch.float64)
    w[:, 0::2] = table[(raw.int() % 16).long()]
    w[:, 1::2] = table[(raw.int() // 16).long()]
    s = scales[e].cpu()
    group = 2 * half // s.shape[1]
    s = torch.pow(2.0, s.double() - 127.0) if fmt == MXFP4 else s.double()
    return (w.reshape(n, -1, group) * s[:, :, None]).half().double().reshape(n, 2 * half).cuda()


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("permute", "unpermute", "backward"):
        ids = st["ids"].cpu().reshape(-1).tolist()
        t, topk, E = case["t"], case["topk"], case["experts"]
        buckets = [[] for _ in range(E)]
        for p, e in enumerate(ids):
            if 0 <= e < E:
                buckets[e].append(p)
        offsets, perm = [0], []
        for b in buckets:
            perm += b
            offsets.append(len(perm))
        rows = [-1] * len(ids)
        for r, p in enumerate(perm):
            rows[p] = r
        p = torch.tensor(perm, dtype=torch.int64, device="cuda")
        r = torch.arange(len(perm), device="cuda")
        if kind == "permute":
            xs = torch.zeros(t * topk, case["d"], dtype=torch.float64, device="cuda")
            xs[r] = st["x"].double()[p // topk]
            full = torch.tensor(perm + [-1] * (t * topk - len(perm)), dtype=torch.int32)
            return (torch.tensor(offsets, dtype=torch.int32), full,
                    torch.tensor(rows, dtype=torch.int32).reshape(t, topk), xs)
        w = st["w"].double().reshape(-1)
        if kind == "unpermute":
            out = torch.zeros(t, case["d"], dtype=torch.float64, device="cuda")
            return out.index_add_(0, p // topk, st["ys"].double()[r] * w[p, None])
        dx = torch.zeros(t, case["d"], dtype=torch.float64, device="cuda")
        dx.index_add_(0, p // topk, st["dxs"].double()[r])
        dys = torch.zeros(t * topk, case["d"], dtype=torch.float64, device="cuda")
        dys[r] = st["dout"].double()[p // topk] * w[p, None]
        dw = torch.zeros(t * topk, dtype=torch.float64, device="cuda")
        dw[p] = torch.einsum("ij,ij->i", st["ys"].double()[r], st["dout"].double()[p // topk])
        return dx, dys, dw.reshape(t, topk)
    if kind == "experts":
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            r0, r1 = st["host_offsets"][e], st["host_offsets"][e + 1]
            if r0 < r1:
                x = st["xs"][r0:r1].double()
                z = [float(packed[2]) * (x @ _decode64(case["fmt"], packed, e).t()) for packed in st["w"]]
                y[r0:r1] = z[0] * torch.sigmoid(z[0]) * z[1] if case["swiglu"] else z[0]
        return y
    y = st["base"].double()
    for a in st["host_ids"]:
        at = torch.tensor([i for i, v in enumerate(st["ids"].tolist()) if v == a], device="cuda")
        r = case["rank"] if st["ranks"] is None else int(st["ranks"][a])
        delta = (st["x"][at].double() @ st["a"][a, :r].double().t()) @ st["b"][a, :, :r].double().t()
        y[at] += float(st["scales"][a]) * delta
    return y
