"""Cases that measure the router, the grouping of its choices and the experts' 8-bit products.

Each case runs one pass of an operator in one of two ways: through the
package's entry points (``own`` true), or as elementary torch operations in 32
bits (``own`` false), the definition the kernels are compared with.  ``exact``
gives the same outputs computed in 64 bits, written apart from both.

Operators:
  gate      router logits -> the K experts of every token and their weights
  gate_loss the same with the balance loss and per-expert counts, and the
            gradient of both with respect to the logits
  group     expert ids -> rows grouped by slot (offsets, order, place)
  product   tokens x expert weights in 8-bit floating point with a scale for
            each block of 128, rows grouped by expert
  train     one training step of that product: weights and activations
            quantised, the product, and its gradients
"""
from __future__ import annotations

import torch

own = False

EPS = 1e-20                  # added to a sum of scores before it divides
F8_MAX = 448.0               # largest finite value of the 8-bit format (4 exponent bits, 3 of mantissa)
AMAX_MIN = 2.0 ** -100       # blocks of smaller values are scaled as if this were their largest
BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded token through the router of a 256-expert layer (8 groups, 4 kept): latency only
        {"name": "gate_one_token", "op": "gate", "T": 1, "E": 256, "K": 8, "G": 8, "top_groups": 4,
         "scoring": "sigmoid", "dtype": "f32"},
        # prefill step of the 58-layer deployment: 16384 tokens of one layer, 8 of 256 experts
        {"name": "gate_prefill", "op": "gate", "T": 16384, "E": 256, "K": 8, "G": 8, "top_groups": 4,
         "scoring": "sigmoid", "dtype": "bf16"},
        # a small training batch of ragged sequences (one of them empty), plain softmax routing, odd expert count
        {"name": "loss_ragged", "op": "gate_loss", "T": 999, "E": 60, "K": 6, "G": 1, "top_groups": 1, "S": 7,
         "scoring": "softmax", "dtype": "bf16"},
        # a training batch: 16384 tokens in 4 sequences, 256 experts, router logits kept in 32 bits
        {"name": "loss_train", "op": "gate_loss", "T": 16384, "E": 256, "K": 8, "G": 8, "top_groups": 4, "S": 4,
         "scoring": "sigmoid", "dtype": "f32"},
        # a decode batch of 64 tokens grouped by 320 physical slots: launch latency counts
        {"name": "group_decode", "op": "group", "L": 1, "T": 64, "K": 8, "P": 320},
        # a prefill step grouped by the 288 slots of the placement
        {"name": "group_prefill", "op": "group", "L": 1, "T": 16384, "K": 8, "P": 288},
        # one token through its 8 experts of 32 on this GPU: 8 rows, the weights are what is read
        {"name": "product_one_token", "op": "product", "T": 1, "K": 8, "G": 32, "H": 2048, "N": 4096, "dtype": "bf16"},
        # a decode step's rows on one rank of 9 slots (288 slots on 32 ranks)
        {"name": "product_decode", "op": "product", "T": 256, "K": 2, "G": 9, "H": 4096, "N": 2048, "dtype": "bf16"},
        # a shared expert (one group) at sizes that fill no tile
        {"name": "product_odd", "op": "product", "T": 1000, "K": 1, "G": 1, "H": 1040, "N": 1391, "dtype": "f16"},
        # a prefill step's rows on one rank of 9 slots: the matrix cores are what counts
        {"name": "product_prefill", "op": "product", "T": 8192, "K": 2, "G": 9, "H": 4096, "N": 4096, "dtype": "bf16"},
        # a fine-tuning micro-batch over 5 experts, sizes that fill no tile
        {"name": "train_odd", "op": "train", "T": 301, "K": 2, "G": 5, "H": 1040, "N": 720, "dtype": "bf16"},
        # a training micro-batch on one rank of 9 slots
        {"name": "train_step", "op": "train", "T": 8192, "K": 2, "G": 9, "H": 4096, "N": 2048, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["gate", "gate_loss", "group", "product", "product", "train"])
    if op in ("gate", "gate_loss"):
        G = rng.choice([1, 1, 4, 8])
        E = G * log(8, 512 // G)
        top_groups = G if G == 1 else rng.randint(G // 2, G)
        K = rng.randint(1, min(8, top_groups * (E // G)))
        case = {"op": op, "T": log(1, 16384), "E": E, "K": K, "G": G, "top_groups": top_groups,
                "scoring": rng.choice(["sigmoid", "softmax"]), "dtype": rng.choice(["f32", "bf16", "f16"])}
        if case["T"] * E > 16384 * 256:
            case["T"] = 16384 * 256 // E
        if op == "gate_loss":
            case["S"] = rng.randint(1, 16)
        return case
    if op == "group":
        return {"op": op, "L": rng.randint(1, 4), "T": log(1, 4096), "K": rng.randint(1, 8), "P": log(8, 512)}
    G = rng.randint(1, 16)
    K = rng.randint(1, min(4, G))
    H, N = 16 * log(8, 256), (16 * log(8, 256) if op == "train" else log(128, 4096))
    T = log(1, 8192)
    while T * K * H * N > 8192 * 2 * 4096 * 2048:
        T = T // 2 + 1
    return {"op": op, "T": T, "K": K, "G": G, "H": H, "N": N, "dtype": rng.choice(["f32", "bf16", "f16"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _slot_ids(g, T, K, P):
    """K distinct slots for every token, mildly uneven as a balanced placement
    leaves them; one id in fifty is -1 (a choice served elsewhere)."""
    key = torch.rand((T, P), generator=g, device="cuda") + 0.2 * torch.rand((P,), generator=g, device="cuda")
    ids = key.topk(K, dim=1).indices.to(torch.int32)
    away = torch.rand((T, K), generator=g, device="cuda") < 0.02
    return torch.where(away, torch.full_like(ids, -1), ids)


def _grouped(ids, P):
    """offsets [L, P + 1], order [L, n], place [L, n] of ids [L, n]; ids outside
    [0, P) come last."""
    L, n = ids.shape
    key = torch.where((ids >= 0) & (ids < P), ids, torch.full_like(ids, P))
    order = torch.sort(key, dim=1, stable=True).indices
    place = torch.empty_like(order)
    place.scatter_(1, order, torch.arange(n, device=ids.device).expand(L, n).contiguous())
    count = (key.unsqueeze(1) == torch.arange(P, device=ids.device).view(1, P, 1)).sum(2) if n <= 4096 else \
        torch.zeros((L, P + 1), dtype=torch.int64, device=ids.device).scatter_add_(
            1, key.long(), torch.ones_like(key, dtype=torch.int64))[:, :P]
    offsets = torch.zeros((L, P + 1), dtype=torch.int64, device=ids.device)
    offsets[:, 1:] = count.cumsum(1)
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("gate", "gate_loss"):
        T, E, K = case["T"], case["E"], case["K"]
        dt = DTYPES[case["dtype"]]
        st["logits"] = (1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)).to(dt)
        # the selection bias of a router trained without an auxiliary loss: multiples of its update step
        st["bias"] = 0.001 * torch.randint(-80, 81, (E,), generator=g, device="cuda").float() \
            if case["scoring"] == "sigmoid" else None
        st["mask"] = torch.rand((T,), generator=g, device="cuda") >= (0.03 if T > 1 else 0.0)   # padding rows
        if op == "gate_loss":
            S = case["S"]
            cut = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
            seg = torch.zeros((S + 1,), dtype=torch.int32, device="cuda")
            seg[1:S] = cut
            if S > 2:
                seg[2] = seg[1]                                           # an empty sequence
            seg[S] = T
            st["seg"] = seg
            st["d_weights"] = 1e-2 * _randn(g, T, K)
            st["d_loss"] = torch.rand((S,), generator=g, device="cuda") + 0.5
            st["alpha"] = 0.1
        return st
    if op == "group":
        ids = [_slot_ids(g, case["T"], min(case["K"], case["P"]), case["P"]) for _ in range(case["L"])]
        st["ids"] = torch.stack(ids)
        return st
    T, K, G, H, N = (case[k] for k in "TKGHN")
    dt = DTYPES[case["dtype"]]
    # activations: unit normal with a few channels an order of magnitude larger
    channel = torch.where(torch.rand((H,), generator=g, device="cuda") < 0.01, 12.0, 1.0)
    st["x"] = (_randn(g, T, H) * channel).to(dt)
    w = (_randn(g, G, N, H) * H ** -0.5).to(dt)
    offsets, order, _ = _grouped(_slot_ids(g, T, K, G).view(1, -1), G)
    st["offsets"], st["order"] = offsets[0].contiguous(), order[0].contiguous()
    st["cap"] = max(1, int((st["offsets"][1:] - st["offsets"][:-1]).max()))   # rows of the fullest expert
    if op == "product":
        st["wq"], st["ws"] = _quantize_weights(w)
    else:
        st["w"] = w
        st["dy"] = (1e-3 * _randn(g, T * K, N)).to(dt)
    return st


# ------------------------------------------------------------------ plain forms
def _ranked(key, K):
    """The K largest of each row, ties to the lowest index: (values, indices)."""
    v, i = torch.sort(key, dim=1, descending=True, stable=True)
    return v[:, :K], i[:, :K]


def _scores(st):
    x = st["logits"].float()
    if st["case"]["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
        key = s + st["bias"]
    else:
        m = x.max(1, keepdim=True).values
        e = torch.exp(x - torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m))
        s = e / (e.sum(1, keepdim=True) + EPS)
        key = x
    return s, torch.where(torch.isnan(key), torch.full_like(key, -torch.inf), key)


def _select(st, s, key):
    c = st["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    if c["top_groups"] < G:
        per = key.view(T, G, E // G)
        top = 2 if c["scoring"] == "sigmoid" else 1
        score = _ranked(per.reshape(T * G, E // G), top)[0].sum(1).view(T, G)
        kept = _ranked(score, c["top_groups"])[1]
        keep = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, kept, True)
        key = torch.where(keep.unsqueeze(2), per, torch.full_like(per, -torch.inf)).view(T, E)
    v, i = _ranked(key, K)
    ok = (v > -torch.inf) & st["mask"].unsqueeze(1)
    w = torch.where(ok, s.gather(1, i), torch.zeros_like(v))
    total = w.sum(1, keepdim=True) + EPS
    return torch.where(ok, i, torch.full_like(i, -1)).to(torch.int32), w, total


def _segments(st):
    """[S, T]: one where the row is a real token of the segment."""
    seg, T, S = st["seg"], st["case"]["T"], st["case"]["S"]
    row = torch.arange(T, device=seg.device)
    inside = (row >= seg[:-1].unsqueeze(1)) & (row < seg[1:].unsqueeze(1))
    return (inside & st["mask"]).float()


def _gate_loss_plain(st):
    c = st["case"]
    T, E, K = c["T"], c["E"], c["K"]
    s, key = _scores(st)
    ids, w, total = _select(st, s, key)
    member = _segments(st)
    ok = ids >= 0
    picked = torch.zeros((T, E + 1), device=s.device).scatter_(1, torch.where(ok, ids, E).long(), 1.0)[:, :E]
    counts = member @ picked
    tokens = member.sum(1)
    share = s / (s.sum(1, keepdim=True) + EPS) if c["scoring"] == "sigmoid" else s
    n = tokens.clamp(min=1.0).unsqueeze(1)
    prob = (member @ share) / n
    f = counts * E / (K * n)
    loss = st["alpha"] * (f * prob).sum(1)
    # gradient of sum(d_weights * weights) + sum(d_loss * loss)
    gw = torch.where(ok, st["d_weights"], torch.zeros_like(w)) * 2.5
    gsel = (gw - (gw * w).sum(1, keepdim=True) / total) / total
    gs = torch.zeros((T, E + 1), device=s.device).scatter_(1, torch.where(ok, ids, E).long(), gsel)[:, :E]
    a = member.t() @ (f * (st["alpha"] * st["d_loss"]).unsqueeze(1) / n)
    if c["scoring"] == "sigmoid":
        gs = gs + (a - (a * share).sum(1, keepdim=True)) / (s.sum(1, keepdim=True) + EPS)
        dx = gs * s * (1.0 - s)
    else:
        gs = gs + a
        dx = s * (gs - (gs * s).sum(1, keepdim=True))
    dx = torch.where(st["mask"].unsqueeze(1), dx, torch.zeros_like(dx)).to(st["logits"].dtype)
    return {"ids": ids, "weights": 2.5 * w / total, "loss": loss, "counts": counts.to(torch.int32), "prob": prob,
            "tokens": tokens.to(torch.int32), "d_logits": dx}


def _quantize(x):
    """x [..., C] as 8-bit values and a scale for each block of 128 of the last axis."""
    C = x.shape[-1]
    nb = -(-C // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - C)).view(*x.shape[:-1], nb, BLOCK)
    amax = v.abs().amax(-1).clamp(min=AMAX_MIN)
    q = (v * (F8_MAX / amax).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(*x.shape[:-1], nb * BLOCK)[..., :C], amax / F8_MAX


def _dequantize(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]


def _quantize_weights(w):
    """w [G, N, K] as 8-bit values and a scale for each 128 x 128 block."""
    G, N, K = w.shape
    nn, nk = -(-N // BLOCK), -(-K // BLOCK)
    v = torch.nn.functional.pad(w.float(), (0, nk * BLOCK - K, 0, nn * BLOCK - N)).view(G, nn, BLOCK, nk, BLOCK)
    amax = v.abs().amax((2, 4)).clamp(min=AMAX_MIN)
    q = (v * (F8_MAX / amax)[:, :, None, :, None]).to(torch.float8_e4m3fn).view(G, nn * BLOCK, nk * BLOCK)
    return q[:, :N, :K].contiguous(), amax / F8_MAX


def _dequantize_weights(q, scale):
    G, N, K = q.shape
    return q.float() * scale.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]


def _layout(st, rows):
    """Where row r of the grouped order stands in a [G * cap + 1] padded layout (rows of no expert: the last)."""
    off, cap = st["offsets"].long(), st["cap"]
    r = torch.arange(rows, device=off.device)
    g = torch.searchsorted(off[1:], r, right=True)
    inside = g < off.numel() - 1
    g = g.clamp(max=off.numel() - 2)
    return torch.where(inside, g * cap + r - off[g], (off.numel() - 1) * cap)


def _pad(v, at, G, cap):
    out = torch.zeros((G * cap + 1, v.shape[1]), device=v.device)
    out[at] = v
    return out[:G * cap].view(G, cap, v.shape[1])


def _unpad(v, at):
    flat = torch.cat([v.reshape(-1, v.shape[2]), torch.zeros((1, v.shape[2]), device=v.device)])
    return flat[at]


def _column_blocks(v):
    """v [G, cap, C] quantised down the rows in blocks of 128 and taken back: what the weight gradient's product reads."""
    G, cap, C = v.shape
    nb = -(-cap // BLOCK)
    b = torch.nn.functional.pad(v, (0, 0, 0, nb * BLOCK - cap)).view(G, nb, BLOCK, C)
    amax = b.abs().amax(2, keepdim=True).clamp(min=AMAX_MIN)
    q = (b * (F8_MAX / amax)).to(torch.float8_e4m3fn).float() * (amax / F8_MAX)
    return q.view(G, nb * BLOCK, C)


def _product_plain(st, wq, ws):
    c = st["case"]
    T, K, G = c["T"], c["K"], c["G"]
    at = _layout(st, T * K)
    x = _dequantize(*_quantize(st["x"]))[st["order"].long() // K]
    w = _dequantize_weights(wq, ws).transpose(1, 2).contiguous()
    return _unpad(torch.bmm(_pad(x, at, G, st["cap"]), w), at).to(torch.bfloat16)


def _train_plain(st):
    c = st["case"]
    T, K, G = c["T"], c["K"], c["G"]
    wq, ws = _quantize_weights(st["w"])
    y = _product_plain(st, wq, ws)
    at = _layout(st, T * K)
    dy = _dequantize(*_quantize(st["dy"]))
    dx = _unpad(torch.bmm(_pad(dy, at, G, st["cap"]), _dequantize_weights(wq, ws)), at).to(torch.bfloat16)
    xc = _column_blocks(_pad(st["x"].float()[st["order"].long() // K], at, G, st["cap"]))
    dyc = _column_blocks(_pad(st["dy"].float(), at, G, st["cap"]))
    return {"y": y, "dx": dx, "dw": torch.bmm(dyc.transpose(1, 2).contiguous(), xc)}


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import moe_expert_load_eplb_amd as eplb
        if op in ("gate", "gate_loss"):
            how = dict(scoring=c["scoring"], normalize=True, scale=2.5, mask=st["mask"])
            pick = dict(bias=st["bias"], G=c["G"], top_groups=c["top_groups"],
                        group_top=2 if c["scoring"] == "sigmoid" else 1)
        if op == "gate":
            ids, weights = eplb.gate(st["logits"], c["K"], **how, **pick)
            return {"ids": ids, "weights": weights}
        if op == "gate_loss":
            ids, weights, loss, counts, prob, tokens = eplb.gate_loss(
                st["logits"], c["K"], st["seg"], st["alpha"], **how, **pick)
            dx = eplb.gate_backward(st["logits"], ids, st["d_weights"], seg=st["seg"], alpha=st["alpha"],
                                    counts=counts, tokens=tokens, d_loss=st["d_loss"], **how)
            return {"ids": ids, "weights": weights, "loss": loss, "counts": counts, "prob": prob, "tokens": tokens,
                    "d_logits": dx}
        if op == "group":
            return list(eplb.group_rows(st["ids"], c["P"]))
        q, s = eplb.quantize_rows(st["x"])
        if op == "product":
            return eplb.expert_matmul(q, s, st["wq"], st["ws"], st["offsets"], rows=st["order"], K=c["K"])
        wq, ws, wqt, wst = eplb.quantize_weights(st["w"], transpose=True)
        y = eplb.expert_matmul(q, s, wq, ws, st["offsets"], rows=st["order"], K=c["K"])
        dq, ds = eplb.quantize_rows(st["dy"])
        dx = eplb.expert_matmul(dq, ds, wqt, wst, st["offsets"])
        xc, xcs = eplb.quantize_columns(st["x"], st["offsets"], rows=st["order"], K=c["K"])
        dyc, dycs = eplb.quantize_columns(st["dy"], st["offsets"])
        return {"y": y, "dx": dx, "dw": eplb.expert_wgrad(dyc, dycs, xc, xcs, st["offsets"])}
    if op == "gate":
        s, key = _scores(st)
        ids, w, total = _select(st, s, key)
        return {"ids": ids, "weights": 2.5 * w / total}
    if op == "gate_loss":
        return _gate_loss_plain(st)
    if op == "group":
        ids = st["ids"]
        return list(_grouped(ids.view(ids.shape[0], -1), c["P"]))
    if op == "product":
        return _product_plain(st, st["wq"], st["ws"])
    return _train_plain(st)


def work(case):
    """Bytes with each input read once and each output written once, and operations, of one pass."""
    op = case["op"]
    size = 4 if case.get("dtype") == "f32" else 2
    if op in ("gate", "gate_loss"):
        T, E, K = case["T"], case["E"], case["K"]
        per = T * E * size + T + 4 * E
        if op == "gate":
            return {"bytes": per + 8 * T * K, "flops": 4 * T * E}
        S = case["S"]
        return {"bytes": per + T * E * size + 12 * T * K + 8 * S * E + 16 * S, "flops": 12 * T * E}
    if op == "group":
        n = case["L"] * case["T"] * case["K"]
        return {"bytes": 12 * n + 4 * case["L"] * (case["P"] + 1), "flops": n}
    T, K, G, H, N = (case[k] for k in "TKGHN")
    R = T * K
    blocks = -(-H // BLOCK) * -(-N // BLOCK)
    if op == "product":
        used = min(G, R)
        return {"bytes": T * H * size + used * (N * H + 4 * blocks) + 2 * R * N + 4 * R, "flops": 2 * R * N * H}
    return {"bytes": size * (T * H + R * N + G * N * H) + 2 * R * (N + H) + 4 * G * N * H + 4 * R,
            "flops": 6 * R * N * H}


# ------------------------------------------------------------------ the definition in 64 bits
def _round_f8(v):
    """v to the nearest 8-bit value (1 sign, 4 exponent, 3 mantissa bits; ties to even)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-F8_MAX, F8_MAX)


def _blocked(v, dims):
    """v taken to 8 bits and back, one scale for each block of 128 along every axis in dims.  Scales and scaled values
    are 32-bit numbers by definition (they decide which 8-bit value is the nearest); what they stand for is 64-bit."""
    amax = v.abs()
    for d in dims:
        parts = amax.split(BLOCK, d)
        amax = torch.cat([p.amax(d, keepdim=True).expand_as(p) for p in parts], d)
    amax = amax.clamp(min=AMAX_MIN).float()
    return _round_f8((v.float() * (F8_MAX / amax)).double()) * (amax / F8_MAX).double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "group":
        return None
    if op in ("gate", "gate_loss"):
        return _exact_gate(st)
    T, K, G, H, N = (case[k] for k in "TKGHN")
    R = T * K
    off = st["offsets"].tolist()
    x64 = st["x"].double()
    token = st["order"].long() // K
    xr = _blocked(x64, (1,))
    y = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    if op == "product":
        for g in range(G):
            lo, hi = off[g], off[g + 1]
            w = st["wq"][g].double() * st["ws"][g].double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :H]
            y[lo:hi] = xr[token[lo:hi]] @ w.t()
        return y
    dx = torch.zeros((R, H), dtype=torch.float64, device="cuda")
    dw = torch.zeros((G, N, H), dtype=torch.float64, device="cuda")
    dy64 = st["dy"].double()
    dyr = _blocked(dy64, (1,))
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            continue
        w = _blocked(st["w"][g].double(), (0, 1))
        y[lo:hi] = xr[token[lo:hi]] @ w.t()
        dx[lo:hi] = dyr[lo:hi] @ w
        dw[g] = _blocked(dy64[lo:hi], (0,)).t() @ _blocked(x64[token[lo:hi]], (0,))
    return {"y": y, "dx": dx, "dw": dw}


def _exact_gate(st):
    c = st["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    sigmoid = c["scoring"] == "sigmoid"
    x = st["logits"].double()
    s = torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)
    # the choice is made by 32-bit keys: equal ones go to the lowest index
    key = (s.float() + st["bias"]) if sigmoid else st["logits"].float()
    lowest_first = torch.arange(E, device="cuda")
    if c["top_groups"] < G:
        per = key.view(T, G, -1)
        score = per.topk(2, dim=2).values.sum(2) if sigmoid else per.amax(2)
        place = ((score.unsqueeze(1) > score.unsqueeze(2)) | ((score.unsqueeze(1) == score.unsqueeze(2)) & (
            torch.arange(G, device="cuda").view(1, 1, G) < torch.arange(G, device="cuda").view(1, G, 1)))).sum(2)
        key = torch.where((place < c["top_groups"]).repeat_interleave(E // G, 1), key, -torch.inf)
    left = key.clone()
    cols = []
    for _ in range(K):
        best = left.amax(1, keepdim=True)
        at = torch.where(left == best, lowest_first, E).amin(1, keepdim=True)
        cols.append(at)
        left.scatter_(1, at, -torch.inf)
    at = torch.cat(cols, 1)
    live = st["mask"].unsqueeze(1)
    sel = s.gather(1, at) * live
    weights = 2.5 * sel / (sel.sum(1, keepdim=True) + EPS)
    if c["op"] == "gate":
        return {"ids": None, "weights": weights}
    share = s / s.sum(1, keepdim=True)
    S = c["S"]
    seg = st["seg"].tolist()
    chosen = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, at, 1.0) * live
    loss = torch.zeros((S,), dtype=torch.float64, device="cuda")
    prob = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    d_share = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    for i in range(S):
        lo, hi = seg[i], seg[i + 1]
        n = int(st["mask"][lo:hi].sum())
        if n == 0:
            continue
        prob[i] = (share[lo:hi] * live[lo:hi]).sum(0) / n
        f = chosen[lo:hi].sum(0) * E / (K * n)
        loss[i] = st["alpha"] * (f * prob[i]).sum()
        d_share[lo:hi] = st["alpha"] * st["d_loss"][i].double() * f / n
    # d weights / d score: 2.5 (delta / D - s / D^2) over the chosen
    D = sel.sum(1, keepdim=True) + EPS
    gw = st["d_weights"].double() * live
    d_s = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    d_s.scatter_(1, at, 2.5 * (gw / D - (gw * sel).sum(1, keepdim=True) / D ** 2))
    if sigmoid:
        d_s += (d_share - (d_share * share).sum(1, keepdim=True)) / s.sum(1, keepdim=True)
        dx = d_s * s * (1 - s)
    else:
        d_s += d_share
        dx = s * (d_s - (d_s * s).sum(1, keepdim=True))
    return {"ids": None, "weights": weights, "loss": loss, "counts": None, "prob": prob, "tokens": None,
            "d_logits": dx * live}
