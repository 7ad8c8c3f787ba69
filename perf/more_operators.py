"""Cases that measure the experts' products in 16 bits and with 4-bit weights, and the joining of their rows.

Each case runs one pass of an operator in one of two ways: through the
package's entry points (``own`` true), or as elementary torch operations in 32
bits (``own`` false), the definition the kernels are compared with.  ``exact``
gives the same outputs computed in 64 bits, written apart from both.

Operators:
  linear   tokens x expert weights, both in 16 bits, rows grouped by expert
  step     one training step of that product: the product, the gradient of the
           tokens (the sum over their rows) and the gradient of the weights
  w4       tokens in 16 bits x expert weights of 4-bit floating point (1 sign, 2
           exponent, 1 mantissa bit) with a power of two for each 32; with
           ``place`` the weights are taken to 4 bits in the same pass, as after
           a new placement
  combine  the experts' rows joined to tokens by the router's weights
  combine_step  the same with the gradients of the rows and of the weights
"""
from __future__ import annotations

import torch

own = False

GROUP = 32                   # elements that a scale of the 4-bit format covers
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded token through its 8 experts of 32 on this GPU: the experts' 16-bit weights are what is read
        {"name": "linear_one_token", "op": "linear", "T": 1, "K": 8, "G": 32, "H": 2048, "N": 4096, "dtype": "bf16"},
        # a decode step's rows on one rank of 9 slots (288 slots on 32 ranks)
        {"name": "linear_decode", "op": "linear", "T": 256, "K": 2, "G": 9, "H": 4096, "N": 2048, "dtype": "f16"},
        # a prefill step's rows on one rank of 9 slots: the matrix cores are what counts
        {"name": "linear_prefill", "op": "linear", "T": 8192, "K": 2, "G": 9, "H": 4096, "N": 4096, "dtype": "bf16"},
        # a fine-tuning micro-batch over 5 experts, sizes that fill no tile
        {"name": "step_odd", "op": "step", "T": 301, "K": 2, "G": 5, "H": 1048, "N": 712, "dtype": "f16"},
        # a training micro-batch on one rank of 9 slots
        {"name": "step_train", "op": "step", "T": 8192, "K": 2, "G": 9, "H": 4096, "N": 2048, "dtype": "bf16"},
        # the decoded token of the first case with 4-bit weights
        {"name": "w4_one_token", "op": "w4", "T": 1, "K": 8, "G": 32, "H": 2048, "N": 4096, "dtype": "bf16",
         "place": False},
        # a small decode batch on one rank of 9 slots, 4-bit weights
        {"name": "w4_decode", "op": "w4", "T": 64, "K": 2, "G": 9, "H": 4096, "N": 4096, "dtype": "bf16", "place": False},
        # a prefill step through the same weights
        {"name": "w4_prefill", "op": "w4", "T": 4096, "K": 2, "G": 9, "H": 4096, "N": 2048, "dtype": "bf16",
         "place": False},
        # a new placement of small experts, at sizes that fill no tile: weights to 4 bits, then the first batch
        {"name": "w4_place_odd", "op": "w4", "T": 100, "K": 2, "G": 6, "H": 1056, "N": 1391, "dtype": "f16",
         "place": True},
        # a decode batch's rows joined: launch latency counts
        {"name": "combine_decode", "op": "combine", "T": 64, "K": 8, "H": 4096, "dtype": "bf16"},
        # a prefill step of the 58-layer deployment: 16384 tokens of 8 rows each
        {"name": "combine_prefill", "op": "combine", "T": 16384, "K": 8, "H": 2048, "dtype": "bf16"},
        # a training micro-batch, an odd width, both gradients
        {"name": "combine_train", "op": "combine_step", "T": 4097, "K": 6, "H": 2050, "dtype": "f16"},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["linear", "linear", "step", "w4", "w4", "combine", "combine_step"])
    if op in ("combine", "combine_step"):
        K = rng.randint(1, 8)
        H = log(16, 8192)
        T = log(1, 16384)
        most = 16384 * 8 * 2048 if op == "combine" else 4097 * 6 * 2050
        while T * K * H > most:
            T = T // 2 + 1
        return {"op": op, "T": T, "K": K, "H": H, "dtype": rng.choice(["f32", "bf16", "f16"])}
    G = rng.randint(1, 16)
    K = rng.randint(1, min(4, G))
    dtype = rng.choice(["bf16", "f16"])
    T = log(1, 8192)
    if op == "w4":
        H, N = 32 * log(4, 128), log(64, 4096)
        most = 4096 * 2 * 4096 * 2048
    else:
        H, N = 8 * log(16, 512), (8 * log(16, 512) if op == "step" else log(64, 4096))
        most = 8192 * 2 * 4096 * (2048 if op == "step" else 4096)
    while T * K * H * N > most:
        T = T // 2 + 1
    case = {"op": op, "T": T, "K": K, "G": G, "H": H, "N": N, "dtype": dtype}
    if op == "w4":
        case["place"] = T <= 512 and rng.random() < 0.4
    return case


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
    away = torch.rand((T, K), generator=g, device="cuda") < (0.02 if T > 1 else 0.0)
    return torch.where(away, torch.full_like(ids, -1), ids)


def _grouped(ids, P):
    """offsets [P + 1], order [n], place [n] of ids [T, K]; ids outside [0, P) come last."""
    key = torch.where((ids >= 0) & (ids < P), ids, torch.full_like(ids, P)).view(-1).long()
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    offsets = torch.zeros((P + 1,), dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.bincount(key, minlength=P + 1)[:P].cumsum(0)
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, T, K, H = case["op"], case["T"], case["K"], case["H"]
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if op in ("combine", "combine_step"):
        P = 32
        ids = _slot_ids(g, T, K, P)
        offsets, st["order"], st["place"] = _grouped(ids, P)
        y = _randn(g, T * K, H)
        y[int(offsets[P]):] = 0.0                    # rows of choices served elsewhere: zeros, as a product leaves them
        st["y"] = y.to(dt)
        score = torch.rand((T, K), generator=g, device="cuda") + 0.05
        st["weights"] = 2.5 * score / score.sum(1, keepdim=True)
        if op == "combine_step":
            st["d_out"] = (1e-2 * _randn(g, T, H)).to(dt)
        return st
    G, N = case["G"], case["N"]
    # activations: unit normal with a few channels an order of magnitude larger
    channel = torch.where(torch.rand((H,), generator=g, device="cuda") < 0.01, 12.0, 1.0)
    st["x"] = (_randn(g, T, H) * channel).to(dt)
    w = (_randn(g, G, N, H) * H ** -0.5).to(dt)
    st["offsets"], st["order"], st["place"] = _grouped(_slot_ids(g, T, K, G), G)
    st["cap"] = max(1, int((st["offsets"][1:] - st["offsets"][:-1]).max()))   # rows of the fullest expert
    if op == "w4" and not case["place"]:
        st["q"], st["s"] = _quantize4(w)
    else:
        st["w"] = w
    if op == "step":
        st["dy"] = (1e-2 * _randn(g, T * K, N)).to(dt)
    return st


# ------------------------------------------------------------------ plain forms
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
    out[G * cap] = 0.0
    return out[:G * cap].view(G, cap, v.shape[1])


def _unpad(v, at):
    flat = torch.cat([v.reshape(-1, v.shape[2]), torch.zeros((1, v.shape[2]), device=v.device)])
    return flat[at]


def _linear_plain(st, w):
    """Rows of x in grouped order times the transposed 32-bit weights of their expert."""
    c = st["case"]
    at = _layout(st, c["T"] * c["K"])
    x = st["x"].float()[st["order"].long() // c["K"]]
    return _unpad(torch.bmm(_pad(x, at, c["G"], st["cap"]), w.transpose(1, 2).contiguous()), at).to(st["x"].dtype)


def _step_plain(st):
    c = st["case"]
    T, K, G, cap = c["T"], c["K"], c["G"], st["cap"]
    dt = st["x"].dtype
    at = _layout(st, T * K)
    w = st["w"].float()
    x = _pad(st["x"].float()[st["order"].long() // K], at, G, cap)
    dy = _pad(st["dy"].float(), at, G, cap)
    y = _unpad(torch.bmm(x, w.transpose(1, 2).contiguous()), at)
    dx = _unpad(torch.bmm(dy, w), at)[st["place"].long()].view(T, K, -1).sum(1)
    dw = torch.bmm(dy.transpose(1, 2).contiguous(), x)
    return {"y": y.to(dt), "dx": dx.to(dt), "dw": dw.to(dt)}


def _quantize4(w):
    """w [G, N, H] in 4 bits: codes, two to a byte, the even element in the low half, and a scale byte for each 32 of a
    row.  A scale is 2^e with the least e for which 7 * 2^e reaches the block's largest magnitude, held as e + 127."""
    G, N, H = w.shape
    v = w.float().view(G, N, H // GROUP, GROUP)
    amax = v.abs().amax(3).clamp(min=2.0 ** -98)
    m, k = torch.frexp(amax)                                         # amax = m * 2^k, 0.5 <= m < 1
    e = torch.where(m <= 0.875, k - 3, k - 2).clamp(min=-100)
    u = torch.ldexp(v, -e.unsqueeze(3))
    a = u.abs()
    # the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(u).to(torch.uint8)).view(G, N, H // 2, 2)
    return code[..., 0] + 16 * code[..., 1], (e + 127).to(torch.uint8)


def _dequantize4(q, s):
    G, N, half = q.shape
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    values = torch.cat([values, -values])
    v = values[torch.stack([q & 15, q >> 4], 3).view(G, N, 2 * half).int()]
    scale = torch.ldexp(torch.ones((), device=q.device), s.int() - 127)
    return (v.view(G, N, -1, GROUP) * scale.unsqueeze(3)).view(G, N, 2 * half)


def _combine_plain(st):
    c = st["case"]
    T, K, H = c["T"], c["K"], c["H"]
    w = st["weights"]
    y = st["y"].float()[st["place"].long()].view(T, K, H)
    out = (y * w.unsqueeze(2)).sum(1).to(st["y"].dtype)
    if c["op"] == "combine":
        return out
    d = st["d_out"].float()
    dy = d[st["order"].long() // K] * w.view(-1)[st["order"].long()].unsqueeze(1)
    return {"out": out, "d_y": dy.to(st["y"].dtype), "d_weights": (y * d.unsqueeze(1)).sum(2)}


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    op, K = c["op"], c["K"]
    if own:
        import moe_expert_load_eplb_amd as eplb
        if op == "linear":
            return eplb.expert_matmul16(st["x"], st["w"], st["offsets"], rows=st["order"], K=K)
        if op == "step":
            y = eplb.expert_matmul16(st["x"], st["w"], st["offsets"], rows=st["order"], K=K)
            rows = eplb.expert_matmul16(st["dy"], st["w"], st["offsets"], transpose=True, dtype=torch.float32)
            dx = eplb.combine_rows(rows, st["place"].view(-1, K), None, dtype=st["x"].dtype)
            return {"y": y, "dx": dx,
                    "dw": eplb.expert_wgrad16(st["dy"], st["x"], st["offsets"], rows=st["order"], K=K)}
        if op == "w4":
            q, s = eplb.quantize_weights4(st["w"]) if c["place"] else (st["q"], st["s"])
            return eplb.expert_matmul4(st["x"], q, s, st["offsets"], rows=st["order"], K=K)
        out = eplb.combine_rows(st["y"], st["place"], st["weights"])
        if op == "combine":
            return out
        dy, dw = eplb.combine_rows_backward(st["d_out"], st["y"], st["place"], st["order"], st["weights"])
        return {"out": out, "d_y": dy, "d_weights": dw}
    if op == "linear":
        return _linear_plain(st, st["w"].float())
    if op == "step":
        return _step_plain(st)
    if op == "w4":
        return _linear_plain(st, _dequantize4(*(_quantize4(st["w"]) if c["place"] else (st["q"], st["s"]))))
    return _combine_plain(st)


def work(case):
    """Bytes with each input read once and each output written once, and operations, of one pass."""
    op, T, K, H = (case[k] for k in ("op", "T", "K", "H"))
    size = 4 if case["dtype"] == "f32" else 2
    R = T * K
    if op == "combine":
        return {"bytes": size * H * (R + T) + 8 * R, "flops": 2 * R * H}
    if op == "combine_step":
        return {"bytes": size * H * (2 * R + 2 * T) + 16 * R, "flops": 5 * R * H}
    G, N = case["G"], case["N"]
    used = min(G, R)
    if op == "linear":
        return {"bytes": 2 * (T * H + used * N * H + R * N) + 4 * R, "flops": 2 * R * N * H}
    if op == "step":
        return {"bytes": 2 * (2 * T * H + 2 * R * N + 2 * G * N * H) + 8 * R, "flops": 6 * R * N * H}
    weights = N * H // 2 + N * H // GROUP
    if case["place"]:
        return {"bytes": 2 * (T * H + R * N + G * N * H) + G * weights + 4 * R, "flops": 2 * R * N * H + 4 * G * N * H}
    return {"bytes": 2 * (T * H + R * N) + used * weights + 4 * R, "flops": 2 * R * N * H}


# ------------------------------------------------------------------ the definition in 64 bits
def _four_bits(w):
    """One expert's weights [N, H] as the 4-bit format holds them, in 64 bits."""
    N, H = w.shape
    v = w.double().view(N, H // GROUP, GROUP)
    top = v.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(top / 7.0).clamp(min=-100.0))
    e = torch.where(7.0 * torch.exp2(e - 1.0) >= top, e - 1.0, e)     # log2 may be off at a border
    e = torch.where(7.0 * torch.exp2(e) < top, e + 1.0, e).clamp(min=-100.0)
    u = v / torch.exp2(e)
    a = u.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    return (torch.round(a / step) * step * torch.sign(u) * torch.exp2(e)).view(N, H)


def exact(case, seed):
    st = prepare(case, seed)
    op, T, K, H = (case[k] for k in ("op", "T", "K", "H"))
    R = T * K
    if op in ("combine", "combine_step"):
        y, w, place = st["y"], st["weights"].double(), st["place"].long().view(T, K)
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for k in range(K):
            out += w[:, k:k + 1] * y[place[:, k]].double()
        if op == "combine":
            return out
        d = st["d_out"].double()
        d_y = torch.zeros((R, H), dtype=torch.float64, device="cuda")
        d_w = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for k in range(K):
            d_y[place[:, k]] = w[:, k:k + 1] * d
            d_w[:, k] = (d * y[place[:, k]].double()).sum(1)
        return {"out": out, "d_y": d_y, "d_weights": d_w}
    G, N = case["G"], case["N"]
    off = st["offsets"].tolist()
    token = st["order"].long() // K
    y = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    if op == "step":
        rows = torch.zeros((R, H), dtype=torch.float64, device="cuda")
        dw = torch.zeros((G, N, H), dtype=torch.float64, device="cuda")
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            continue
        x = st["x"][token[lo:hi]].double()
        if op == "w4":
            if case["place"]:
                w = _four_bits(st["w"][g])
            else:
                w = _dequantize4(st["q"][g:g + 1], st["s"][g:g + 1])[0].double()     # exact in 32 bits already
        else:
            w = st["w"][g].double()
        y[lo:hi] = x @ w.t()
        if op == "step":
            dy = st["dy"][lo:hi].double()
            rows[lo:hi] = dy @ w
            dw[g] = dy.t() @ x
    if op != "step":
        return y
    dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    dx.index_add_(0, token, rows)
    return {"y": y, "dx": dx, "dw": dw}
