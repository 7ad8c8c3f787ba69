"""The router, its balance loss and the gradients, and the grouping of rows by
slot: HIP path against plain implementations in 64 bits (needs an MI355X).

Tolerances.  A score is a few correctly rounded 32-bit operations and one
exponential of an argument that is itself rounded to 2^-24 of its magnitude
(below 40 here): 40 * 2^-24 + 4 * 2^-24 < 3e-6 relative; sums of positive terms
add at most 200 * 2^-24 = 1.2e-5.  Weights and probabilities are held to 2e-5,
losses to 4e-5.  A gradient is a difference of such terms: 4e-5 of the largest
term of its row, plus the rounding of its type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def note(*a):
    print("[router]", *a, flush=True)


# ------------------------------------------------------------------ plain forms (numpy, 64 bits)
def scores(x, scoring):
    with np.errstate(all="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = x.max(1, keepdims=True)
        m = np.where(m == -np.inf, 0.0, m)
        e = np.exp(x - m)
        return e / (e.sum(1, keepdims=True) + 1e-20)


def choose(key, K, G, top_groups, group_top):
    """ids [T, K] by the rule, row by row, from keys as given."""
    T, E = key.shape
    ids = np.full((T, K), -1, dtype=np.int32)
    for t in range(T):
        k = np.where(np.isnan(key[t]), -np.inf, key[t]).copy()
        if top_groups < G:
            per = k.reshape(G, E // G)
            with np.errstate(invalid="ignore"):
                sc = np.sort(per, axis=1)[:, ::-1][:, :group_top].sum(1)
            sc = np.where(np.isnan(sc), -np.inf, sc)
            keep = np.argsort(-sc, kind="stable")[:top_groups]
            drop = np.setdiff1d(np.arange(G), keep)
            per[drop] = -np.inf
            k = per.reshape(E)
        order = np.argsort(-k, kind="stable")[:K]
        ok = k[order] > -np.inf
        ids[t, :ok.sum()] = order[ok]
    return ids


def weights_of(s, ids, normalize, scale):
    sel = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    return scale * sel / (sel.sum(1, keepdims=True) + 1e-20) if normalize else scale * sel


def loss_of(s, scoring, ids, seg, mask, alpha, E):
    S, K = len(seg) - 1, ids.shape[1]
    share = s / (s.sum(1, keepdims=True) + 1e-20) if scoring == "sigmoid" else s
    loss, prob = np.zeros(S), np.zeros((S, E))
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    for i in range(S):
        rows = np.arange(seg[i], seg[i + 1])
        rows = rows[mask[rows]]
        tokens[i] = len(rows)
        if len(rows) == 0:
            continue
        got = ids[rows].ravel()
        counts[i] = np.bincount(got[(got >= 0) & (got < E)], minlength=E)
        prob[i] = share[rows].mean(0)
        loss[i] = alpha * (E * counts[i] / (K * len(rows)) * prob[i]).sum()
    return loss, counts, prob, tokens


def objective(x, scoring, ids, mask, normalize, scale, gw, seg, alpha, gl, counts, tokens):
    """sum(d_weights * weights) + sum(d_loss * loss), the choice and counts held fixed."""
    s = scores(x, scoring)
    E, K = x.shape[1], ids.shape[1]
    live = np.where(mask[:, None], ids, -1)
    live = np.where((live >= 0) & (live < E), live, -1)
    total = (gw * weights_of(s, live, normalize, scale) * (live >= 0)).sum() if gw is not None else 0.0
    if gl is not None:
        share = s / (s.sum(1, keepdims=True) + 1e-20) if scoring == "sigmoid" else s
        for i in range(len(seg) - 1):
            rows = np.arange(seg[i], seg[i + 1])
            rows = rows[mask[rows]]
            if len(rows):
                total += gl[i] * alpha * (E * counts[i] / (K * len(rows)) * share[rows].mean(0)).sum()
    return total


def gradient(x, scoring, ids, mask, normalize, scale, gw, seg, alpha, gl, counts, tokens):
    """The formula; also the magnitude of the largest term of each row."""
    T, E = x.shape
    K = ids.shape[1]
    s = scores(x, scoring)
    g, big = np.zeros((T, E)), np.zeros((T, 1))
    if gw is not None:
        for t in range(T):
            if not mask[t]:
                continue
            ok = [k for k in range(K) if 0 <= ids[t, k] < E]
            sel = s[t, ids[t, ok]]
            gk = scale * gw[t, ok]
            if normalize:
                D = sel.sum() + 1e-20
                big[t] = max(big[t], np.abs(gk).max(initial=0.0) / D)
                gk = (gk - (gk * sel).sum() / D) / D
            else:
                big[t] = max(big[t], np.abs(gk).max(initial=0.0))
            np.add.at(g[t], ids[t, ok], gk)
    if gl is not None:
        Z = s.sum(1, keepdims=True) + 1e-20
        for i in range(len(seg) - 1):
            if tokens[i] == 0:
                continue
            rows = np.arange(seg[i], seg[i + 1])
            rows = rows[mask[rows]]
            a = alpha * gl[i] * E * counts[i] / (K * tokens[i] ** 2)
            if scoring == "sigmoid":
                share = s[rows] / Z[rows]
                g[rows] += (a - (a * share).sum(1, keepdims=True)) / Z[rows]
                big[rows] = np.maximum(big[rows], np.abs(a).max() / Z[rows])
            else:
                g[rows] += a
                big[rows] = np.maximum(big[rows], np.abs(a).max())
    if scoring == "sigmoid":
        dx = g * s * (1 - s)
    else:
        dx = s * (g - (g * s).sum(1, keepdims=True))
    return np.where(mask[:, None], dx, 0.0), big


def make(T, E, dtype, seed, ties=False):
    rng = np.random.default_rng(seed)
    x = rng.integers(-6, 7, size=(T, E)) * 0.5 if ties else rng.normal(size=(T, E)) * 2
    x = torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])
    return x, x.double().numpy(), rng


# ------------------------------------------------------------------ the choice
@pytest.mark.parametrize("T,E,K,G,top,gtop,dtype,seed", [
    (1, 1, 1, 1, 1, 1, "f32", 0), (3, 2, 2, 1, 1, 1, "bf16", 1), (70, 7, 3, 1, 1, 1, "f16", 2),
    (129, 60, 6, 1, 1, 1, "bf16", 3), (64, 64, 8, 8, 4, 2, "f32", 4), (65, 65, 64, 1, 1, 1, "f32", 5),
    (33, 256, 8, 8, 4, 2, "bf16", 6), (40, 256, 8, 8, 3, 1, "f32", 7), (17, 160, 6, 8, 3, 1, "f16", 8),
    (21, 192, 16, 64, 9, 2, "f32", 9), (16, 100, 10, 50, 7, 1, "bf16", 10), (9, 1000, 33, 4, 2, 2, "f32", 11),
    (5, 4096, 64, 32, 8, 2, "bf16", 12), (4, 2049, 20, 1, 1, 1, "f16", 13), (300, 12, 4, 4, 2, 2, "bf16", 14),
    (50, 384, 12, 16, 5, 2, "f32", 15), (50, 512, 8, 2, 1, 2, "bf16", 16), (11, 320, 17, 10, 10, 1, "f32", 17),
    (260, 288, 9, 9, 2, 2, "f16", 18), (31, 33, 5, 11, 4, 2, "f32", 19)])
def test_choice_with_ties(T, E, K, G, top, gtop, dtype, seed):
    """Keys on a coarse grid: equal ones abound and every sum is exact, so the
    ids have to be the rule's."""
    x, x64, rng = make(T, E, dtype, seed, ties=True)
    bias = rng.integers(-4, 5, size=E).astype(np.float32) * 0.25
    mask = rng.random(T) > 0.2
    x64[rng.random((T, E)) < 0.05] = -np.inf
    x64[0] = -np.inf                                    # a row with nothing to choose
    if T > 2:
        x64[1] = float(torch.finfo(TYPES[dtype]).min)   # the type's lowest value is a value like others
        x64[2, E // 2:] = np.nan
    x = torch.from_numpy(x64).to(TYPES[dtype])
    note("choice", T, E, K, G, top, gtop, dtype)
    ids, w = eplb.gate(x.to(DEV), K, scoring="softmax", bias=torch.from_numpy(bias).to(DEV), G=G, top_groups=top,
                       group_top=gtop, scale=1.5, mask=torch.from_numpy(mask).to(DEV))
    key = (x.float().numpy() + bias).astype(np.float32)
    want = choose(key, K, G, top, gtop)
    want[~mask] = -1
    assert np.array_equal(ids.cpu().numpy(), want)
    ref = weights_of(scores(x.double().numpy(), "softmax"), want, True, 1.5)
    fine = ~np.isnan(x64).any(1)
    np.testing.assert_allclose(w.cpu().numpy()[fine], ref[fine], rtol=2e-5, atol=1e-30)
    assert (w.cpu().numpy()[~mask] == 0).all()


@pytest.mark.parametrize("T,E,K,G,top,dtype,normalize", [
    (200, 256, 8, 8, 4, "bf16", True), (200, 256, 8, 8, 4, "f32", False), (77, 61, 4, 1, 1, "f16", True),
    (513, 128, 6, 4, 2, "f32", True), (30, 1024, 24, 16, 4, "bf16", True)])
def test_sigmoid_choice(T, E, K, G, top, dtype, normalize):
    """Random keys: the chosen ones are the largest up to the keys' rounding."""
    x, x64, rng = make(T, E, dtype, T + E)
    bias = (rng.normal(size=E) * 0.05).astype(np.float32)
    s = scores(x64, "sigmoid")
    key = s + bias
    note("sigmoid", T, E, K, G, top, dtype)
    ids, w = (t.cpu().numpy() for t in eplb.gate(x.to(DEV), K, bias=torch.from_numpy(bias).to(DEV), G=G,
                                                 top_groups=top, group_top=2, normalize=normalize, scale=2.5))
    want = choose(key, K, G, top, 2)
    same = (ids == want).all(1)
    assert same.mean() > 0.95
    for t in np.flatnonzero(~same):                     # near ties only
        assert len(set(ids[t])) == K
        assert np.abs(np.sort(key[t, ids[t]]) - np.sort(key[t, want[t]])).max() < 1e-6
    np.testing.assert_allclose(w, weights_of(s, ids, normalize, 2.5), rtol=2e-5)


def test_infinite_and_strided_logits():
    x = torch.full((4, 600), 7.0)
    x[:, 40:140] = torch.linspace(-3, 3, 100)
    x[0, 50] = float("inf")
    x[1, 60] = float("nan")
    x[2, 40:140] = -float("inf")
    x[2, 70] = 2.0
    view = x.to(DEV)[:, 40:140]
    assert not view.is_contiguous()
    ids, w = (t.cpu().numpy() for t in eplb.gate(view, 3, scoring="sigmoid"))
    assert ids[0].tolist() == [10, 99, 98] and w[0, 0] > w[0, 1]
    assert ids[1].tolist() == [99, 98, 97] and np.isfinite(w[1]).all()
    assert ids[2].tolist() == [30, -1, -1] and w[2, 0] == 1.0 and (w[2, 1:] == 0).all()
    ids, w = (t.cpu().numpy() for t in eplb.gate(view, 2, scoring="softmax"))
    assert ids[0].tolist() == [10, 99] and np.isnan(w[0, 0])
    assert ids[3].tolist() == [99, 98]
    odd = x.to(DEV).bfloat16()[:, 41:140]               # rows that start at odd addresses
    ids = eplb.gate(odd, 2)[0].cpu().numpy()
    assert ids[3].tolist() == [98, 97]


# ------------------------------------------------------------------ the loss and the gradients
LOSS_CASES = [
    (1, 3, 2, 1, "sigmoid", "f32", [0, 1]), (5, 8, 2, 3, "softmax", "f32", [0, 0, 3, 5]),
    (200, 60, 6, 5, "softmax", "bf16", [0, 64, 64, 65, 190, 200]), (333, 256, 8, 4, "sigmoid", "f32", [0, 100, 101, 300, 333]),
    (150, 256, 8, 2, "sigmoid", "bf16", [3, 80, 140]), (64, 130, 3, 1, "softmax", "f16", [0, 64]),
    (1000, 17, 4, 3, "sigmoid", "f16", [0, 1, 999, 1000]), (70, 520, 9, 2, "softmax", "f32", [0, 63, 70]),
    (40, 1500, 5, 2, "sigmoid", "f32", [0, 39, 40]), (12, 4096, 8, 2, "softmax", "bf16", [0, 5, 12])]


@pytest.mark.parametrize("T,E,K,S,scoring,dtype,seg", LOSS_CASES)
@pytest.mark.parametrize("given", [False, True])
def test_loss_and_gradient(T, E, K, S, scoring, dtype, seg, given):
    x, x64, rng = make(T, E, dtype, T * 7 + E)
    S = len(seg) - 1
    mask = rng.random(T) > 0.15
    if S > 1:
        mask[seg[-2]:seg[-1]] = T > 100 and mask[seg[-2]:seg[-1]]   # a segment whose mask leaves nothing (small cases)
    seg_d = torch.tensor(seg, dtype=torch.int32, device=DEV)
    xd, md = x.to(DEV), torch.from_numpy(mask).to(DEV)
    note("loss", T, E, K, scoring, dtype, seg, given)
    how = dict(scoring=scoring, mask=md)
    if given:
        ids = rng.integers(-1, E + 1, size=(T, K)).astype(np.int32)      # repeats and ids of no expert among them
        loss, counts, prob, tokens = (t.cpu().numpy() for t in eplb.balance_loss(
            xd, torch.from_numpy(ids).to(DEV), seg_d, 0.3, **how))
    else:
        ids, w, loss, counts, prob, tokens = (t.cpu().numpy() for t in eplb.gate_loss(xd, K, seg_d, 0.3, scale=2.5, **how))
        plain = eplb.gate(xd, K, scale=2.5, **how)
        assert np.array_equal(ids, plain[0].cpu().numpy()) and np.array_equal(w, plain[1].cpu().numpy())
    s = scores(x64, scoring)
    rl, rc, rp, rt = loss_of(s, scoring, np.where(mask[:, None], ids, -1), seg, mask, 0.3, E)
    assert np.array_equal(counts, rc) and np.array_equal(tokens, rt)
    np.testing.assert_allclose(prob, rp, rtol=2e-5, atol=1e-30)
    np.testing.assert_allclose(loss, rl, rtol=4e-5)
    # gradients: both terms, and each alone
    gw = rng.normal(size=(T, K)).astype(np.float32)
    gl = rng.normal(size=S).astype(np.float32)
    for normalize, a, b in ((True, gw, gl), (False, gw, None), (True, None, gl)):
        got = eplb.gate_backward(xd, torch.from_numpy(ids).to(DEV), None if a is None else torch.from_numpy(a).to(DEV),
                                 normalize=normalize, scale=2.5, seg=seg_d, alpha=0.3,
                                 counts=torch.from_numpy(counts).to(DEV), tokens=torch.from_numpy(tokens).to(DEV),
                                 d_loss=None if b is None else torch.from_numpy(b).to(DEV), **how)
        assert got.dtype == TYPES[dtype]
        args = (scoring, ids, mask, normalize, 2.5, a, seg, 0.3, b, rc, rt)
        ref, big = gradient(x64, *args)
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= 4e-5 * big + HALF_ULP[dtype] * np.abs(ref) + 2.0 ** -25).all(), err.max()
        # differences of the 64-bit objective along random directions
        for _ in range(2):
            d = rng.normal(size=(T, E))
            h = 1e-5
            slope = (objective(x64 + h * d, *args) - objective(x64 - h * d, *args)) / (2 * h)
            dot = (got.double().cpu().numpy() * d).sum()
            room = np.sqrt((((4e-5 * big + HALF_ULP[dtype] * np.abs(ref) + 2.0 ** -25) * d) ** 2).sum()) * 6
            assert abs(dot - slope) <= room + 1e-7 * (1 + abs(slope)), (dot, slope, room)


def test_loss_is_deterministic_and_large():
    """Equal bits from call to call, over enough rows for many partial sums."""
    T, E, K = 40000, 256, 8
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((T, E), generator=g, device=DEV)
    seg = torch.tensor([0, 1, 30000, 30000, T], dtype=torch.int32, device=DEV)
    first = eplb.gate_loss(x, K, seg, 0.1)
    for _ in range(3):
        again = eplb.gate_loss(x, K, seg, 0.1)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    ids, w, loss, counts, prob, tokens = first
    assert tokens.tolist() == [1, 29999, 0, 10000]
    assert counts.sum(1).tolist() == [8 * n for n in tokens.tolist()]
    s = torch.sigmoid(x.double())
    share = s / s.sum(1, keepdim=True)
    torch.testing.assert_close(prob[1].double(), share[1:30000].mean(0), rtol=2e-5, atol=0)
    assert (prob[2] == 0).all() and loss[2] == 0


def test_router_no_rows():
    x = torch.zeros((0, 16), device=DEV)
    seg = torch.zeros((3,), dtype=torch.int32, device=DEV)
    ids, w, loss, counts, prob, tokens = eplb.gate_loss(x, 4, seg, 0.1)
    assert ids.shape == (0, 4) and loss.tolist() == [0, 0] and not counts.any() and not tokens.any() and not prob.any()
    assert eplb.gate_backward(x, ids, w).shape == (0, 16)


# ------------------------------------------------------------------ grouping
def check_group(ids, first, P):
    """ids [L, n] on the host."""
    L, n = ids.shape
    off, order, place = (t.cpu().numpy() for t in eplb.group_rows(torch.from_numpy(ids).to(DEV), P, first=first))
    slot = ids.astype(np.int64) - first
    slot = np.where((slot >= 0) & (slot < P), slot, P)
    for l in range(L):
        want = np.argsort(slot[l], kind="stable")
        assert np.array_equal(order[l], want)
        assert np.array_equal(off[l], np.concatenate([[0], np.cumsum(np.bincount(slot[l], minlength=P + 1)[:P])]))
        inv = np.empty(n, np.int64)
        inv[want] = np.arange(n)
        assert np.array_equal(place[l], inv)


@pytest.mark.parametrize("L,n,P,first", [
    (1, 0, 5, 0), (3, 1, 1, 0), (2, 64, 7, 0), (1, 63, 320, 0), (4, 512, 288, 0), (1, 2048, 9, 27), (1, 2049, 9, -3),
    (2, 5000, 1, 0), (1, 16384, 288, 0), (3, 4097, 512, 100), (1, 20000, 4096, 0), (2, 9000, 8192, 0),
    (1, 131072, 288, 0), (1, 700001, 64, 5), (58, 1000, 288, 0), (1, 3000, 4095, 0)])
def test_group_rows(L, n, P, first):
    rng = np.random.default_rng(n + P)
    note("group", L, n, P, first)
    ids = (first + rng.integers(-2, P + 2, size=(L, n))).astype(np.int32)
    if n > 10:
        ids[0, 5], ids[0, 7] = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    check_group(ids, first, P)
    check_group(np.full((L, n), first, np.int32), first, P)          # all in one slot
    check_group(np.sort(ids, axis=1), first, P)


def test_group_rows_workspace_and_shapes():
    ids = torch.randint(0, 40, (2, 1500, 4), dtype=torch.int32, device=DEV)
    need = eplb.group_rows_workspace_bytes(2, 6000, 40)
    a = eplb.group_rows(ids, 40, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    b = eplb.group_rows(ids.view(2, 6000), 40)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(eplb.EplbError):
        eplb.group_rows(ids, 40, workspace=torch.empty((need - 4,), dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ many rows: four to a wave
@pytest.mark.parametrize("E,K,G,top,gtop,dtype", [
    (16, 4, 1, 1, 1, "f32"), (60, 6, 1, 1, 1, "bf16"), (64, 16, 8, 4, 2, "f16"), (120, 8, 4, 2, 2, "bf16"),
    (256, 8, 8, 4, 2, "f32"), (250, 7, 10, 3, 1, "bf16"), (512, 16, 16, 5, 2, "bf16"), (300, 9, 1, 1, 1, "f32"),
    (256, 17, 8, 4, 2, "f32")])
def test_choice_many_rows(E, K, G, top, gtop, dtype):
    T = 2048 + 37
    x, x64, rng = make(T, E, dtype, E * K, ties=True)
    x64[rng.random((T, E)) < 0.05] = -np.inf
    x64[5] = -np.inf
    x64[7] = 1.0                                        # all keys equal but for the bias
    x64[9, : E // 2] = np.nan
    bias = rng.integers(-4, 5, size=E).astype(np.float32) * 0.25
    if E == 300:
        bias[:] = 0
    mask = rng.random(T) > 0.1
    x = torch.from_numpy(x64).to(TYPES[dtype])
    note("many", E, K, G, top, gtop, dtype)
    ids, w = eplb.gate(x.to(DEV), K, scoring="softmax", bias=torch.from_numpy(bias).to(DEV), G=G, top_groups=top,
                       group_top=gtop, mask=torch.from_numpy(mask).to(DEV))
    want = choose((x.float().numpy() + bias).astype(np.float32), K, G, top, gtop)
    want[~mask] = -1
    assert np.array_equal(ids.cpu().numpy(), want)
    fine = ~np.isnan(x64).any(1)
    ref = weights_of(scores(x.double().numpy(), "softmax"), want, True, 1.0)
    np.testing.assert_allclose(w.cpu().numpy()[fine], ref[fine], rtol=2e-5, atol=1e-30)


def test_equal_logits():
    """A router that has learned nothing: the lowest experts, by rows of 64 lanes and of 16."""
    for T in (3, 2100):
        ids, w = eplb.gate(torch.zeros((T, 256), device=DEV), 8, G=8, top_groups=4, group_top=2)
        assert (ids.cpu().numpy() == np.arange(8)).all() and (w == 0.125).all()


@pytest.mark.parametrize("scoring,dtype", [("sigmoid", "f32"), ("softmax", "bf16")])
def test_loss_and_gradient_many_rows(scoring, dtype):
    T, E, K = 2500, 72, 5
    x, x64, rng = make(T, E, dtype, 3)
    seg = [0, 700, 700, 2100, 2490]
    mask = rng.random(T) > 0.1
    ids_d, w, loss, counts, prob, tokens = eplb.gate_loss(
        x.to(DEV), K, torch.tensor(seg, dtype=torch.int32, device=DEV), 0.2, scoring=scoring,
        mask=torch.from_numpy(mask).to(DEV))
    ids = ids_d.cpu().numpy()
    rl, rc, rp, rt = loss_of(scores(x64, scoring), scoring, ids, seg, mask, 0.2, E)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    np.testing.assert_allclose(prob.cpu().numpy(), rp, rtol=2e-5, atol=1e-30)
    np.testing.assert_allclose(loss.cpu().numpy(), rl, rtol=4e-5)
    ids[11] = ids[11, 0]                                # one expert named K times
    gw, gl = rng.normal(size=(T, K)).astype(np.float32), rng.normal(size=4).astype(np.float32)
    got = eplb.gate_backward(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(gw).to(DEV), scoring=scoring,
                             mask=torch.from_numpy(mask).to(DEV), seg=torch.tensor(seg, dtype=torch.int32, device=DEV),
                             alpha=0.2, counts=counts, tokens=tokens, d_loss=torch.from_numpy(gl).to(DEV))
    ref, big = gradient(x64, scoring, ids, mask, True, 1.0, gw, seg, 0.2, gl, rc, rt)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= 4e-5 * big + HALF_ULP[dtype] * np.abs(ref) + 2.0 ** -25).all(), err.max()


@pytest.mark.parametrize("E,K,G,top,gtop,dtype", [
    (120, 8, 4, 2, 2, "bf16"), (128, 16, 1, 1, 1, "f32"), (250, 7, 10, 3, 1, "bf16"), (256, 8, 8, 4, 2, "f32"),
    (256, 16, 1, 1, 1, "f16")])
def test_rows_of_a_long_call_are_those_of_short_ones(E, K, G, top, gtop, dtype):
    """Rows by 16 lanes against rows by 64: the same choices, and weights and
    gradients within the rounding of E 32-bit operations in another order."""
    T, step = 32 * E + 37, 1000
    x, x64, rng = make(T, E, dtype, E + K, ties=True)
    x64[rng.random((T, E)) < 0.05] = -np.inf
    x64[5] = -np.inf
    x64[7] = 1.0
    x = torch.from_numpy(x64).to(TYPES[dtype]).to(DEV)
    bias = torch.from_numpy(rng.integers(-4, 5, size=E).astype(np.float32) * 0.25).to(DEV)
    note("long", E, K, G, top, gtop, dtype)
    gw = torch.from_numpy(rng.normal(size=(T, K)).astype(np.float32)).to(DEV)
    for scoring in ("sigmoid", "softmax"):
        kw = dict(scoring=scoring, bias=bias, G=G, top_groups=top, group_top=gtop)
        ids, w = eplb.gate(x, K, **kw)
        d = eplb.gate_backward(x, ids, gw, scoring=scoring)
        for t in range(0, T, step):
            a, b = eplb.gate(x[t:t + step], K, **kw)
            assert torch.equal(a, ids[t:t + step])
            torch.testing.assert_close(b, w[t:t + step], rtol=2e-5, atol=1e-30, equal_nan=True)
            e = eplb.gate_backward(x[t:t + step], a, gw[t:t + step].contiguous(), scoring=scoring)
            room = 4e-5 * (gw[t:t + step].abs().sum(1, keepdim=True) + 1) + 2 * HALF_ULP[dtype] * e.float().abs()
            assert ((e.float() - d[t:t + step].float()).abs() <= room)[~e.isnan()].all()
            assert torch.equal(e.isnan(), d[t:t + step].isnan())


def test_group_rows_few_layers():
    """Segments shorter than a long layer's."""
    rng = np.random.default_rng(1)
    for L, n, P in ((1, 2050, 30), (16, 4000, 8), (3, 32768, 288), (17, 2500, 40), (2, 32769, 5), (1, 8192, 8192)):
        check_group(rng.integers(-1, P + 1, size=(L, n)).astype(np.int32), 0, P)
