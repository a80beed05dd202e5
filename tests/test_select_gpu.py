"""The choice of experts in groups and its backward against a plain implementation in 64 bits.

Indices have to be equal throughout, on near ties too: the choice is that of the 64-bit values.
Scores and gates are fp32: with u = 2^-24, expf is within one ulp (2 u relative), so a sigmoid is
off by at most 4 u relative, a sum of the chosen ones by 5 u more, and a gate by 2 * 4 u + 5 u + 2 u
= 15 u; 16 u is the bound. A softmax score's exponent l - max is rounded too: (R + 40) u with R the
range of the row's finite logits bounds the score, its sum over at most 256 terms (13 roundings in
a tree) and their quotient, and twice that the gate."""
import numpy as np
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MODE = {"sigmoid": ops.MODE_SIGMOID, "softmax": ops.MODE_SOFTMAX}
RULE = {"max": ops.GROUP_MAX, "top2": ops.GROUP_TOP2}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _select(l, b, k, mode, G=1, tg=1, rule="top2", renorm=True, scale=1.0, stream=None):
    T, E = l.shape
    o = dict(idx=torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
             gate=torch.full((T, k), 7.0, device="cuda"), score=torch.full((T, k), 7.0, device="cuda"),
             lse=torch.full((T,), 7.0, device="cuda") if mode == "softmax" else None)
    ops.moe_select_experts(l, b, k, MODE[mode], G, tg, RULE[rule], renorm, scale, o["idx"],
                           o["gate"], o["score"], o["lse"], stream=stream)
    return o


def _scores(l, mode):
    """64-bit scores and logsumexp of rows of logits."""
    with np.errstate(all="ignore"):
        if mode == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l)), None
        m = np.fmax.reduce(l, axis=1, keepdims=True)
        e = np.where(m == -np.inf, 0.0 * (l != l), np.exp(l - m))
        S = e.sum(1, keepdims=True)
        p = np.where(S == 0, 0.0, e / np.where(S == 0, 1.0, S))
        return p, np.where(S == 0, -np.inf, m + np.log(S))[:, 0]


def _reference(l, b, k, mode, G, tg, rule, renorm, scale):
    T, E = l.shape
    p, lse = _scores(l, mode)
    v = p if b is None else p + b[None]
    order = l if b is None else v
    v, order = (np.where(np.isnan(a), -np.inf, a) for a in (v, order))
    idx = np.empty((T, k), np.int64)
    per = E // G
    for t in range(T):
        ok = np.ones(E, bool)
        if G > 1:
            gs = []
            for g in range(G):
                if rule == "max":
                    gs.append(order[t, g * per:(g + 1) * per].max())
                else:
                    with np.errstate(invalid="ignore"):
                        s = np.sort(v[t, g * per:(g + 1) * per])[-2:].sum()
                    gs.append(-np.inf if np.isnan(s) else s)
            keep = sorted(range(G), key=lambda g: (-gs[g], g))[:tg]
            ok = np.isin(np.arange(E) // per, keep)
        idx[t] = sorted(np.nonzero(ok)[0], key=lambda e: (-order[t, e], e))[:k]
    s = np.take_along_axis(p, idx, 1)
    S = s.sum(1, keepdims=True)
    gate = scale * (np.where(S == 0, 0.0, s / np.where(S == 0, 1.0, S)) if renorm else s)
    return idx, gate, s, lse


def _check(l, b, k, mode, G=1, tg=1, rule="top2", renorm=True, scale=1.0):
    o = _select(l, b, k, mode, G, tg, rule, renorm, scale)
    torch.cuda.synchronize()
    l64 = l.double().cpu().numpy()
    idx, gate, s, lse = _reference(l64, None if b is None else b.double().cpu().numpy(), k, mode, G,
                                   tg, rule, renorm, scale)
    got = o["idx"].cpu().numpy()
    wrong = np.nonzero((got != idx).any(1))[0]
    assert len(wrong) == 0, f"{len(wrong)} rows differ, e.g. {wrong[0]}: {got[wrong[0]]} for {idx[wrong[0]]}"
    if mode == "softmax":
        fin = np.where(np.isfinite(l64), l64, np.nan)
        with np.errstate(all="ignore"):
            R = np.nan_to_num(np.nanmax(fin, 1, keepdims=True) - np.nanmin(fin, 1, keepdims=True), nan=0.0)
        rel = (np.minimum(R, 200.0) + 40) * U
    else:
        rel = np.full((len(l64), 1), 4 * U)
    tiny = 2.0 ** -126  # below it fp32 has no relative precision
    for name, want, r in (("score", s, rel), ("gate", gate, 2 * rel + 8 * U)):
        g = o[name].double().cpu().numpy()
        assert (np.isnan(g) == np.isnan(want)).all(), name
        ok = ~np.isnan(want)
        floor = tiny * max(1.0, abs(scale)) * (1 if name == "score" else 4)
        assert (np.abs(g - want)[ok] <= (r * np.abs(want) + floor)[ok]).all(), name
    if mode == "softmax":
        g = o["lse"].double().cpu().numpy()
        assert (np.isnan(g) == np.isnan(lse)).all()
        f = np.isfinite(lse)
        assert (g[~f & ~np.isnan(lse)] == lse[~f & ~np.isnan(lse)]).all()
        assert (np.abs(g - lse)[f] <= rel[f, 0] + 4 * U * (np.abs(lse[f]) + 8)).all()
    return o


# T, E, k, n_group, topk_group: powers of two, odd counts, groups of one expert, groups that no
# tile divides, every group kept, the most experts and slots
SHAPES = [(1, 8, 2, 1, 1), (1, 256, 8, 8, 4), (3, 1, 1, 1, 1), (300, 64, 8, 1, 1), (257, 64, 8, 8, 3),
          (129, 256, 8, 8, 4), (100, 256, 32, 4, 2), (65, 128, 6, 4, 2), (33, 160, 6, 8, 3),
          (70, 100, 5, 10, 4), (50, 44, 4, 4, 2), (40, 255, 7, 5, 2), (64, 32, 4, 32, 4),
          (64, 31, 31, 1, 1), (20, 256, 8, 32, 8), (31, 72, 9, 8, 8), (17, 7, 3, 7, 3),
          (128, 96, 8, 2, 1), (61, 36, 4, 4, 1), (45, 16, 16, 2, 2), (19, 200, 32, 20, 20),
          (5000, 64, 8, 4, 2), (2000, 256, 8, 8, 4), (3000, 128, 8, 1, 1)]


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,G,tg", SHAPES)
def test_choice_matches_64_bits(T, E, k, G, tg, bias, mode):
    g = torch.Generator().manual_seed(T * 7 + E + k)
    l = (torch.randn(T, E, generator=g) * 1.5).cuda()
    b = (torch.rand(E, generator=g) * 0.2 - 0.1).cuda() if bias else None
    for rule in ("max", "top2"):
        _check(l, b, k, mode, G, tg, rule, renorm=rule == "top2", scale=2.5 if bias else 1.0)


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,tg", [(400, 64, 8, 8, 4), (200, 256, 8, 8, 4), (300, 24, 4, 1, 1),
                                        (200, 100, 5, 10, 4)])
def test_choice_on_ties_and_near_ties(T, E, k, G, tg, mode):
    """Values that are equal, or differ by less than 32 bits resolve: logits one ulp apart, biases
    that differ by 2^-30, whole rows of equal logits. The lower index wins equal values only."""
    g = torch.Generator().manual_seed(E + k)
    base = torch.randint(0, 4, (T, E), generator=g).float() * 0.25 - 0.5
    l = torch.nextafter(base, base + (torch.randint(0, 3, (T, E), generator=g) - 1).float())
    l[::5] = 0.5
    b = torch.randint(0, 2, (E,), generator=g).float() * 2.0 ** -30
    for bias in (None, b, torch.zeros(E)):
        for rule in ("max", "top2"):
            _check(l.cuda(), None if bias is None else bias.cuda(), k, mode, G, tg, rule)


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_choice_with_masked_and_extreme_logits(mode, bias):
    """Experts masked by -inf or the type's lowest value, rows where nothing is left, saturated
    scores, infinities and NaN: the indices are valid and distinct, and the defined ones exact."""
    T, E, k, G, tg = 96, 64, 6, 8, 3
    g = torch.Generator().manual_seed(11)
    l = torch.randn(T, E, generator=g)
    low = torch.finfo(torch.float32).min
    l[0] = -float("inf")
    l[1, 5:] = -float("inf")                      # fewer experts left than chosen
    l[2] = low
    l[3, ::2] = low
    l[4, torch.randperm(E, generator=g)[:40]] = -float("inf")
    l[5] = 20 + l[5]                              # sigmoids that round to 1 in fp32
    l[6] = -30 + l[6]
    l[7] = 200 * l[7]
    l[8] = -200 - l[8].abs()                      # sigmoids that vanish in fp32
    l[9, 3] = float("inf")
    l[10, 7] = float("nan")
    l[11] = float("nan")
    l[12, 1::2] = float("nan")
    l[13, :8] = float("inf")
    b = (torch.rand(E, generator=g) * 0.1 - 0.05) if bias else None
    if bias:
        b[9], b[10], b[40] = -float("inf"), 3.0, float("nan")
    for rule in ("max", "top2"):
        for GG, tt in ((G, tg), (1, 1)):
            o = _check(l.cuda(), None if b is None else b.cuda(), k, mode, GG, tt, rule)
            i = o["idx"].cpu().numpy()
            assert ((i >= 0) & (i < E)).all() and all(len(set(r)) == k for r in i.tolist())


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,tg", [(64, 8, 8, 4), (256, 8, 8, 4), (100, 5, 10, 4), (160, 12, 16, 5),
                                      (256, 16, 2, 1), (72, 3, 3, 2), (255, 32, 5, 3), (24, 4, 1, 1)])
def test_choice_of_many_tokens(E, k, G, tg, mode):
    """More tokens than are chosen a warp each: ordinary rows, ties and near ties, masks, infinities
    and NaN among them, with biases and without."""
    T = 2600
    g = torch.Generator().manual_seed(E + k + G)
    l = torch.randn(T, E, generator=g)
    base = torch.randint(0, 4, (T // 4, E), generator=g).float() * 0.25 - 0.5
    l[:T // 4] = torch.nextafter(base, base + (torch.randint(0, 3, base.shape, generator=g) - 1).float())
    l[5::50] = 0.0
    l[6::50, ::3] = -float("inf")
    l[7::50] = -float("inf")
    l[8::50] *= 100
    l[9::400, 1] = float("nan")
    l[10::400, 2] = float("inf")
    l[11::50] = torch.finfo(torch.float32).min
    b = (torch.rand(E, generator=g) * 0.2 - 0.1).cuda()
    for bias in (None, b, torch.zeros_like(b)):
        for rule in ("max", "top2"):
            _check(l.cuda(), bias, k, mode, G, tg, rule)


def test_choice_with_large_biases():
    g = torch.Generator().manual_seed(12)
    l = torch.randn(500, 64, generator=g).cuda()
    for size in (1.0, 7.0, 40.0, 1e6):
        b = (torch.randn(64, generator=g) * size).cuda()
        _check(l, b, 8, "sigmoid", 8, 4)
        _check(l, b, 8, "softmax", 8, 4)


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,tg", [(256, 8, 8, 1), (256, 8, 4, 1), (128, 6, 8, 1), (256, 32, 8, 1),
                                      (200, 20, 5, 1), (24, 24, 1, 1), (96, 12, 24, 3), (40, 6, 20, 3),
                                      (256, 16, 1, 1)])
def test_choice_of_many_tokens_from_few_lanes(E, k, G, tg, mode):
    """All of a token's experts in one group (so that few lanes hold them), or all experts chosen,
    with biases so far apart that some values are clamped in the fast keys, expert 0's among them."""
    T = 2600
    g = torch.Generator().manual_seed(E + 3 * k)
    l = torch.randn(T, E, generator=g)
    l[::4] = l[::4] * 1e-6
    l[1::64] = 0.0
    far = torch.randn(E, generator=g) * 12
    far[0] = -50.0
    for bias in (None, torch.rand(E, generator=g) * 0.1, far):
        for rule in ("max", "top2"):
            _check(l.cuda(), None if bias is None else bias.cuda(), k, mode, G, tg, rule)


def test_choice_agrees_with_the_router_without_groups():
    """One group and renormalised sigmoid gates is moe_route's own choice."""
    T, d, E, k = 1000, 256, 64, 8
    g = torch.Generator().manual_seed(13)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn(E, d, generator=g) * d ** -0.5).cuda()
    b = (torch.rand(E, generator=g) * 0.1 - 0.05).cuda()
    ws = torch.empty(ops.moe_workspace_bytes(T, d, E, k), dtype=torch.uint8, device="cuda")
    r = dict(logits=torch.empty(T, E, device="cuda"), idx=torch.empty(T, k, dtype=torch.int32, device="cuda"),
             gate=torch.empty(T, k, device="cuda"), score=torch.empty(T, k, device="cuda"))
    ops.moe_route(x, W, b, k, ops.MODE_SIGMOID, 0.0, r["logits"], r["idx"], r["gate"], r["score"],
                  None, None, ws)
    logits, lse, z = torch.empty(T, E, device="cuda"), torch.empty(T, device="cuda"), torch.zeros(1, device="cuda")
    ops.moe_router_logits(x, W, logits, ws, lse, z, 1e-3)
    torch.cuda.synchronize()
    assert torch.equal(logits, r["logits"])
    l64 = logits.double()
    want = torch.logsumexp(l64, 1)
    R = (l64.amax(1) - l64.amin(1)).max()
    assert ((lse.double() - want).abs() <= (R + 40) * U + 4 * U * (want.abs() + 8)).all()
    assert float(z) == pytest.approx(float(1e-3 * (lse.double() ** 2).mean()), rel=1e-6)
    o = _check(logits, b, k, "sigmoid")
    same = (o["idx"] == r["idx"]).all(1)
    assert same.float().mean() > 0.99  # moe_route leaves near ties open
    torch.testing.assert_close(o["gate"][same], r["gate"][same], rtol=32 * U, atol=0)


@pytest.mark.parametrize("T,d,E", [(300, 256, 40), (1000, 384, 128), (77, 128, 200), (1, 128, 3)])
def test_router_weight_gradient(T, d, E):
    g = torch.Generator().manual_seed(E)
    dl = torch.randn(T, E, generator=g).cuda()
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
    dW = torch.full((E, d), float("nan"), device="cuda")
    ws = torch.empty(ops.moe_workspace_bytes(T, d, E, 1), dtype=torch.uint8, device="cuda")
    ops.moe_router_dw(dl, x, dW, ws)
    torch.cuda.synchronize()
    want = dl.double().t() @ x.double()
    mag = dl.double().abs().t() @ x.double().abs()
    assert ((dW.double() - want).abs() <= (T + 8) * U * mag).all()


# ------------------------------------------------------------------------------- backward

def _bwd(dg, idx, score, l, lse, mode, renorm, scale, E, **kw):
    out = torch.full((dg.shape[0], E), float("nan"), device="cuda")
    ops.moe_select_experts_bwd(dg, idx, score, l, lse, MODE[mode], renorm, scale, out, **kw)
    return out


def _bwd_reference(dg, idx, s, l, mode, renorm, scale, z_coef=0.0):
    T, E = l.shape
    S = s.sum(1, keepdims=True)
    if renorm:
        with np.errstate(all="ignore"):
            ds = np.where(S == 0, 0.0, scale / S * (dg - (s / S * dg).sum(1, keepdims=True)))
    else:
        ds = scale * dg
    up = np.zeros((T, E))
    for i in range(idx.shape[1]):
        up[np.arange(T), idx[:, i]] += ds[:, i] * (s[:, i] * (1 - s[:, i]) if mode == "sigmoid" else 1)
    if mode == "sigmoid":
        return up
    p, lse = _scores(l, "softmax")
    lse = np.where(np.isfinite(lse), lse, 0.0)[:, None]
    c = 0.0 if renorm else (s * ds).sum(1, keepdims=True)
    return p * (up - c) + 2 * z_coef / T * lse * p


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k,G,tg", [(1, 8, 2, 1, 1), (1, 256, 8, 8, 4), (65, 64, 8, 8, 3),
                                        (300, 100, 5, 10, 4), (33, 31, 31, 1, 1), (129, 255, 32, 5, 2),
                                        (3000, 128, 8, 1, 1), (9, 1, 1, 1, 1)])
def test_choice_bwd_matches_64_bits(T, E, k, G, tg, renorm, mode):
    """Bounds: a slot's gradient is a product and quotient of values off by at most 4 u (the scores
    are this test's input) and a difference of sums over k terms; 64 u of the magnitudes that
    meet in it covers every case, and the softmax probabilities are off by (R + 40) u."""
    g = torch.Generator().manual_seed(T + E)
    l = torch.randn(T, E, generator=g).cuda()
    b = (torch.rand(E, generator=g) * 0.1).cuda()
    o = _select(l, b, k, mode, G, tg, "top2", renorm, 2.5)
    dg = torch.randn(T, k, generator=g).cuda()
    extra = torch.randn(T, E, generator=g).cuda()
    z = 1e-2 if mode == "softmax" else 0.0
    l64, dg64, s64 = (t.double().cpu().numpy() for t in (l, dg, o["score"]))
    idx = o["idx"].cpu().numpy()
    R = l64.max() - l64.min()
    S = s64.sum(1, keepdims=True) if renorm else 1.0
    p = _scores(l64, "softmax")[0] if mode == "softmax" else 1.0
    mag = 2.5 / S * (np.abs(dg64).max(1, keepdims=True) * 2) * p
    for zc, ex in ((0.0, None), (z, extra)):
        got = _bwd(dg, o["idx"], o["score"], l, o["lse"], mode, renorm, 2.5, E, z_coef=zc, dlogits_extra=ex)
        torch.cuda.synchronize()
        want = _bwd_reference(dg64, idx, s64, l64, mode, renorm, 2.5, zc)
        tol = (64 + (R + 40 if mode == "softmax" else 0)) * U * (mag + np.abs(want))
        if ex is not None:
            want = want + ex.double().cpu().numpy()
            tol = tol + 2 * U * np.abs(want)
        off = np.abs(got.double().cpu().numpy() - want)
        assert (off <= tol + 1e-37).all(), float((off - tol).max())
    inplace = extra.clone()
    ops.moe_select_experts_bwd(dg, o["idx"], o["score"], l, o["lse"], MODE[mode], renorm, 2.5, inplace,
                               z_coef=z, dlogits_extra=inplace)
    torch.cuda.synchronize()
    assert torch.equal(inplace, got)


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_choice_gradient_against_differences(mode, renorm):
    """The kernel's gradient of <gate, dg>, against central differences of the 64-bit gates with
    the choice held."""
    T, E, k, h = 4, 24, 4, 1e-5
    g = torch.Generator().manual_seed(21)
    l = torch.randn(T, E, generator=g).cuda()
    dg = torch.randn(T, k, generator=g).cuda()
    o = _select(l, None, k, mode, 4, 2, "top2", renorm, 1.5)
    got = _bwd(dg, o["idx"], o["score"], l, o["lse"], mode, renorm, 1.5, E).double().cpu().numpy()
    l64, idx, dg64 = l.double().cpu().numpy(), o["idx"].cpu().numpy(), dg.double().cpu().numpy()

    def loss(l):
        s = np.take_along_axis(_scores(l, mode)[0], idx, 1)
        return (1.5 * (s / s.sum(1, keepdims=True) if renorm else s) * dg64).sum()
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(l64)
            d[t, e] = h
            assert abs((loss(l64 + d) - loss(l64 - d)) / (2 * h) - got[t, e]) < 2e-6


def test_choice_bwd_of_rows_without_scores():
    """Rows whose logits are all -inf, or whose chosen sigmoids vanish, have a gradient of zero."""
    l = torch.randn(4, 16).cuda()
    l[1] = -float("inf")
    l[2] = -1000.0
    dg = torch.randn(4, 3).cuda()
    for mode in ("sigmoid", "softmax"):
        for renorm in (False, True):
            o = _select(l, None, 3, mode, 1, 1, "max", renorm)
            d = _bwd(dg, o["idx"], o["score"], l, o["lse"], mode, renorm, 1.0, 16,
                     z_coef=1e-2 if mode == "softmax" else 0.0)
            torch.cuda.synchronize()
            assert (d[1] == 0).all() and torch.isfinite(d).all()
            if mode == "sigmoid":
                assert (d[2] == 0).all()


@pytest.mark.parametrize("mode,z", [("sigmoid", 0.0), ("softmax", 0.0), ("softmax", 1e-2)])
def test_choice_bwd_of_scores_below_the_normal_range(mode, z):
    """Renormalised gates of chosen scores around e^-95: 1 / S is no fp32 number, but the gates'
    gradient is of their ordinary size. A slot's share of S is off by 9 u (eight terms' sum, a
    division), the mean over the slots by as much again and their products' roundings: 64 u of
    scale * share * 2 max|dg| covers them. The z-loss's part is that of test_choice_bwd_matches_64_bits."""
    T, E, k = 37, 64, 8
    g = torch.Generator().manual_seed(77)
    l = torch.randn(T, E, generator=g) - 95
    if mode == "softmax":
        l[:, -1] = 0.0  # takes all the probability, and a bias keeps it out of the choice
    l = l.cuda()
    b = torch.zeros(E, device="cuda")
    b[-1] = -4.0
    o = _select(l, b, k, mode, scale=2.5)
    dg = torch.randn(T, k, generator=g).cuda()
    got = _bwd(dg, o["idx"], o["score"], l, o["lse"], mode, True, 2.5, E, z_coef=z)
    torch.cuda.synchronize()
    idx = o["idx"].cpu().numpy()
    s, dg64 = o["score"].double().cpu().numpy(), dg.double().cpu().numpy()
    assert (s > 0).all() and (s < 1e-38).all() and (idx != E - 1).all()
    share = s / s.sum(1, keepdims=True)
    want, tol = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, idx, 2.5 * share * (dg64 - (share * dg64).sum(1, keepdims=True)), 1)
    np.put_along_axis(tol, idx, 64 * U * 2.5 * share * 2 * np.abs(dg64).max(1, keepdims=True), 1)
    if z:
        p, lse = _scores(l.double().cpu().numpy(), mode)
        zl = 2 * z / T * lse[:, None] * p
        want, tol = want + zl, tol + (64 + 100 + 40) * U * np.abs(zl) + U * np.abs(want)
    assert (np.abs(got.double().cpu().numpy() - want) <= tol + 1e-37).all()


def test_choice_bwd_drops_bad_indices_and_adds_repeated_ones():
    T, E, k = 5, 40, 4
    g = torch.Generator().manual_seed(5)
    l = torch.randn(T, E, generator=g).cuda()
    dg = torch.randn(T, k, generator=g).cuda()
    o = _select(l, None, k, "sigmoid")
    idx, s = o["idx"].clone(), o["score"].clone()
    idx[1, 2], idx[3, 0] = E, -1
    idx[2, 3] = idx[2, 1]
    s[2, 3] = s[2, 1]
    ops.moe_clear_device_status()
    d = _bwd(dg, idx, s, None, None, "sigmoid", False, 1.0, E)
    code, site = ops.moe_device_status()
    ops.moe_clear_device_status()
    assert (code, site) == (5, 60)
    i64, s64, dg64 = idx.cpu().numpy().astype(np.int64), s.double().cpu().numpy(), dg.double().cpu().numpy()
    want = np.zeros((T, E))
    for t in range(T):
        for i in range(k):
            if 0 <= i64[t, i] < E:
                want[t, i64[t, i]] += dg64[t, i] * s64[t, i] * (1 - s64[t, i])
    assert np.abs(d.double().cpu().numpy() - want).max() <= 16 * U * np.abs(dg64).max() * 2


def test_choice_on_a_stream_and_in_a_graph():
    T, E, k = 333, 256, 8
    g = torch.Generator().manual_seed(6)
    l = torch.randn(T, E, generator=g).cuda()
    b = (torch.rand(E, generator=g) * 0.1).cuda()
    want = _select(l, b, k, "sigmoid", 8, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _select(l, b, k, "sigmoid", 8, 4, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got["idx"], want["idx"]) and torch.equal(got["gate"], want["gate"])
    dg, dl = torch.randn(T, k, generator=g).cuda(), torch.empty(T, E, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_select_experts(l, b, k, 0, 8, 4, 1, True, 2.5, got["idx"], got["gate"], got["score"])
        ops.moe_select_experts_bwd(dg, got["idx"], got["score"], None, None, 0, True, 2.5, dl)
    for seed in (7, 8):
        l.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        o = _select(l, b, k, "sigmoid", 8, 4, scale=2.5)
        d = _bwd(dg, o["idx"], o["score"], None, None, "sigmoid", True, 2.5, E)
        torch.cuda.synchronize()
        assert torch.equal(got["idx"], o["idx"]) and torch.equal(got["gate"], o["gate"])
        assert torch.equal(dl, d)


def test_choice_refuses_mismatched_tensors():
    l, b = torch.randn(4, 32).cuda(), torch.zeros(32).cuda()
    i, f = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(4, 2, device="cuda")
    f2 = torch.empty_like(f)
    bad = [(l.half(), b, i, f, f2), (l, b[:16], i, f, f2), (l, b.double(), i, f, f2), (l, b, i.long(), f, f2),
           (l, b, i[:3].contiguous(), f, f2), (l, b, i, f[:, :1].contiguous(), f2), (l, b, i, f, None)]
    for a in bad:
        with pytest.raises(ops.MoEError):
            ops.moe_select_experts(a[0], a[1], 2, 0, 1, 1, 1, True, 1.0, a[2], a[3], a[4])
    with pytest.raises(ops.MoEError, match="invalid argument"):
        ops.moe_select_experts(l, b, 2, 0, 5, 1, 1, True, 1.0, i, f, f2)  # 32 experts in 5 groups
