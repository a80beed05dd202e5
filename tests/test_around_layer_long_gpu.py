"""The operators around the layer on enough rows that every buffer of their pipelines is used again:
each warp or CTA of a kernel that walks rows gets at least two more of them than it has stages (or
row buffers), whatever the GPU's SM count. References are in 64 bits on the GPU; bounds are those
of test_norm_gpu and test_select_gpu, which are derived there: sums of a row pass at most 69 roundings
(80 u, u = 2^-24), a sum over T tokens T + 3; an fp32 sigmoid is off by 4 u and a gate by 16 u, a
softmax score by (R + 40) u with R the range of its row's logits."""
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
MODE = {"sigmoid": ops.MODE_SIGMOID, "softmax": ops.MODE_SOFTMAX}
RULE = {"max": ops.GROUP_MAX, "top2": ops.GROUP_TOP2}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(*shape, gen):
    return torch.randn(*shape, generator=gen, device="cuda")


# d, rows at once per SM (at most), rows that each of them has to see: the warp-per-row kernel has 3
# stages and 4 warps in each of 4 CTAs per SM, the ring of 4 stages up to 4 CTAs, that of 2 stages up
# to 2, the kernel for wide rows 608 CTAs in all
LONG = [(128, 16, 5), (256, 16, 5), (512, 16, 5), (1000, 16, 5), (2048, 4, 6), (4096, 2, 6), (8192, 2, 4),
        (9216, 4, 3), (16384, 4, 3)]


@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,per_sm,rows", LONG)
def test_norm_bwd_of_many_rows(d, per_sm, rows, rdtype):
    T = per_sm * _sms() * rows + 3
    g = _gen(d)
    dy, z, w = _randn(T, d, gen=g).to(torch.bfloat16), _randn(T, d, gen=g).to(rdtype), 1 + 0.2 * _randn(d, gen=g)
    dres = _randn(T, d, gen=g).to(rdtype)
    rstd = 1.0 / torch.sqrt(z.float().square().mean(1) + 1e-6)
    dz, dw = torch.full_like(z, float("nan")), torch.full((d,), float("nan"), device="cuda")
    dx = torch.full_like(dy, float("nan")) if rdtype is torch.float32 else None
    ws = torch.full((ops.moe_workspace_bytes(T, d, 1, 1),), 255, dtype=torch.uint8, device="cuda")
    ops.moe_rms_norm_bwd(dy, dres, z, rstd, w, dz, dx, dw, ws)
    # w's gradient column by column block, the rest row by row block: 64-bit temporaries stay small
    r64 = rstd.double()[:, None]
    for c in range(0, d, 512):
        prod = dy[:, c:c + 512].double() * (z[:, c:c + 512].double() * r64)
        off = (dw[c:c + 512].double() - prod.sum(0)).abs()
        assert (off <= (T + 3) * U * prod.abs().sum(0)).all(), c
    for t in range(0, T, 1024):
        s = slice(t, min(t + 1024, T))
        h, gg, dr = z[s].double() * r64[s], dy[s].double() * w.double(), dres[s].double()
        c = (gg * h).mean(1, keepdim=True)
        want = r64[s] * (gg - h * c) + dr
        e = (80 * U * (gg * h).abs().mean(1, keepdim=True) + 2 * U * c.abs()) * h.abs() * r64[s]
        e = e + r64[s] * 5 * U * (gg.abs() + (h * c).abs()) + 2 * U * (want.abs() + dr.abs())
        assert ((dz[s].double() - want).abs() <= e + HALF[rdtype] * (want.abs() + e)).all(), t
        if dx is not None:
            assert ((dx[s].double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all(), t


def _scores(l, mode):
    """64-bit scores of finite logits; softmax: their logsumexp and range too."""
    if mode == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l)), None, 0.0
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    S = e.sum(1, keepdim=True)
    return e / S, (m + torch.log(S))[:, 0], m - l.amin(1, keepdim=True)


def _first(v, n):
    """The n largest of each row, the lower index first among equals."""
    return torch.sort(v, dim=1, descending=True, stable=True)[1][:, :n]


def _choose(s, order, v, k, G, tg, rule):
    T, E = s.shape
    if G > 1:
        per = E // G
        if rule == "max":
            gs = order.view(T, G, per).amax(2)
        else:
            gs = v.view(T, G, per).topk(min(2, per), 2)[0].sum(2)
        ok = torch.zeros(T, G, dtype=torch.bool, device=s.device).scatter_(1, _first(gs, tg), True)
        order = torch.where(ok.repeat_interleave(per, 1), order, -float("inf"))
    return _first(order, k)


# experts, slots, groups, groups kept: whole vectors a lane and single loads, 8, 16 and 32 lanes a token
SHAPES = [(64, 8, 1, 1), (256, 8, 8, 4), (160, 6, 8, 3), (100, 5, 10, 4), (72, 8, 1, 1), (256, 16, 2, 1),
          (255, 12, 5, 3), (256, 32, 8, 4)]


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", ["none", "spread", "levels"])
@pytest.mark.parametrize("E,k,G,tg", SHAPES)
def test_choice_of_more_tokens_than_are_resident(E, k, G, tg, bias, mode):
    """At least three steps for every warp (64 tokens per SM at once, with 8 lanes a token), one row in
    64 of equal logits as padding makes them; biases of few levels, equal ones among them, as a rule
    that moves each by a step makes them. (Levels and the padded rows' scores are such that sums of
    them are exact or equal in any order, so that equal values are equal for the reference too.)"""
    T = 3 * 64 * _sms() + 817
    g = _gen(E + k)
    l = _randn(T, E, gen=g)
    l[::64] = 0.0
    b = None
    if bias == "spread":
        b = torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1
    elif bias == "levels":
        b = torch.randint(-3, 4, (E,), generator=g, device="cuda").float() * 2.0 ** -10
    l64, b64 = l.double(), None if b is None else b.double()
    s, lse, R = _scores(l64, mode)
    v = s if b is None else s + b64
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate, score = torch.empty(T, k, device="cuda"), torch.empty(T, k, device="cuda")
    lse32 = torch.empty(T, device="cuda") if mode == "softmax" else None
    for rule in ("max", "top2"):
        want = _choose(s, l64 if b is None else v, v, k, G, tg, rule)
        for t in (idx, gate, score):
            t.fill_(-7)
        ops.moe_select_experts(l, b, k, MODE[mode], G, tg, RULE[rule], True, 2.5, idx, gate, score, lse32)
        wrong = (idx != want).any(1).nonzero()[:, 0]
        assert len(wrong) == 0, f"{len(wrong)} rows, e.g. {int(wrong[0])}: {idx[wrong[0]]} for {want[wrong[0]]}"
        ws = s.gather(1, want)
        wg = 2.5 * ws / ws.sum(1, keepdim=True)
        rel = 4 * U if mode == "sigmoid" else (R + 40) * U
        assert ((score.double() - ws).abs() <= rel * ws).all()
        assert ((gate.double() - wg).abs() <= (2 * rel + 8 * U) * wg).all()
        if mode == "softmax":
            assert ((lse32.double() - lse).abs() <= rel[:, 0] + 4 * U * (lse.abs() + 8)).all()


@pytest.mark.parametrize("mode,renorm,z", [("sigmoid", True, 0.0), ("sigmoid", False, 0.0), ("softmax", True, 0.0),
                                           ("softmax", False, 0.0), ("softmax", True, 1e-2)])
@pytest.mark.parametrize("E,k", [(256, 8), (100, 5), (64, 12), (96, 32)])
def test_choice_bwd_of_more_tokens_than_are_resident(E, k, mode, renorm, z):
    """At least three passes of every warp's loop (128 tokens per SM at once, with 8 lanes a token).
    Bounds as in test_choice_bwd_matches_64_bits: 64 u of the magnitudes that meet, and the
    probabilities' (R + 40) u."""
    T, scale = 2 * 128 * _sms() + 1091, 2.5
    g = _gen(E + k)
    l = _randn(T, E, gen=g)
    s_all, lse, R = _scores(l.double(), mode)
    idx = _first(l, k)
    score = s_all.gather(1, idx).float()
    dg, extra = _randn(T, k, gen=g), _randn(T, E, gen=g)
    got = torch.full((T, E), float("nan"), device="cuda")
    ops.moe_select_experts_bwd(dg, idx.int(), score, l, None if lse is None else lse.float(), MODE[mode], renorm,
                               scale, got, z_coef=z, dlogits_extra=extra)
    s, dg64 = score.double(), dg.double()
    S = s.sum(1, keepdim=True) if renorm else 1.0
    ds = scale / S * (dg64 - (s / S * dg64).sum(1, keepdim=True)) if renorm else scale * dg64
    up = torch.zeros_like(s_all).scatter_(1, idx, ds * s * (1 - s) if mode == "sigmoid" else ds)
    if mode == "sigmoid":
        want, p = up, 1.0
    else:
        p, L = s_all, lse[:, None]
        c = 0.0 if renorm else (s * ds).sum(1, keepdim=True)
        want = p * (up - c) + 2 * z / T * L * p
    mag = scale / S * (dg64.abs().amax(1, keepdim=True) * 2) * p
    tol = (64 + (float(R.max()) + 40 if mode == "softmax" else 0)) * U * (mag + want.abs())
    want = want + extra.double()
    assert ((got.double() - want).abs() <= tol + 2 * U * want.abs() + 1e-37).all()


@pytest.mark.parametrize("E", [200, 256])
def test_router_logits_and_weight_gradient_of_many_experts(E):
    """Above 128 experts, tokens that fill no tile: logits, their logsumexp and dW_r. A logit sums d
    products in order (d + 1 roundings), a weight's gradient T of them."""
    T, d = 64 * _sms() + 5, 256
    g = _gen(E)
    x, W = _randn(T, d, gen=g).to(torch.bfloat16), _randn(E, d, gen=g) / 16
    ws = torch.empty(ops.moe_workspace_bytes(T, d, E, 1), dtype=torch.uint8, device="cuda")
    logits, lse = torch.empty(T, E, device="cuda"), torch.empty(T, device="cuda")
    ops.moe_router_logits(x, W, logits, ws, lse)
    want, mag = x.double() @ W.double().t(), x.double().abs() @ W.double().abs().t()
    assert ((logits.double() - want).abs() <= (d + 1) * U * mag).all()
    ref = torch.logsumexp(logits.double(), 1)
    R = (logits.amax(1) - logits.amin(1)).double()
    assert ((lse.double() - ref).abs() <= (R + 40) * U + 4 * U * (ref.abs() + 8)).all()
    dl, dW = _randn(T, E, gen=g), torch.empty(E, d, device="cuda")
    ops.moe_router_dw(dl, x, dW, ws)
    want, mag = dl.double().t() @ x.double(), dl.double().abs().t() @ x.double().abs()
    assert ((dW.double() - want).abs() <= (T + 8) * U * mag).all()
