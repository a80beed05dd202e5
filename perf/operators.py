"""Workloads of the operators around the MoE layer in a pretraining step, each in a plain form
(elementary torch operations) and as the calls of the library's entry points.

* norm, norm_bwd: the residual stream's addition and the root-mean-square norm in front of the
  layer, with the E4M3 codes that the FP8 experts read; and its backward.
* select, select_bwd: the choice of experts from router logits (sigmoid or softmax scores, a
  selection bias, groups of experts, top-k, renormalised and scaled gates); and its backward.
* clip: the global norm over a step's gradients, and the clipped gradients.

Sizes are those of the layer workloads in ``configs.py`` where a case says so. ``run`` makes
one pass; ``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6          # of the norm
E4M3_MAX = 448.0
MAX_NORM = 1.0      # of the clipped gradients
SCALE = 2.5         # of renormalised sigmoid gates


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through an FP8 layer in serving (d of the large layer): latency
        dict(name="norm_token_codes", op="norm", T=1, d=4096, residual="bf16", codes=True),
        # the small fine-grained layer's tokens, less one (a ragged batch), training
        dict(name="norm_train_ragged", op="norm", T=8191, d=1024, residual="bf16", codes=False),
        # the large layer with FP8 experts and a residual stream kept in fp32
        dict(name="norm_large_f32_codes", op="norm", T=65536, d=4096, residual="f32", codes=True),
        # backward of the small fine-grained layer's norm
        dict(name="norm_bwd_train", op="norm_bwd", T=8192, d=1024, residual="bf16"),
        # backward of the large layer's norm
        dict(name="norm_bwd_large", op="norm_bwd", T=65536, d=4096, residual="bf16"),
        # one token in serving: many experts in eight groups
        dict(name="select_token_groups", op="select", T=1, E=256, k=8, mode="sigmoid", bias=True,
             n_group=8, topk_group=4, rule="top2", renorm=True),
        # the large layer's tokens, the widest router, in groups
        dict(name="select_large_groups", op="select", T=65536, E=256, k=8, mode="sigmoid",
             bias=True, n_group=8, topk_group=4, rule="top2", renorm=True),
        # softmax scores over an expert count that is no power of two, ragged token count
        dict(name="select_softmax_ragged", op="select", T=16383, E=160, k=6, mode="softmax",
             bias=False, n_group=8, topk_group=3, rule="max", renorm=False),
        # backward of the large choice: few chosen experts, a dense output
        dict(name="select_bwd_large", op="select_bwd", T=65536, E=256, k=8, mode="sigmoid",
             renorm=True),
        # softmax without renormalised gates: every expert's logit has a gradient
        dict(name="select_bwd_softmax", op="select_bwd", T=32768, E=128, k=8, mode="softmax",
             renorm=False),
        # gradients of the tiny layer: latency
        dict(name="clip_tiny", op="clip", layers=1, E=8, f=128, d=256),
        # gradients of the large layer's routed experts and router
        dict(name="clip_large", op="clip", layers=1, E=64, f=1536, d=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "select", "select", "select_bwd", "clip"])
    if op in ("norm", "norm_bwd"):
        d = 8 * _log_int(rng, 16, 2048)
        T = _log_int(rng, 1, 65536 * 4096 // max(d, 4096))
        case = dict(op=op, T=T, d=d, residual=rng.choice(["bf16", "f32"]))
        if op == "norm":
            case["codes"] = rng.random() < 0.5
        return case
    if op == "select":
        n_group = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(-(-8 // n_group), 256 // n_group)
        E = n_group * per
        topk_group = rng.randint(-(-n_group // 2), n_group)
        mode = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=rng.randint(1, min(8, topk_group * per)),
                    mode=mode, bias=mode == "sigmoid" or rng.random() < 0.5, n_group=n_group,
                    topk_group=topk_group, rule=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.7)
    if op == "select_bwd":
        E = rng.randint(8, 256)
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=rng.randint(1, 8),
                    mode=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.5)
    f, d = 128 * rng.randint(1, 8), 128 * rng.randint(1, 16)
    E = rng.choice([4, 8, 16, 32, 64])
    return dict(op=op, layers=rng.randint(1, max(1, min(10, (1 << 29) // (3 * E * f * d)))), E=E,
                f=f, d=d)


def _clip_shapes(c):
    """(shape, dtype) of every gradient: per layer the experts' three matrices (bf16), the
    router's and the norm's weights (fp32), and a vector of odd length."""
    E, f, d = c["E"], c["f"], c["d"]
    one = [((E, f, d), torch.bfloat16), ((E, f, d), torch.bfloat16), ((E, d, f), torch.bfloat16),
           ((E, d), torch.float32), ((d,), torch.float32), ((d + 1,), torch.bfloat16)]
    return one * c["layers"]


def work(c):
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        n, r = c["T"] * c["d"], 2 if c["residual"] == "bf16" else 4
        if op == "norm":  # x and the residual in, the residual, y (and the codes) out
            return {"bytes": n * (2 + r + r + 2 + (1 if c["codes"] else 0)) + 4 * c["d"]
                    + c["T"] * (8 if c["codes"] else 4), "flops": 7 * n}
        # dy, the residual's gradient and z in, the gradients out
        out = 2 if r == 2 else 6
        return {"bytes": n * (2 + r + r + out) + 8 * c["d"] + 4 * c["T"], "flops": 11 * n}
    if op == "select":
        T, E, k = c["T"], c["E"], c["k"]
        lse = 4 * T if c["mode"] == "softmax" else 0
        return {"bytes": 4 * T * E + 12 * T * k + lse + (4 * E if c["bias"] else 0),
                "flops": 8 * T * E}
    if op == "select_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        dense = c["mode"] == "softmax" and not c["renorm"]
        return {"bytes": 4 * T * E + 12 * T * k + ((4 * T * E + 4 * T) if dense else 0),
                "flops": (4 * T * E if dense else 0) + 10 * T * k}
    shapes = _clip_shapes(c)
    n = sum(math.prod(s) for s, _ in shapes)
    b = sum(math.prod(s) * t.itemsize for s, t in shapes)
    return {"bytes": 2 * b + 8, "flops": 3 * n}


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE)


def _rdtype(c):
    return torch.bfloat16 if c["residual"] == "bf16" else torch.float32


def _norm_inputs(c, g):
    """A block's output and a residual stream with a few channels far larger than the rest (the
    streams of trained models have them)."""
    T, d = c["T"], c["d"]
    chan = 1.0 + 7.0 * (torch.rand((d,), generator=g, device=DEVICE) > 0.99).float()
    return dict(x=_randn(g, T, d).to(torch.bfloat16),
                residual=(2.0 * _randn(g, T, d) * chan).to(_rdtype(c)),
                w=1.0 + 0.1 * _randn(g, d))


def _logits(T, E, g):
    """Router logits with experts of unequal popularity; every 64th token is padding, whose
    logits are all zero."""
    l = _randn(g, T, E) + 0.3 * _randn(g, E)
    l[63::64] = 0.0
    return l.contiguous()


def _choice(l, c, g):
    """Distinct experts of each token, and their scores, as a forward pass leaves them."""
    T, E = l.shape
    s = torch.sigmoid(l) if c["mode"] == "sigmoid" else torch.softmax(l, -1)
    idx = torch.argsort(torch.rand((T, E), generator=g, device=DEVICE) * 0.05 + s, dim=-1,
                        descending=True)[:, :c["k"]].contiguous()
    return idx.to(torch.int32), torch.gather(s, 1, idx).contiguous()


def _clip_inputs(c, g):
    """Gradients whose scale differs from tensor to tensor; every eighth expert saw no token
    and has none."""
    grads = []
    for i, (shape, dtype) in enumerate(_clip_shapes(c)):
        t = torch.empty(shape, device=DEVICE, dtype=dtype).normal_(0.0, 10.0 ** -(2 + i % 3),
                                                                   generator=g)
        if len(shape) == 3:
            t[7::8] = 0
        grads.append(t)
    return grads


def prepare(c, seed):
    g, dev, op = _gen(seed), DEVICE, c["op"]
    f32, bf16 = torch.float32, torch.bfloat16
    s = {"case": c}
    if op == "norm":
        T, d = c["T"], c["d"]
        s.update(_norm_inputs(c, g))
        s.update(z=torch.empty((T, d), dtype=_rdtype(c), device=dev),
                 y=torch.empty((T, d), dtype=bf16, device=dev),
                 rstd=torch.empty((T,), dtype=f32, device=dev), yq=None, sy=None)
        if c["codes"]:
            s.update(yq=torch.empty((T, d), dtype=torch.uint8, device=dev),
                     sy=torch.empty((T,), dtype=f32, device=dev))
    elif op == "norm_bwd":
        T, d = c["T"], c["d"]
        i = _norm_inputs(c, g)
        z = i["residual"]
        s.update(z=z, w=i["w"], dy=i["x"], dres=_randn(g, T, d).to(_rdtype(c)),
                 rstd=1.0 / torch.sqrt(z.float().square().mean(-1) + EPS),
                 dz=torch.empty((T, d), dtype=_rdtype(c), device=dev),
                 dx=torch.empty((T, d), dtype=bf16, device=dev) if c["residual"] == "f32" else None,
                 dw=torch.empty((d,), dtype=f32, device=dev))
        s["ws"] = _workspace(T, d, 1, 1)
    elif op == "select":
        T, E, k = c["T"], c["E"], c["k"]
        s.update(logits=_logits(T, E, g),
                 b=torch.rand((E,), generator=g, device=dev) * 0.1 - 0.05 if c["bias"] else None,
                 idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                 gate=torch.empty((T, k), dtype=f32, device=dev),
                 score=torch.empty((T, k), dtype=f32, device=dev),
                 lse=torch.empty((T,), dtype=f32, device=dev) if c["mode"] == "softmax" else None)
    elif op == "select_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        l = _logits(T, E, g)
        idx, score = _choice(l, c, g)
        s.update(idx=idx, score=score, dg=_randn(g, T, k),
                 logits=l if c["mode"] == "softmax" else None,
                 lse=torch.logsumexp(l, -1) if c["mode"] == "softmax" else None,
                 dlogits=torch.empty((T, E), dtype=f32, device=dev))
    else:
        grads = _clip_inputs(c, g)
        s.update(grads=grads, out=[torch.empty_like(t) for t in grads],
                 norm=torch.empty((2,), dtype=f32, device=dev), ws=_workspace(1, 128, 1, 1))
    return s


def _workspace(T, d, E, k):
    """The library's scratch for these sizes, which a program allocates once."""
    if own:
        from pretraining_sigmoid_softmax_gb300 import ops
        return torch.empty((ops.moe_workspace_bytes(T, d, E, k),), dtype=torch.uint8, device=DEVICE)
    return None


def _scale(c):
    return SCALE if c["mode"] == "sigmoid" and c["renorm"] else 1.0


# ------------------------------------------------------------------- the framework's calls

def _run_own(s):
    from pretraining_sigmoid_softmax_gb300 import ops
    c = s["case"]
    op = c["op"]
    if op == "norm":
        ops.moe_rms_norm(s["x"], s["residual"], s["w"], EPS, s["z"], s["y"], s["yq"], s["sy"],
                         s["rstd"])
        out = {"z": s["z"], "y": s["y"], "rstd": s["rstd"]}
        if c["codes"]:
            out.update(yq=s["yq"].view(torch.float8_e4m3fn), sy=s["sy"])
        return out
    if op == "norm_bwd":
        ops.moe_rms_norm_bwd(s["dy"], s["dres"], s["z"], s["rstd"], s["w"], s["dz"], s["dx"],
                             s["dw"], s["ws"])
        out = {"dz": s["dz"], "dw": s["dw"]}
        if s["dx"] is not None:
            out["dx"] = s["dx"]
        return out
    if op in ("select", "select_bwd"):
        mode = ops.MODE_SIGMOID if c["mode"] == "sigmoid" else ops.MODE_SOFTMAX
    if op == "select":
        rule = ops.GROUP_TOP2 if c["rule"] == "top2" else ops.GROUP_MAX
        ops.moe_select_experts(s["logits"], s["b"], c["k"], mode, c["n_group"], c["topk_group"],
                               rule, c["renorm"], _scale(c), s["idx"], s["gate"], s["score"],
                               s["lse"])
        out = {"idx": s["idx"], "gate": s["gate"], "score": s["score"]}
        if s["lse"] is not None:
            out["lse"] = s["lse"]
        return out
    if op == "select_bwd":
        ops.moe_select_experts_bwd(s["dg"], s["idx"], s["score"], s["logits"], s["lse"], mode,
                                   c["renorm"], _scale(c), s["dlogits"])
        return {"dlogits": s["dlogits"]}
    ops.moe_clip_grads(s["grads"], MAX_NORM, s["out"], s["norm"], s["ws"])
    return {"norm": s["norm"], "out": s["out"]}


# ------------------------------------------------------------------------- the plain forms

def _plain_norm(s):
    c = s["case"]
    z = (s["x"].float() + s["residual"].float()).to(_rdtype(c))
    zf = z.float()
    rstd = 1.0 / torch.sqrt(zf.square().mean(-1) + EPS)
    y = zf * rstd[:, None] * s["w"]
    out = {"z": z, "y": y.to(torch.bfloat16), "rstd": rstd}
    if c["codes"]:
        amax = y.abs().amax(-1)
        sy = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        q = (y / sy[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        out.update(yq=q.to(torch.float8_e4m3fn), sy=sy)
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    xhat = s["z"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    gw = dy * s["w"]
    dz = s["rstd"][:, None] * (gw - xhat * (gw * xhat).mean(-1, keepdim=True)) + s["dres"].float()
    out = {"dz": dz.to(_rdtype(c)), "dw": (dy * xhat).sum(0)}
    if s["dx"] is not None:
        out["dx"] = dz.to(torch.bfloat16)
    return out


def _plain_select(s):
    """The choice is made in 64 bits: two values may lie closer than 32 bits tell apart."""
    c, l = s["case"], s["logits"].double()
    T, E = l.shape
    k, G, per = c["k"], c["n_group"], E // c["n_group"]
    if c["mode"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(-1, keepdim=True)
        e = torch.exp(l - m)
        total = e.sum(-1, keepdim=True)
        p = e / total
    v = p + s["b"].double() if c["bias"] else p
    by = v if c["bias"] else l  # without a bias the scores have the logits' order
    if G > 1:
        if c["rule"] == "max":
            score = by.view(T, G, per).amax(-1)
        else:
            top = v.view(T, G, per).sort(-1, descending=True).values
            score = top[..., :2].sum(-1)
        kept = score.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        mask = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        by = torch.where(mask.repeat_interleave(per, 1), by, torch.full_like(by, -math.inf))
    idx = by.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    chosen = torch.gather(p, 1, idx)
    gate = chosen / chosen.sum(-1, keepdim=True) if c["renorm"] else chosen
    out = {"idx": idx.to(torch.int32), "gate": (gate * _scale(c)).float(), "score": chosen.float()}
    if c["mode"] == "softmax":
        out["lse"] = (m + torch.log(total))[:, 0].float()
    return out


def _plain_select_bwd(s):
    c = s["case"]
    sc, dg, idx = s["score"], s["dg"], s["idx"].long()
    a = _scale(c)
    if c["renorm"]:
        S = sc.sum(-1, keepdim=True)
        ds = a / S * (dg - (sc / S * dg).sum(-1, keepdim=True))
    else:
        ds = a * dg
    out = torch.zeros_like(s["dlogits"])
    if c["mode"] == "sigmoid":
        return {"dlogits": out.scatter_(1, idx, ds * sc * (1.0 - sc))}
    out.scatter_(1, idx, ds)
    p = torch.exp(s["logits"] - s["lse"][:, None])
    return {"dlogits": p * (out - (sc * ds).sum(-1, keepdim=True))}


def _plain_clip(s):
    sums = torch.stack([t.float().square().sum() for t in s["grads"]])
    norm = sums.double().sum().sqrt().float()
    coef = torch.where(torch.isfinite(norm) & (norm > MAX_NORM), MAX_NORM / norm,
                       torch.ones_like(norm))
    return {"norm": torch.stack([norm, coef]),
            "out": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "select": _plain_select,
          "select_bwd": _plain_select_bwd, "clip": _plain_clip}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- definitions in 64 bits

def exact(c, seed):
    """The definitions in 64 bits, from the same inputs. The choice of experts is made here by
    counting how many experts come before each one."""
    s = prepare(c, seed)
    op, f64 = c["op"], torch.float64
    if op == "norm":
        z = (s["x"].to(f64) + s["residual"].to(f64)).to(_rdtype(c))
        q = z.to(f64)
        ms = torch.einsum("td,td->t", q, q) / c["d"]
        r = (ms + EPS).rsqrt()
        y = torch.einsum("td,t,d->td", q, r, s["w"].to(f64))
        out = {"z": z.to(f64), "y": y, "rstd": r}
        if c["codes"]:
            top = torch.maximum(y.amax(1), -y.amin(1))
            sy = torch.where(top > 0, top / E4M3_MAX, 1.0)
            out.update(yq=(y / sy[:, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).to(f64),
                       sy=sy)
        return out
    if op == "norm_bwd":
        z, dy, w, r = (s[n].to(f64) for n in ("z", "dy", "w", "rstd"))
        inner = torch.einsum("td,td,d->t", dy, z, w) * r ** 3 / c["d"]
        dz = dy * w * r[:, None] - z * inner[:, None] + s["dres"].to(f64)
        out = {"dz": dz, "dw": torch.einsum("td,td,t->d", dy, z, r)}
        if s["dx"] is not None:
            out["dx"] = dz
        return out
    if op == "select":
        return _exact_select(c, s)
    if op == "select_bwd":
        sc, dg, idx = s["score"].to(f64), s["dg"].to(f64), s["idx"].long()
        a, T, E = _scale(c), c["T"], c["E"]
        if c["renorm"]:  # the Jacobian of s / sum(s), row by row
            S = sc.sum(1)
            ds = a * (dg / S[:, None] - ((sc * dg).sum(1) / S ** 2)[:, None])
        else:
            ds = a * dg
        up = torch.zeros((T, E), dtype=f64, device=DEVICE)
        if c["mode"] == "sigmoid":
            up[torch.arange(T, device=DEVICE)[:, None], idx] = ds * (sc - sc ** 2)
            return {"dlogits": up}
        up[torch.arange(T, device=DEVICE)[:, None], idx] = ds
        p = torch.softmax(s["logits"].to(f64), 1)
        return {"dlogits": p * up - p * (sc * ds).sum(1, keepdim=True)}
    total = sum(float(torch.linalg.vector_norm(t, dtype=f64)) ** 2 for t in s["grads"])
    norm = math.sqrt(total)
    coef = MAX_NORM / norm if norm > MAX_NORM else 1.0
    return {"norm": torch.tensor([norm, coef], dtype=f64, device=DEVICE),
            "out": [t.to(f64) * coef for t in s["grads"]]}


def _before(v):
    """For each entry of the last axis, how many come before it: larger ones, and equal ones of
    a lower index."""
    n = v.shape[-1]
    i = torch.arange(n, device=v.device)
    lower = i[None, :] < i[:, None]
    a, b = v[..., :, None], v[..., None, :]
    return ((b > a) | ((b == a) & lower)).sum(-1)


def _exact_select(c, s):
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    outs = []
    for t0 in range(0, T, 4096):
        l = s["logits"][t0:t0 + 4096].double()
        n = l.shape[0]
        lse = torch.logsumexp(l, 1)
        p = torch.special.expit(l) if c["mode"] == "sigmoid" else torch.exp(l - lse[:, None])
        v = p + s["b"].double()[None, :] if c["bias"] else p
        order = v if c["bias"] else l
        ok = torch.ones((n, E), dtype=torch.bool, device=l.device)
        if G > 1:
            per = E // G
            if c["rule"] == "max":
                gs = order.reshape(n, G, per).max(-1).values
            else:
                gs = torch.topk(v.reshape(n, G, per), min(2, per), dim=-1).values.sum(-1)
            ok = (_before(gs) < c["topk_group"])[:, :, None].expand(n, G, per).reshape(n, E)
        rank = _before(torch.where(ok, order, torch.full_like(order, -math.inf)))
        idx = torch.argsort(rank, dim=1)[:, :k]
        sc = p[torch.arange(n, device=l.device)[:, None], idx]
        gate = _scale(c) * (sc / sc.sum(1, keepdim=True) if c["renorm"] else sc)
        o = {"idx": idx.to(torch.int32), "gate": gate, "score": sc}
        if c["mode"] == "softmax":
            o["lse"] = lse
        outs.append(o)
    return {key: torch.cat([o[key] for o in outs]) for key in outs[0]}
