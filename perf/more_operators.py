"""Workloads of the experts on microscaled 4-bit floating point (E2M1 codes with a scale for each
block along the contraction), each in a plain form (elementary torch operations) and as the calls
of the library's entry points.

* quant: a matrix's rows to codes and scales, and back to the values that they stand for;
  quant_t: weights scaled along their columns, codes transposed (the backward's operand).
* product: the rows of each expert times that expert's weights, from codes.
* experts: token rows quantised, dispatched to their experts and run through SwiGLU experts.
* dgrad: the data gradients of those experts.

Formats: "mx", blocks of 32 under a power of two (E8M0); "nv", blocks of 16 under an E4M3 scale, with
one power of two for each row. Sizes are those of the layer workloads in ``configs.py`` where a
case says so. ``run`` makes one pass; ``exact`` gives the same outputs from the definitions in 64
bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
ALIGN = 128       # rows of an expert's segment are padded to a multiple of this


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token's row in front of an expert layer (d of the large layer): latency
        dict(name="quant_token", op="quant", rows=1, cols=4096, fmt="nv"),
        # the large layer's tokens, less one (a ragged batch)
        dict(name="quant_large_ragged", op="quant", rows=65535, cols=4096, fmt="mx"),
        # the small fine-grained layer's down projections, for its data gradients
        dict(name="quant_t_small", op="quant_t", E=64, K0=1024, N=256, stack=False, fmt="nv"),
        # the skewed layer's gate and up projections as one operand
        dict(name="quant_t_stack", op="quant_t", E=128, K0=768, N=2048, stack=True, fmt="mx"),
        # one token's eight rows through the large layer's gate projections: serving
        dict(name="product_token", op="product", T=1, E=64, k=8, K=4096, N=1536, fmt="mx"),
        # the softmax layer's gate projections
        dict(name="product_softmax", op="product", T=16384, E=32, k=4, K=2048, N=1024, fmt="nv"),
        # the large layer's down projections
        dict(name="product_large", op="product", T=65536, E=64, k=8, K=1536, N=4096, fmt="mx"),
        # one token through the large layer's experts, nothing kept for a backward: serving
        dict(name="experts_token", op="experts", T=1, E=64, k=8, d=4096, f=1536, keep=False,
             fmt="mx"),
        # the small fine-grained layer's experts, training, one token less
        dict(name="experts_train_ragged", op="experts", T=8191, E=64, k=8, d=1024, f=256,
             keep=True, fmt="nv"),
        # the layer with the most experts, training
        dict(name="experts_train_large", op="experts", T=32768, E=128, k=8, d=2048, f=768,
             keep=True, fmt="mx"),
        # data gradients of the small fine-grained layer's experts
        dict(name="dgrad_small", op="dgrad", T=8192, E=64, k=8, d=1024, f=256, fmt="nv"),
        # data gradients of the layer with the most experts
        dict(name="dgrad_large", op="dgrad", T=32768, E=128, k=8, d=2048, f=768, fmt="mx"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "quant_t", "product", "product", "experts", "experts", "dgrad"])
    fmt = rng.choice(["mx", "nv"])
    if op == "quant":
        cols = 128 * _log_int(rng, 1, 64)
        return dict(op=op, rows=_log_int(rng, 1, 65535 * 4096 // max(cols, 4096)), cols=cols,
                    fmt=fmt)
    if op == "quant_t":
        K0, N = 128 * rng.randint(1, 16), 128 * rng.randint(1, 16)
        return dict(op=op, E=_log_int(rng, 1, max(1, min(128, 128 * 768 * 2048 // (K0 * N)))),
                    K0=K0, N=N, stack=rng.random() < 0.5, fmt=fmt)
    a, b = 128 * _log_int(rng, 1, 32), 128 * _log_int(rng, 1, 32)
    E = _log_int(rng, 1, min(128, (1 << 29) // (a * b)))
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, max(1, min(65536, (1 << 38) // (k * a * b))))
    if op == "product":
        return dict(op=op, T=T, E=E, k=k, K=a, N=b, fmt=fmt)
    case = dict(op=op, T=T, E=E, k=k, d=a, f=b, fmt=fmt)
    if op == "experts":
        case["keep"] = rng.random() < 0.7
    return case


def _block(fmt):
    return 32 if fmt == "mx" else 16


def _code_bytes(rows, cols, fmt):
    """Codes, block scales and (nv) the rows' scales."""
    return rows * cols // 2 + rows * cols // _block(fmt) + (4 * rows if fmt == "nv" else 0)


def work(c):
    op, fmt = c["op"], c["fmt"]
    if op == "quant":  # read once; codes, scales and the values written
        n = c["rows"] * c["cols"]
        return {"bytes": 4 * n + _code_bytes(c["rows"], c["cols"], fmt), "flops": 4 * n}
    if op == "quant_t":
        K = c["K0"] * (2 if c["stack"] else 1)
        n = c["E"] * K * c["N"]
        return {"bytes": 4 * n + _code_bytes(c["E"] * c["N"], K, fmt), "flops": 4 * n}
    R, A = c["T"] * c["k"], min(c["E"], c["T"] * c["k"])
    if op == "product":
        K, N = c["K"], c["N"]
        return {"bytes": _code_bytes(R, K, fmt) + _code_bytes(A * N, K, fmt) + 2 * R * N,
                "flops": 2 * R * K * N}
    d, f = c["d"], c["f"]
    if op == "experts":
        kept = 6 * R * f if c["keep"] else 0
        return {"bytes": 2 * c["T"] * d + _code_bytes(2 * A * f, d, fmt) + _code_bytes(A * d, f, fmt)
                + kept + 2 * R * d, "flops": 6 * R * d * f}
    return {"bytes": 2 * R * d + 4 * R * f + _code_bytes(A * f, d, fmt) + _code_bytes(A * d, 2 * f, fmt)
            + 4 * R * f + 2 * R * d, "flops": 6 * R * d * f}


# ------------------------------------------------------------- codes and scales, plain form

_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nibbles(v):
    """E2M1 codes of v: to the nearest value, ties to the even code, at most 6."""
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    return code + (v < 0).to(torch.uint8) * 8


def _power(e):
    """2^e as fp32 for whole e from -127 to 127, made of its bits (a computed power may be rounded)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantize(x, fmt):
    """Codes [rows, cols] (one a byte), block scales [rows, blocks] as bytes and as numbers, and the
    rows' scales (nv), of a bf16 matrix."""
    rows, cols = x.shape
    b = _block(fmt)
    v = x.float().view(rows, cols // b, b)
    amax = v.abs().amax(-1)
    if fmt == "mx":
        e = torch.frexp(amax).exponent.to(torch.int32) - 1  # floor(log2(amax))
        byte = torch.where(amax > 0, (e - 2 + 127).clamp(0, 254), torch.zeros_like(e))
        s = _power(byte - 127)
        return _nibbles(v / s[..., None]).view(rows, cols), byte.to(torch.uint8), s, None
    top = amax.amax(-1)
    q = torch.frexp(top / 2688.0)  # the smallest power of two g with top <= 2688 g
    e = torch.where(q.mantissa > 0.5, q.exponent, q.exponent - 1).clamp(-126, 127)
    g = torch.where(top > 0, _power(e), torch.ones_like(top))
    s8 = (amax / g[:, None] / 6.0).to(torch.float8_e4m3fn)
    s = s8.float()
    z = v / g[:, None, None] / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    z = torch.where(s[..., None] > 0, z, torch.zeros_like(z))
    return _nibbles(z).view(rows, cols), s8.view(torch.uint8), s, g


def _decode(code, s, g):
    """The values (fp32) that codes, block scales as numbers and the rows' scales stand for."""
    rows, cols = code.shape
    lut = torch.tensor(_VALUES + tuple(-t for t in _VALUES), device=code.device)
    v = lut[code.int()].view(rows, s.shape[1], -1) * s[..., None]
    if g is not None:
        v = v * g[:, None, None]
    return v.view(rows, cols)


def _pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _unpack(q):
    return torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1)


def _tile(s):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 blocks: byte (r % 32) * 16 +
    (r % 128) / 32 * 4 + j % 4 of tile (r / 128, j / 4)."""
    rows, nb = s.shape
    rt = -(-rows // 128)
    full = torch.zeros((rt * 128, nb), dtype=torch.uint8, device=s.device)
    full[:rows] = s
    return full.view(rt, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untile(t, rows, nb):
    rt = -(-rows // 128)
    return t.view(rt, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, nb)[:rows]


def _numbers(byte, fmt):
    """Scale bytes as numbers."""
    if fmt == "mx":
        return _power(byte.int() - 127)
    return byte.view(torch.float8_e4m3fn).float()


def _made(x, fmt):
    """Codes, tiled scales and rows' scales of a matrix, as a program keeps its weights."""
    code, byte, _, g = _quantize(x, fmt)
    return dict(q=_pack(code), s=_tile(byte), g=g)


def _values(m, fmt):
    rows, cols = m["q"].shape[0], 2 * m["q"].shape[1]
    byte = _untile(m["s"], rows, cols // _block(fmt)).contiguous()
    return _decode(_unpack(m["q"]), _numbers(byte, fmt), m["g"])


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.empty(shape, device=DEVICE, dtype=torch.bfloat16).normal_(generator=g)


def _activations(g, T, d):
    """Token rows with a few channels far larger than the rest (those of trained models have
    them); every 61st token is padding, all zeros."""
    chan = 1.0 + 15.0 * (torch.rand((d,), generator=g, device=DEVICE) > 0.99).float()
    x = (_randn(g, T, d) * chan.to(torch.bfloat16))
    x[60::61] = 0
    return x


def _weights(g, E, n, k):
    return _randn(g, E * n, k).mul_(k ** -0.5)


def _layout(c, g):
    """A routing (experts of unequal popularity, one in sixteen never chosen) and the expert-major
    layout that the dispatch makes of it."""
    T, E, k = c["T"], c["E"], c["k"]
    u = torch.rand((T, E), generator=g, device=DEVICE) + 0.1 * torch.rand((E,), generator=g,
                                                                          device=DEVICE)
    if E - len(range(15, E, 16)) >= k:
        u[:, 15::16] = -1.0
    idx = torch.argsort(u, dim=1, descending=True)[:, :k]
    flat = idx.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    seg = -(-counts // ALIGN) * ALIGN
    off = torch.zeros(E + 1, dtype=torch.int64, device=DEVICE)
    off[1:] = torch.cumsum(seg, 0)
    R = -(-(T * k + E * (ALIGN - 1)) // ALIGN) * ALIGN
    order = torch.argsort(flat, stable=True)
    first = torch.cumsum(counts, 0) - counts
    e = flat[order]
    row = off[e] + torch.arange(T * k, device=DEVICE) - first[e]
    token = torch.full((R,), -1, dtype=torch.int32, device=DEVICE)
    token[row] = (order // k).to(torch.int32)
    slot = torch.empty(T * k, dtype=torch.int32, device=DEVICE)
    slot[order] = row.to(torch.int32)
    # rows of the experts that have any, side by side: what the plain form multiplies in one batch
    some = torch.nonzero(counts).view(-1)
    most = int(counts.max())
    batch = off[some][:, None] + torch.arange(most, device=DEVICE)
    filled = torch.arange(most, device=DEVICE)[None, :] < counts[some][:, None]
    return dict(row_offsets=off, perm_token=token, slot_to_row=slot.view(T, k), R=R, some=some,
                batch=torch.where(filled, batch, R), counts=counts)


def prepare(c, seed):
    g, op, fmt, bf16 = _gen(seed), c["op"], c["fmt"], torch.bfloat16
    s = {"case": c}

    def new(*shape):
        return torch.zeros(shape, dtype=bf16, device=DEVICE)

    def codes(rows, cols):
        return dict(q=torch.zeros((rows, cols // 2), dtype=torch.uint8, device=DEVICE),
                    s=torch.zeros(-(-rows // 128) * 128 * cols // _block(fmt), dtype=torch.uint8,
                                  device=DEVICE),
                    g=torch.ones(rows, device=DEVICE) if fmt == "nv" else None)

    if op == "quant":
        s.update(x=_activations(g, c["rows"], c["cols"]), codes=codes(c["rows"], c["cols"]),
                 out=new(c["rows"], c["cols"]))
    elif op == "quant_t":
        E, K0, N = c["E"], c["K0"], c["N"]
        K = 2 * K0 if c["stack"] else K0
        s.update(x0=_weights(g, E, K0, N).view(E, K0, N),
                 x1=_weights(g, E, K0, N).view(E, K0, N) if c["stack"] else None,
                 codes=codes(E * N, K), out=new(E * N, K))
    else:
        lay = _layout(c, g)
        s.update(lay)
        E, R = c["E"], lay["R"]
        if op == "product":
            x = _activations(g, c["T"], c["K"])
            rows = torch.where(lay["perm_token"][:, None] >= 0, x[lay["perm_token"].long()], 0)
            s.update(X=_made(rows, fmt), W=_made(_weights(g, E, c["N"], c["K"]), fmt),
                     Y=new(R, c["N"]))
        elif op == "experts":
            d, f = c["d"], c["f"]
            s.update(x=_activations(g, c["T"], d), W_g=_made(_weights(g, E, f, d), fmt),
                     W_u=_made(_weights(g, E, f, d), fmt), W_d=_made(_weights(g, E, d, f), fmt),
                     xc=codes(c["T"], d), X=codes(R, d), Hc=codes(R, f), H=new(R, f), Y=new(R, d))
            s.update(A=new(R, f) if c["keep"] else None, U=new(R, f) if c["keep"] else None)
        else:
            d, f = c["d"], c["f"]
            there = (lay["perm_token"] >= 0)[:, None]
            s.update(dY=_randn(g, R, d).mul_(0.1) * there, A=_randn(g, R, f) * there,
                     U=_randn(g, R, f) * there,
                     # columns of W_d, and of W_g over W_u: each output channel's codes side by side
                     W_d=_made(_weights(g, E, f, d), fmt), W_gu=_made(_weights(g, E, d, 2 * f), fmt),
                     dYc=codes(R, d), AUc=codes(R, 2 * f), dA=new(R, f), dU=new(R, f), dX=new(R, d))
    return s


# ------------------------------------------------------------------- the framework's calls

def _run_own(s):
    from pretraining_sigmoid_softmax_gb300 import ops
    c = s["case"]
    op, fmt = c["op"], ops.FP4_MX if c["fmt"] == "mx" else ops.FP4_NV

    def codes(m, *shape):
        q = m["q"].view(*shape) if shape else m["q"]
        return ops.Fp4(q, m["s"], m["g"], fmt)

    if op == "quant":
        q = codes(s["codes"])
        ops.moe_quantize_rows_fp4(s["x"], q)
        ops.moe_dequantize_fp4(q, s["out"])
        return {"values": s["out"]}
    if op == "quant_t":
        q = codes(s["codes"], c["E"], c["N"], -1)
        ops.moe_quantize_cols_fp4(s["x0"], s["x1"], q)
        ops.moe_dequantize_fp4(q, s["out"])
        return {"values": s["out"]}
    E = c["E"]
    if op == "product":
        ops.moe_grouped_gemm_fp4(codes(s["X"]), s["row_offsets"], codes(s["W"], E, c["N"], -1),
                                 s["Y"])
        return {"Y": s["Y"]}
    d, f = c["d"], c["f"]
    if op == "experts":
        xc, X, Hc = codes(s["xc"]), codes(s["X"]), codes(s["Hc"])
        ops.moe_quantize_rows_fp4(s["x"], xc)
        ops.moe_permute_fp4(xc, s["slot_to_row"], s["perm_token"], s["row_offsets"], X)
        ops.moe_expert_fwd_fp4(X, s["row_offsets"], codes(s["W_g"], E, f, -1),
                               codes(s["W_u"], E, f, -1), codes(s["W_d"], E, d, -1), s["A"], s["U"],
                               s["H"], Hc, s["Y"])
        out = {"Y": s["Y"]}
        if c["keep"]:
            out.update(A=s["A"], U=s["U"], H=s["H"])
        return out
    dYc, AUc = codes(s["dYc"]), codes(s["AUc"])
    ops.moe_quantize_rows_fp4(s["dY"], dYc, rows_limit=s["row_offsets"][E:])
    ops.moe_expert_bwd_fp4(dYc, None, None, s["A"], s["U"], None, s["row_offsets"],
                           codes(s["W_d"], E, f, -1), codes(s["W_gu"], E, d, -1), s["dX"], s["dA"],
                           s["dU"], AUc, None, None, None, None,
                           parts=ops.BWD_DH | ops.BWD_DX)
    return {"dX": s["dX"], "dA": s["dA"], "dU": s["dU"]}


# ------------------------------------------------------------------------- the plain forms

def _hat(x, fmt):
    """The values that the codes of a bf16 matrix stand for, in fp32."""
    code, _, s, g = _quantize(x, fmt)
    return _decode(code, s, g)


def _gather(t, s):
    """Rows of the experts that have any, [experts, most rows, columns], zeros where one has fewer."""
    return torch.cat([t, t.new_zeros((1, t.shape[1]))])[s["batch"]]


def _scatter(t, s):
    out = t.new_zeros((s["R"] + 1, t.shape[2]))
    out[s["batch"].view(-1)] = t.reshape(-1, t.shape[2])
    return out[:-1]


def _times(x, w, s, E):
    """Rows of each expert times its weights, [experts, rows, outputs]."""
    return torch.bmm(x, w.view(E, -1, x.shape[2])[s["some"]].transpose(1, 2))


def _plain(s):
    c = s["case"]
    op, fmt, bf16 = c["op"], c["fmt"], torch.bfloat16
    if op == "quant":
        return {"values": _hat(s["x"], fmt).to(bf16)}
    if op == "quant_t":
        x = s["x0"] if s["x1"] is None else torch.cat([s["x0"], s["x1"]], 1)
        return {"values": _hat(x.transpose(1, 2).reshape(-1, x.shape[1]), fmt).to(bf16)}
    E = c["E"]
    if op == "product":
        y = _times(_gather(_values(s["X"], fmt), s), _values(s["W"], fmt), s, E)
        return {"Y": _scatter(y.to(bf16), s)}
    if op == "experts":
        token = torch.where(s["perm_token"] >= 0, s["perm_token"], c["T"]).long()
        x = _hat(s["x"], fmt)
        x = _gather(torch.cat([x, x.new_zeros((1, x.shape[1]))])[token], s)
        a = _times(x, _values(s["W_g"], fmt), s, E)
        u = _times(x, _values(s["W_u"], fmt), s, E)
        h = (a / (1.0 + torch.exp(-a)) * u).to(bf16)
        hh = _hat(h.view(-1, c["f"]), fmt).view(h.shape)
        y = _times(hh, _values(s["W_d"], fmt), s, E)
        out = {"Y": _scatter(y.to(bf16), s)}
        if c["keep"]:
            out.update(A=_scatter(a.to(bf16), s), U=_scatter(u.to(bf16), s), H=_scatter(h, s))
        return out
    r = _times(_gather(_hat(s["dY"], fmt), s), _values(s["W_d"], fmt), s, E)
    a, u = _gather(s["A"], s).float(), _gather(s["U"], s).float()
    p = 1.0 / (1.0 + torch.exp(-a))
    da, du = (r * u * p * (1.0 + a * (1.0 - p))).to(bf16), (r * a * p).to(bf16)
    both = torch.cat([da, du], 2)
    dx = _times(_hat(both.view(-1, both.shape[2]), fmt).view(both.shape), _values(s["W_gu"], fmt), s, E)
    return {"dX": _scatter(dx.to(bf16), s), "dA": _scatter(da, s), "dU": _scatter(du, s)}


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------- definitions in 64 bits

def _pow2(e):
    """2^e in 64 bits for whole e, made of its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_float(v, bits, low):
    """v >= 0 in 64 bits to the nearest number with `bits` bits behind the leading one and a least
    exponent `low`, ties to even."""
    e = torch.frexp(v).exponent - 1
    step = _pow2(e.clamp(min=low) - bits)
    return torch.round(v / step) * step


def _exact_hat(x, fmt):
    """The values of the codes, in 64 bits, block by block of the definition."""
    v = x.double().unflatten(-1, (-1, _block(fmt)))
    top = torch.maximum(v.amax(-1, keepdim=True), -v.amin(-1, keepdim=True))
    if fmt == "mx":
        s = _pow2(torch.frexp(top.clamp(min=2.0 ** -125)).exponent - 3)
    else:
        row = top.amax(-2, keepdim=True)
        e = torch.frexp(row.clamp(min=2.0 ** -133)).exponent - 12  # 2688 = 1.3125 * 2^11
        g = _pow2((e + (row > 2688 * _pow2(e))).clamp(min=-126))
        s = g * _round_float(top / g / 6, 3, -6).clamp(max=448)
    z = (v.abs() / torch.where(s > 0, s, 1.0)).clamp(max=6)
    return (torch.sign(v) * _round_float(z, 1, 0) * s).flatten(-2)


def _exact_values(m, fmt):
    """Codes, tiled scales and rows' scales as 64-bit values, each scale byte found by its place."""
    q, nb = m["q"], 2 * m["q"].shape[1] // _block(fmt)
    r = torch.arange(q.shape[0], device=q.device)[:, None]
    j = torch.arange(nb, device=q.device)[None, :]
    at = ((r // 128) * (nb // 4) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    byte = m["s"][at]
    if fmt == "mx":
        scale = _pow2(byte.long() - 127)
    else:
        scale = byte.view(torch.float8_e4m3fn).double() * m["g"].double()[:, None]
    out = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    for half in (0, 1):
        n = (q >> (4 * half)).int() & 15
        e, m1 = (n >> 1) & 3, (n & 1).double()
        mag = torch.where(e == 0, 0.5 * m1, (1 + 0.5 * m1) * _pow2(e - 1))
        out[:, half::2] = torch.where(n >= 8, -mag, mag)
    return (out.unflatten(1, (nb, -1)) * scale[:, :, None]).flatten(1)


def exact(c, seed):
    """The definitions in 64 bits from the same inputs, expert by expert."""
    s = prepare(c, seed)
    op, fmt = c["op"], c["fmt"]
    if op == "quant":
        return {"values": torch.cat([_exact_hat(x, fmt) for x in s["x"].split(8192)])}
    if op == "quant_t":
        parts = []
        for e in range(c["E"]):
            x = s["x0"][e] if s["x1"] is None else torch.cat([s["x0"][e], s["x1"][e]])
            parts.append(_exact_hat(x.T.contiguous(), fmt))
        return {"values": torch.cat(parts)}
    E, R = c["E"], s["R"]
    lo, n = s["row_offsets"].tolist(), s["counts"].tolist()

    def blank(cols):
        return torch.zeros((R, cols), dtype=torch.float64, device=DEVICE)

    def part(m, e, rows):
        """Matrix e of a stack of codes, in 64 bits (its scale tiles are whole)."""
        t = m["s"].numel() // E
        return _exact_values(dict(q=m["q"][e * rows:(e + 1) * rows], s=m["s"][e * t:(e + 1) * t],
                                  g=None if m["g"] is None else m["g"][e * rows:(e + 1) * rows]), fmt)

    def rows_of(m, a, b):
        """Rows a to b of expert-major codes (a is a whole number of tiles)."""
        t = 128 * (2 * m["q"].shape[1] // _block(fmt))
        return _exact_values(dict(q=m["q"][a:b], s=m["s"][a // 128 * t:],
                                  g=None if m["g"] is None else m["g"][a:b]), fmt)

    if op == "product":
        y = blank(c["N"])
        for e in range(E):
            if n[e]:
                y[lo[e]:lo[e] + n[e]] = rows_of(s["X"], lo[e], lo[e] + n[e]) @ part(s["W"], e, c["N"]).T
        return {"Y": y}
    d, f = c["d"], c["f"]
    if op == "experts":
        out = {"Y": blank(d)}
        if c["keep"]:
            out.update(A=blank(f), U=blank(f), H=blank(f))
        for e in range(E):
            if not n[e]:
                continue
            at = slice(lo[e], lo[e] + n[e])
            x = _exact_hat(s["x"][s["perm_token"][at].long()], fmt)
            a, u = x @ part(s["W_g"], e, f).T, x @ part(s["W_u"], e, f).T
            h = a * torch.special.expit(a) * u
            out["Y"][at] = _exact_hat(h.to(torch.bfloat16), fmt) @ part(s["W_d"], e, d).T
            if c["keep"]:
                out["A"][at], out["U"][at], out["H"][at] = a, u, h
        return out
    out = {"dX": blank(d), "dA": blank(f), "dU": blank(f)}
    for e in range(E):
        if not n[e]:
            continue
        at = slice(lo[e], lo[e] + n[e])
        r = _exact_hat(s["dY"][at], fmt) @ part(s["W_d"], e, f).T
        a, u = s["A"][at].double(), s["U"][at].double()
        p = torch.special.expit(a)
        out["dA"][at], out["dU"][at] = r * u * (p + a * p * (1 - p)), r * a * p
        both = torch.cat([out["dA"][at], out["dU"][at]], 1).to(torch.bfloat16)
        out["dX"][at] = _exact_hat(both, fmt) @ part(s["W_gu"], e, d).T
    return out
