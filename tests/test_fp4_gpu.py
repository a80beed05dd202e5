"""Microscaled 4-bit operands (codes, scales, dispatch), the grouped product and the SwiGLU experts on
them, against the oracle's definition in 64 bits.

Codes and scales are compared bit for bit: every quotient is decided as the exact one is. A product
of the operands is compared with the exact product of the numbers that they stand for: half a bf16
step of it, and (K + 2) 2^-24 of the sum of magnitudes for the fp32 accumulation
(``assert_gemm_exact``)."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from pretraining_sigmoid_softmax_gb300 import ops

from gpu_common import assert_close, assert_gemm_exact, dev, h64, padded_offsets, randn_bf16, require_gpu

pytestmark = pytest.mark.gpu

FMTS = [ops.FP4_MX, ops.FP4_NV]
FILL = 0xEE


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def operand(shape, fmt, fill=FILL):
    m = ops.fp4_empty(shape, fmt)
    m.q.fill_(fill)
    m.s.fill_(fill)
    if m.g is not None:
        m.g.fill_(-7.0)
    return m


def codes_of(m):
    """Codes one a byte, [rows, cols]."""
    q = m.q.reshape(-1, m.q.shape[-1]).cpu().numpy()
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def scale_bytes_of(m):
    """[rows, blocks] scale bytes, each found at its documented place."""
    rows, cols = m.q.numel() // m.q.shape[-1], 2 * m.q.shape[-1]
    b = 16 if m.fmt == ops.FP4_NV else 32
    span = 4 * b
    r, j = np.arange(rows)[:, None], np.arange(cols // b)[None, :]
    at = ((r // 128) * (cols // span) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    return m.s.cpu().numpy()[at], at


def numbers(byte, fmt):
    if fmt == ops.FP4_NV:
        return torch.from_numpy(byte).view(torch.float8_e4m3fn).double().numpy()
    return np.ldexp(1.0, byte.astype(np.int64) - 127)


def check_operand(m, X64, n=None):
    """Rows below n hold the oracle's codes and scales of X64; the others are untouched."""
    nv = m.fmt == ops.FP4_NV
    n = X64.shape[0] if n is None else n
    code, S, g = O.quantize_rows_fp4(X64[:n], nv)
    got = codes_of(m)
    assert np.array_equal(got[:n], code)
    byte, at = scale_bytes_of(m)
    assert np.array_equal(numbers(byte[:n], m.fmt), S)
    raw = m.s.cpu().numpy()
    rest = np.ones(raw.shape, bool)
    rest[at[:n]] = False
    assert (raw[rest] == FILL).all(), "scales of rows that were not given"
    if nv:
        assert np.array_equal(m.g.cpu().numpy()[:n], g)
        assert (m.g[n:] == -7.0).all()
    assert (m.q.reshape(got.shape[0], -1)[n:] == FILL).all()


def rows_in(rows, cols, seed, scale=1.0):
    """Rows of different magnitudes with outliers, ties, zero blocks and a zero row."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * scale
    x *= torch.pow(2.0, torch.randint(-12, 12, (rows, 1), generator=g).float())
    x[:, ::97] *= 64
    x = x.to(torch.bfloat16)
    x[:, 32:64] = 0                                                    # a zero block
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5,
                         -3.5, -5.0, 7.5]).to(torch.bfloat16)
    x[0, 64:80], x[0, 80:96] = grid, grid * 0.5                        # exact midpoints
    if rows > 2:
        x[2] = 0
    return x


SIZES = [(1, 128), (3, 256), (7, 4096), (129, 384), (130, 1024), (1300, 2048), (2500, 128),
         (1230, 4096), (5, 8192), (2, 32768), (3, 8320), (39001, 128), (38999, 384), (39000, 896)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_row_codes_are_bit_exact(rows, cols, fmt):
    x = rows_in(rows, cols, rows + cols)
    m = operand((rows, cols), fmt)
    ops.moe_quantize_rows_fp4(dev(x), m)
    torch.cuda.synchronize()
    check_operand(m, h64(x))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols,n", [(300, 256, 140), (1400, 384, 1290), (9, 4224, 4), (4, 128, 0)])
def test_row_codes_of_two_halves_and_a_limit(rows, cols, n, fmt):
    x0, x1 = rows_in(rows, cols, 1), rows_in(rows, cols, 2, 8.0)
    m = operand((rows, 2 * cols), fmt)
    limit = torch.tensor([n], device="cuda")
    ops.moe_quantize_rows_fp4(dev(x0), m, X1=dev(x1), rows_limit=limit)
    torch.cuda.synchronize()
    check_operand(m, h64(torch.cat([x0, x1], 1)), n)


@pytest.mark.parametrize("fmt", FMTS)
def test_codes_at_the_ends_of_the_range(fmt):
    """Rows of one magnitude each, from bf16's subnormals to its largest numbers, and the magnitudes
    around the border where a row's power of two changes (2688 times a power of two)."""
    g = torch.Generator().manual_seed(5)
    base = torch.randn(40, 256, generator=g).to(torch.bfloat16)
    x = torch.cat([(base[:20].double() * 2.0 ** e).to(torch.bfloat16)[:2] for e in
                   (-130, -126, -120, -110, -60, 0, 60, 110, 120)])
    edge = base[:12].float().clamp(-1, 1).to(torch.bfloat16)
    for i, v in enumerate([2672, 2688, 2704, 1344, 1352, 1336, 448, 6, 5.25, 5.28125, 5.21875, 2 ** 20 * 1.3125]):
        edge[i, 0] = v
    x = torch.cat([x, edge])
    m = operand(tuple(x.shape), fmt)
    ops.moe_quantize_rows_fp4(dev(x), m)
    torch.cuda.synchronize()
    check_operand(m, h64(x))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,K0,N,stack", [(1, 128, 128, False), (3, 256, 384, True), (5, 384, 256, False),
                                          (2, 1024, 128, True), (2, 3456, 128, False),
                                          (1, 1792, 256, True), (1, 1664, 128, True),
                                          (3, 256, 128, False), (2, 640, 128, False),
                                          (1, 768, 384, False)])
def test_column_codes_are_bit_exact(E, K0, N, stack, fmt):
    mats = [torch.stack([rows_in(K0, N, 7 * e + i) for e in range(E)]) for i in range(2 if stack else 1)]
    if E > 1:
        mats[0][1] = 0
    m = operand((E, N, K0 * len(mats)), fmt)
    ops.moe_quantize_cols_fp4(dev(mats[0]), dev(mats[1]) if stack else None, m)
    torch.cuda.synchronize()
    both = torch.cat(mats, 1).transpose(1, 2).reshape(E * N, -1)
    check_operand(m, h64(both))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (333, 640), (4000, 256)])
def test_dequantised_numbers_are_exact(rows, cols, fmt):
    x = rows_in(rows, cols, 3)
    m = operand((rows, cols), fmt)
    ops.moe_quantize_rows_fp4(dev(x), m)
    out = torch.full((rows, cols), -3.0, dtype=torch.bfloat16, device="cuda")
    n = rows - rows // 3
    ops.moe_dequantize_fp4(m, out, rows_limit=torch.tensor([n], device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(h64(out)[:n], O.fp4_dequant_rows(h64(x), fmt == ops.FP4_NV)[:n])
    assert (out[n:] == -3.0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_infinities_and_nan_stay_in_their_block_or_row(fmt):
    x = rows_in(6, 256, 9)
    x[0, 70], x[3, 5], x[5, 200] = float("inf"), float("nan"), -float("inf")
    m = operand((6, 256), fmt)
    ops.moe_quantize_rows_fp4(dev(x), m)
    out = torch.empty(6, 256, dtype=torch.bfloat16, device="cuda")
    ops.moe_dequantize_fp4(m, out)
    torch.cuda.synchronize()
    bad = torch.zeros(6, 256, dtype=torch.bool)
    if fmt == ops.FP4_NV:
        bad[[0, 3, 5]] = True
    else:
        bad[0, 64:96], bad[3, 0:32], bad[5, 192:224] = True, True, True
    assert torch.equal(out.cpu().isnan(), bad)
    clean = x.clone()
    clean[bad] = 0
    want = O.fp4_dequant_rows(h64(clean), fmt == ops.FP4_NV)
    assert np.array_equal(h64(out)[~bad.numpy()], want[~bad.numpy()])


def _routing(T, E, k, g, skew):
    w = torch.tensor([1.0 / (1 + i) ** (1.5 if skew else 0.0) for i in range(E)])
    return torch.stack([torch.multinomial(w, k, generator=g) for _ in range(T)]).to(torch.int32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,d,E,k,skew", [(1000, 256, 8, 2, False), (777, 512, 16, 4, True),
                                          (5, 128, 16, 4, True), (1, 1152, 4, 1, False)])
def test_permuted_codes_equal_quantised_permuted_rows(T, d, E, k, skew, fmt):
    g = torch.Generator().manual_seed(T)
    x = rows_in(T, d, T)
    idx = dev(_routing(T, E, k, g, skew))
    R = ops.moe_padded_rows(T, k, E)
    i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
    counts, off, ro = torch.empty(E, **i32), torch.empty(E + 1, **i64), torch.empty(E + 1, **i64)
    tok, s2r = torch.empty(R, **i32), torch.empty(T, k, **i32)
    Xp = torch.empty(R, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ops.moe_workspace_bytes(T, d, E, k), dtype=torch.uint8, device="cuda")
    ops.moe_permute(idx, dev(x), E, counts, off, ro, tok, s2r, Xp, ws)
    xc, X = operand((T, d), fmt), operand((R, d), fmt)
    ops.moe_quantize_rows_fp4(dev(x), xc)
    ops.moe_permute_fp4(xc, s2r, tok, ro, X)
    torch.cuda.synchronize()
    n = int(ro[-1])
    check_operand(X, h64(torch.cat([Xp[:n].cpu(), torch.zeros(R - n, d, dtype=torch.bfloat16)])), n)


def layout(counts, extra=128):
    """Offsets (or None), capacity, and the rows of each expert."""
    if isinstance(counts, int):
        return None, counts, [(0, counts)]
    ro = padded_offsets(counts)
    return ro, int(ro[-1]) + extra, [(int(ro[e]), int(ro[e]) + c) for e, c in enumerate(counts)]


def made(t, fmt, limit=None):
    m = ops.fp4_empty(tuple(t.shape), fmt)
    ops.moe_quantize_rows_fp4(dev(t.reshape(-1, t.shape[-1])),
                              ops.Fp4(m.q.view(-1, m.q.shape[-1]), m.s, m.g, fmt), rows_limit=limit)
    return m


COUNTS = [1, 600, [300, 0, 129, 1, 513], [0, 0, 128], [1, 1, 1, 127, 256]]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K,N", [(128, 128), (256, 256), (384, 640), (1152, 512), (2048, 256)])
@pytest.mark.parametrize("counts", COUNTS)
def test_product_matches_the_exact_one(counts, K, N, fmt):
    g = torch.Generator().manual_seed(K + N)
    ro, rows, segs = layout(counts)
    E = len(segs)
    X = torch.zeros(rows, K, dtype=torch.bfloat16)
    for lo, hi in segs:
        X[lo:hi] = rows_in(hi - lo, K, lo) if hi - lo > 2 else randn_bf16((hi - lo, K), g)
    W = randn_bf16((E, N, K), g, K ** -0.5)
    ro_d = None if ro is None else dev(torch.from_numpy(ro))
    Xm, Wm = made(X, fmt, None if ro is None else ro_d[E:]), made(W, fmt)
    if ro is not None:  # codes and scales past the layout are garbage, and stay out of the sums
        n = int(ro[-1])
        Xm.q[n:], Xm.s[n * K // (16 if fmt == ops.FP4_NV else 32):] = 0x77, 0x7F
    Y = torch.full((rows, N), -3.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(Xm, ro_d, Wm, Y)
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)
    nv = fmt == ops.FP4_NV
    for e, (lo, hi) in enumerate(segs):
        if hi > lo:
            assert_gemm_exact(Y[lo:hi], O.fp4_dequant_rows(h64(X[lo:hi]), nv),
                              O.fp4_dequant_rows(h64(W[e]), nv).T, f"e{e}")
        if ro is not None:
            assert (Y[hi:int(ro[e + 1])] == 0).all()
    if ro is not None:
        assert (Y[int(ro[-1]):] == -3.0).all()


def _expert_inputs(counts, d, f, seed):
    g = torch.Generator().manual_seed(seed)
    ro, rows, segs = layout(counts)
    E = len(segs)
    t = {n: torch.zeros(rows, c, dtype=torch.bfloat16) for n, c in
         (("X", d), ("dY", d), ("A", f), ("U", f), ("H", f))}
    for lo, hi in segs:
        for n, std in (("X", 1.0), ("dY", 0.3), ("A", 1.0), ("U", 1.0), ("H", 0.5)):
            t[n][lo:hi] = randn_bf16((hi - lo, t[n].shape[1]), g, std)
    W = dict(W_g=randn_bf16((E, f, d), g, d ** -0.5), W_u=randn_bf16((E, f, d), g, d ** -0.5),
             W_d=randn_bf16((E, d, f), g, f ** -0.5))
    return t, W, ro, rows, segs


EXPERTS = [(1, 256, 128), (600, 512, 256), ([300, 0, 129, 1, 513], 512, 256), ([130, 5, 0], 384, 128),
           ([1, 0, 1], 256, 384)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("keep,gates", [(True, False), (False, False), (True, True)])
@pytest.mark.parametrize("counts,d,f", EXPERTS)
def test_expert_forward_matches_the_definition(counts, d, f, keep, gates, fmt):
    """a and u as exact products of the operands; h against silu(a) u of the exact a and u; the operand
    of H as the oracle's of the stored H; y as the exact product of that operand."""
    t, W, ro, rows, segs = _expert_inputs(counts, d, f, d + f)
    nv = fmt == ops.FP4_NV
    ro_d = None if ro is None else dev(torch.from_numpy(ro))
    n = rows if ro is None else int(ro[-1])
    X = made(t["X"], fmt, None if ro is None else ro_d[len(segs):])
    new = lambda c: torch.full((rows, c), -3.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    A, U = (new(f), new(f)) if keep else (None, None)
    H, Y, Hc = new(f), new(d), operand((rows, f), fmt)
    rg = None
    if gates:
        rg = torch.rand(rows, generator=torch.Generator().manual_seed(1)) + 0.5
    ops.moe_expert_fwd_fp4(X, ro_d, made(W["W_g"], fmt), made(W["W_u"], fmt), made(W["W_d"], fmt), A, U, H,
                           Hc, Y, row_gate=None if rg is None else dev(rg))
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)
    check_operand(Hc, h64(H), n)
    for e, (lo, hi) in enumerate(segs):
        if hi == lo:
            continue
        x = O.fp4_dequant_rows(h64(t["X"][lo:hi]), nv)
        wg, wu, wd = (O.fp4_dequant_rows(h64(W[k][e]), nv) for k in ("W_g", "W_u", "W_d"))
        if keep:
            assert_gemm_exact(A[lo:hi], x, wg.T, f"A e{e}")
            assert_gemm_exact(U[lo:hi], x, wu.T, f"U e{e}")
        a, u = x @ wg.T, x @ wu.T
        h = a / (1 + np.exp(-a)) * u * (1.0 if rg is None else h64(rg)[lo:hi, None])
        assert_close(H[lo:hi], h, f"H e{e}", atol=1e-5, rtol=2.0 ** -8 + 1e-5)
        assert_gemm_exact(Y[lo:hi], O.fp4_dequant_rows(h64(H[lo:hi]), nv), wd.T, f"Y e{e}")
    for o in (A, U, H, Y):
        assert o is None or (o[n:] == -3.0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,d,f", EXPERTS)
@pytest.mark.parametrize("router", [False, True])
def test_expert_backward_matches_the_definition(counts, d, f, router, fmt):
    """da and du against the SwiGLU backward of the exact product; the operand of [dA | dU] as the
    oracle's of the stored ones; dX as the exact product of that operand (plus the router's term);
    the weight gradients as exact products of the bf16 tensors."""
    if router and isinstance(counts, int):
        pytest.skip("the router term needs the routed layout")
    t, W, ro, rows, segs = _expert_inputs(counts, d, f, d + f + 1)
    nv, E = fmt == ops.FP4_NV, len(segs)
    ro_d = None if ro is None else dev(torch.from_numpy(ro))
    n = rows if ro is None else int(ro[-1])
    Wd, Wgu = ops.fp4_empty((E, f, d), fmt), ops.fp4_empty((E, d, 2 * f), fmt)
    ops.moe_quantize_cols_fp4(dev(W["W_d"]), None, Wd)
    ops.moe_quantize_cols_fp4(dev(W["W_g"]), dev(W["W_u"]), Wgu)
    new = lambda *c: torch.full(c, -3.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dA, dU, dX = new(rows, f), new(rows, f), new(rows, d)
    dWg, dWu, dWd = new(E, f, d), new(E, f, d), new(E, d, f)
    AUc = operand((rows, 2 * f), fmt)
    dl = torch.randn(rows, generator=torch.Generator().manual_seed(2))
    W_r = torch.randn(E, d, generator=torch.Generator().manual_seed(3))
    ws = torch.empty(ops.moe_workspace_bytes(rows, d, E, 1), dtype=torch.uint8, device="cuda")
    dYc = made(t["dY"], fmt, None if ro is None else ro_d[E:])
    args = (dYc, dev(t["dY"]), dev(t["X"]), dev(t["A"]), dev(t["U"]), dev(t["H"]), ro_d, Wd, Wgu, dX, dA, dU,
            AUc, dWg, dWu, dWd, ws)
    kw = dict(dl_rows=dev(dl), W_r=dev(W_r)) if router else {}
    if router:  # in two calls, as the layer needs the gates' gradient between them
        ops.moe_expert_bwd_fp4(*args, parts=ops.BWD_DH)
        ops.moe_expert_bwd_fp4(*args, parts=ops.BWD_DX | ops.BWD_W, **kw)
    else:
        ops.moe_expert_bwd_fp4(*args)
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)
    check_operand(AUc, np.concatenate([h64(dA), h64(dU)], 1), n)
    for e, (lo, hi) in enumerate(segs):
        if hi == lo:
            assert not any(w[e].any() for w in (dWg, dWu, dWd))
            continue
        x, dy, a, u, h = (h64(t[k][lo:hi]) for k in ("X", "dY", "A", "U", "H"))
        wg, wu, wd = (h64(W[k][e]) for k in ("W_g", "W_u", "W_d"))
        r = O.fp4_dequant_rows(dy, nv) @ O.fp4_dequant_cols(wd, nv)
        da, du = O.swiglu_backward(r, a, u)
        assert_close(dA[lo:hi], da, f"dA e{e}", atol=1e-5, rtol=2.0 ** -8 + 1e-5)
        assert_close(dU[lo:hi], du, f"dU e{e}", atol=1e-5, rtol=2.0 ** -8 + 1e-5)
        AU = O.fp4_dequant_rows(np.concatenate([h64(dA[lo:hi]), h64(dU[lo:hi])], 1), nv)
        Wb = O.fp4_dequant_cols(np.concatenate([wg, wu]), nv)
        if router:  # one more exact column: the slot's logit gradient times the router row
            AU, Wb = np.concatenate([AU, h64(dl)[lo:hi, None]], 1), np.concatenate([Wb, h64(W_r)[e][None]])
        assert_gemm_exact(dX[lo:hi], AU, Wb, f"dX e{e}")
        assert_gemm_exact(dWd[e], dy.T, h, f"dW_d e{e}")
        assert_gemm_exact(dWg[e], h64(dA[lo:hi]).T, x, f"dW_g e{e}")
        assert_gemm_exact(dWu[e], h64(dU[lo:hi]).T, x, f"dW_u e{e}")
    for o in (dA, dU, dX):
        assert (o[n:] == -3.0).all()


# ------------------------------------------------------------------ at the edges of the calls

def _random_operand(shape, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    return made(t, fmt)


def numbers_of(m):
    """[..., rows, cols] in fp64 on the GPU."""
    out = torch.empty((*m.q.shape[:-1], 2 * m.q.shape[-1]), dtype=torch.bfloat16, device="cuda")
    ops.moe_dequantize_fp4(m, out)
    return out.double()


def check_product(Y, X, W, segs):
    """assert_gemm_exact's bound, on the GPU."""
    for e, (lo, hi) in enumerate(segs):
        a, w = numbers_of(X)[lo:hi], numbers_of(W)[e]
        ex, mag = a @ w.t(), a.abs() @ w.abs().t()
        _, p = torch.frexp(ex.abs())
        ulp = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), p.double() - 8)
        off = (Y[lo:hi].double() - ex).abs() - 0.5001 * ulp - (a.shape[1] + 2) * 2.0 ** -24 * mag
        assert (off <= 0).all(), (e, float(off.max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,K,N", [([9000, 3, 0, 4100, 128, 7777], 2048, 1024), (20000, 1536, 2048),
                                        ([130] * 40, 640, 384), ([64] * 64, 4096, 512)])
def test_products_that_use_every_stage_and_buffer_again(counts, K, N, fmt):
    """More tiles than the GPU takes at once, long and short sums, whole and clipped tiles; two runs give
    the same bits."""
    ro, rows, segs = layout(counts)
    ro_d = None if ro is None else dev(torch.from_numpy(ro))
    X, W = _random_operand((rows, K), fmt, 1), _random_operand((len(segs), N, K), fmt, 2)
    Y = torch.full((rows, N), -3.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(X, ro_d, W, Y)
    again = torch.empty_like(Y)
    ops.moe_grouped_gemm_fp4(X, ro_d, W, again)
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)
    n = rows if ro is None else int(ro[-1])
    assert torch.equal(Y[:n], again[:n])
    check_product(Y, X, W, segs)


@pytest.mark.parametrize("fmt", FMTS)
def test_no_rows_at_all(fmt):
    """Experts that are all empty: nothing is written."""
    ro, rows, _ = layout([0, 0, 0])
    X, W = _random_operand((rows, 256), fmt, 1), _random_operand((3, 128, 256), fmt, 2)
    Y = torch.full((rows, 128), -3.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(X, dev(torch.from_numpy(ro)), W, Y)
    torch.cuda.synchronize()
    assert (Y == -3.0).all() and ops.moe_device_status() == (0, 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [100, 700])
def test_infinities_and_nan_stay_in_their_rows_and_columns(rows, fmt):
    """A row of X that holds one makes its row of Y NaN (its block's or its row's scale is NaN), a row of W
    its column; nothing else."""
    g = torch.Generator().manual_seed(4)
    x, w = randn_bf16((rows, 512), g), randn_bf16((1, 384, 512), g)
    x[3, 40], x[rows - 1, 511], w[0, 7, 0], w[0, 300, 130] = float("inf"), float("nan"), float("nan"), -float("inf")
    Y = torch.empty(rows, 384, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(made(x, fmt), None, made(w, fmt), Y)
    torch.cuda.synchronize()
    want = torch.zeros(rows, 384, dtype=torch.bool)
    want[[3, rows - 1]] = True
    want[:, [7, 300]] = True
    assert torch.equal(Y.isnan().cpu(), want)
    x[[3, rows - 1]] = 0
    w[0, [7, 300]] = 0
    nv, ok = fmt == ops.FP4_NV, ~want.numpy()
    ex = O.fp4_dequant_rows(h64(x), nv) @ O.fp4_dequant_rows(h64(w[0]), nv).T
    assert (np.abs(h64(Y) - ex)[ok] <= (2.0 ** -8 * np.abs(ex) + 1e-3)[ok]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [[0, 128, 100, 384], [0, 100, 256, 384], [128, 256, 384, 384],
                                 [0, 128, 256, 4096]])
def test_layouts_that_are_none_are_reported(bad, fmt):
    """A decrease, a segment that is no whole number of tiles, a start other than 0, an end past the
    capacity: the kernels record it and write nothing."""
    X, W = _random_operand((512, 256), fmt, 1), _random_operand((3, 256, 256), fmt, 2)
    ro = torch.tensor(bad, device="cuda")
    Y = torch.full((512, 256), -3.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_clear_device_status()
    ops.moe_grouped_gemm_fp4(X, ro, W, Y)
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (5, 20) and (Y == -3.0).all()
    ops.moe_clear_device_status()


@pytest.mark.parametrize("fmt", FMTS)
def test_dispatch_reports_rows_past_the_capacity(fmt):
    R = ops.moe_padded_rows(4, 2, 2)
    x, X = operand((4, 128), fmt, 0x11), operand((R, 128), fmt)
    s2r = torch.tensor([[0, 128], [1, R], [2, -1], [3, 129]], dtype=torch.int32, device="cuda")
    tok = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    tok[[0, 1, 2, 3, 128, 129]] = torch.tensor([0, 1, 2, 3, 0, 3], dtype=torch.int32, device="cuda")
    for ro, rest in (([0, 128, 256], 0), ([0, 128, R + 128], FILL)):
        ops.moe_clear_device_status()
        for t in (X.q, X.s):
            t.fill_(FILL)
        ops.moe_permute_fp4(x, s2r, tok, torch.tensor(ro, device="cuda"), X)
        torch.cuda.synchronize()
        assert ops.moe_device_status() == (5, 21)
        q = X.q.cpu()
        for r in (0, 1, 2, 3, 128, 129):
            assert (q[r] == 0x11).all(), r
        assert (q[4:128] == 0).all() and (q[130:256] == rest).all() and (q[256:] == FILL).all()
    ops.moe_clear_device_status()


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_calls_replay_on_new_inputs_and_streams(fmt):
    """Quantisation, dispatch and experts recorded once and replayed with other tokens, beside the same on
    another stream."""
    T, d, f, E, k = 70, 256, 256, 8, 2
    g = torch.Generator().manual_seed(1)
    idx = dev(_routing(T, E, k, g, False))
    R = ops.moe_padded_rows(T, k, E)
    i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
    counts, off, ro = torch.empty(E, **i32), torch.empty(E + 1, **i64), torch.empty(E + 1, **i64)
    tok, s2r = torch.empty(R, **i32), torch.empty(T, k, **i32)
    ws = torch.empty(ops.moe_workspace_bytes(T, d, E, k), dtype=torch.uint8, device="cuda")
    x = dev(randn_bf16((T, d), g))
    ops.moe_permute(idx, x, E, counts, off, ro, tok, s2r, torch.empty(R, d, dtype=torch.bfloat16, device="cuda"),
                    ws)
    W = [_random_operand(s, fmt, i) for i, s in enumerate([(E, f, d), (E, f, d), (E, d, f)])]

    class Buffers:
        def __init__(self):
            z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
            self.x, self.A, self.U, self.H, self.Y = z(T, d), z(R, f), z(R, f), z(R, f), z(R, d)
            self.xc, self.X, self.Hc = (ops.fp4_empty(s, fmt) for s in ((T, d), (R, d), (R, f)))

        def run(self, stream=None):
            ops.moe_quantize_rows_fp4(self.x, self.xc, stream=stream)
            ops.moe_permute_fp4(self.xc, s2r, tok, ro, self.X, stream=stream)
            ops.moe_expert_fwd_fp4(self.X, ro, *W, self.A, self.U, self.H, self.Hc, self.Y, stream=stream)

    a, b, want = Buffers(), Buffers(), Buffers()
    a.x.copy_(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for seed in (5, 6):
        new = dev(randn_bf16((T, d), torch.Generator().manual_seed(seed)))
        a.x.copy_(new)
        b.x.copy_(new.flip(0))
        torch.cuda.synchronize()
        graph.replay()
        b.run(side)
        torch.cuda.synchronize()
        for got in (a, b):
            want.x.copy_(got.x)
            want.run()
            torch.cuda.synchronize()
            n = int(ro[-1])
            for t in ("A", "U", "H", "Y"):
                assert torch.equal(getattr(got, t)[:n], getattr(want, t)[:n]), t
    assert ops.moe_device_status() == (0, 0)


def test_swiglu_gradients_against_differences():
    """dA and dU against central differences of <r, silu(a) u> in 64 bits: the differences are off by
    eps^2 / 6 of the third derivative (below 1 for silu), the kernel's values by half a bf16 step."""
    for fmt in FMTS:
        t, W, ro, rows, segs = _expert_inputs(300, 256, 128, 7)
        Wd, new = ops.fp4_empty((1, 128, 256), fmt), lambda c: torch.empty(rows, c, dtype=torch.bfloat16,
                                                                           device="cuda")
        ops.moe_quantize_cols_fp4(dev(W["W_d"]), None, Wd)
        dA, dU = new(128), new(128)
        ops.moe_expert_bwd_fp4(made(t["dY"], fmt), None, None, dev(t["A"]), dev(t["U"]), None, None, Wd, None, None,
                               dA, dU, None, None, None, None, None, parts=ops.BWD_DH)
        torch.cuda.synchronize()
        nv = fmt == ops.FP4_NV
        r = O.fp4_dequant_rows(h64(t["dY"]), nv) @ O.fp4_dequant_cols(h64(W["W_d"][0]), nv)
        a, u, eps = h64(t["A"]), h64(t["U"]), 1e-4
        f = lambda a, u: r * O.silu(a) * u  # noqa: E731
        for got, dif, third in ((dA, (f(a + eps, u) - f(a - eps, u)) / (2 * eps), np.abs(r * u)),
                                (dU, (f(a, u + eps) - f(a, u - eps)) / (2 * eps), 0.0)):
            bound = 2.0 ** -8 * np.abs(dif) + eps * eps * third + 1e-5 * (1 + np.abs(r) * (1 + np.abs(a * u)))
            assert (np.abs(h64(got) - dif) <= bound).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_more_than_2_to_31_elements(fmt):
    """Offsets past 32 bits: the last rows of a large matrix have the codes and numbers they have alone."""
    rows, cols = 530000, 4096
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(
        generator=torch.Generator(device="cuda").manual_seed(1))
    m = ops.fp4_empty((rows, cols), fmt)
    ops.moe_quantize_rows_fp4(x, m)
    out = torch.empty_like(x)
    ops.moe_dequantize_fp4(m, out)
    for lo in (0, 262144, rows - 384):
        part = x[lo:lo + 384].contiguous()
        small, alone = ops.fp4_empty((384, cols), fmt), torch.empty(384, cols, dtype=torch.bfloat16, device="cuda")
        ops.moe_quantize_rows_fp4(part, small)
        ops.moe_dequantize_fp4(small, alone)
        torch.cuda.synchronize()
        assert torch.equal(m.q[lo:lo + 384], small.q) and torch.equal(out[lo:lo + 384], alone)


def test_refusals_on_the_gpu():
    E = ops.MoEError
    m = ops.fp4_empty((4, 256), ops.FP4_NV)
    buf = torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(E, match="invalid argument"):
        ops.moe_quantize_rows_fp4(buf[1:1 + 1024].view(4, 256), m)       # off 16 bytes
    ops.moe_quantize_rows_fp4(buf[8:].view(4, 256), m)                   # a view on them
    with pytest.raises(E, match="contiguous"):
        ops.moe_quantize_rows_fp4(torch.zeros(256, 4, dtype=torch.bfloat16, device="cuda").t(), m)
    with pytest.raises(E, match="must be torch.bfloat16"):
        ops.moe_quantize_rows_fp4(torch.zeros(4, 256, device="cuda"), m)
    with pytest.raises(E, match="rows_limit must have shape"):
        ops.moe_quantize_rows_fp4(buf[8:].view(4, 256), m, rows_limit=torch.zeros(2, dtype=torch.int64,
                                                                                    device="cuda"))
    with pytest.raises(E, match="format"):
        ops.moe_grouped_gemm_fp4(m, None, ops.fp4_empty((1, 128, 256), ops.FP4_MX),
                                 torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(E, match="unsupported"):
        ops.moe_quantize_rows_fp4(torch.zeros(1, 32896, dtype=torch.bfloat16, device="cuda"),
                                  ops.fp4_empty((1, 32896), ops.FP4_MX))
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)
