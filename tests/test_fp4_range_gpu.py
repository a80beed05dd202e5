"""Products of NV operands at the ends of the powers' range. A row's power of two is 2^-126 to 2^118, so a
row's times a column's can leave fp32's range where the product of the operands does not.

Bound of a product: as in test_fp4_gpu, half a bf16 step of the exact one and (K + 2) 2^-24 of the sum of
magnitudes. The magnitudes are chosen so that results are exact zeros, or normal numbers of bf16."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from pretraining_sigmoid_softmax_gb300 import ops

from gpu_common import assert_close, assert_gemm_exact, dev, h64, padded_offsets, randn_bf16, require_gpu

pytestmark = pytest.mark.gpu

NV = ops.FP4_NV


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def made(t):
    m = ops.fp4_empty(tuple(t.shape), NV)
    ops.moe_quantize_rows_fp4(dev(t.reshape(-1, t.shape[-1])), ops.Fp4(m.q.view(-1, m.q.shape[-1]), m.s, m.g, NV))
    return m


def scaled(t, e):
    """t 2^e, exact in bf16 (e by row)."""
    return (t.double() * 2.0 ** torch.as_tensor(e).double()[..., None]).to(torch.bfloat16)


def numbers(t):
    return O.fp4_dequant_rows(h64(t), True)


# row and column exponents whose sum leaves fp32's normal range, or not, on either side of 1 or on both
@pytest.mark.parametrize("rows,K,N", [(100, 256, 384), (600, 512, 512), (600, 384, 640)])
@pytest.mark.parametrize("ex,ew", [(100, -100), (-100, 100), (120, -64), (-60, 118), (0, 0), (-64, -40),
                                   (60, 40), (118, -125)])
def test_products_within_range_of_powers_out_of_it(ex, ew, rows, K, N):
    g = torch.Generator().manual_seed(K + ex)
    x, w = scaled(randn_bf16((rows, K), g), [ex] * rows), scaled(randn_bf16((N, K), g), [ew] * N)
    Y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(made(x), None, made(w[None]), Y)
    torch.cuda.synchronize()
    X, W = numbers(x), numbers(w)
    assert_gemm_exact(Y, X, W.T, "Y")


@pytest.mark.parametrize("rows", [100, 600])
def test_rows_and_columns_of_every_magnitude(rows):
    """Each row and each column of its own magnitude: results past bf16's range are infinite, those below
    its normal numbers are within one of its least steps (2^-133), and the rest as ever."""
    K, N = 256, 512
    g = torch.Generator().manual_seed(rows)
    er, ec = torch.randint(-110, 115, (rows,), generator=g), torch.randint(-110, 115, (N,), generator=g)
    x, w = scaled(randn_bf16((rows, K), g), er), scaled(randn_bf16((N, K), g), ec)
    Y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(made(x), None, made(w[None]), Y)
    torch.cuda.synchronize()
    X, W, got = numbers(x), numbers(w), h64(Y)
    ex, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    slack = (K + 2) * 2.0 ** -24 * mag
    top = float(torch.finfo(torch.bfloat16).max)
    big = np.abs(ex) - slack > top * (1 + 2.0 ** -8)
    assert big.any() and (np.isinf(got[big]) & (np.sign(got[big]) == np.sign(ex[big]))).all()
    sure = np.abs(ex) + slack < top
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(ex), 1e-300))) - 7, -133)
    assert np.isfinite(got[sure]).all()
    # subnormal: half a least step twice, once in fp32 and once in bf16
    assert (np.abs(got - ex)[sure] <= (0.5001 * step + slack + np.where(step == 2.0 ** -133, 2.0 ** -149, 0))[sure]).all()


def test_sums_of_exact_zeros_stay_zero():
    """Rows of 2^100 that meet columns of 2^100 in zeros only: 0, not infinity times 0."""
    rows, K, N = 300, 256, 256
    g = torch.Generator().manual_seed(3)
    x, w = scaled(randn_bf16((rows, K), g), [100] * rows), scaled(randn_bf16((N, K), g), [100] * N)
    x[:, 128:], w[:, :128] = 0, 0
    x[0], w[1] = 0, 0
    Y = torch.full((rows, N), -3.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(made(x), None, made(w[None]), Y)
    torch.cuda.synchronize()
    assert (Y == 0).all()


@pytest.mark.parametrize("rows,N", [(100, 256), (600, 256), (600, 384)])
def test_large_sums_under_small_powers(rows, N):
    """Rows of one number: every product of codes is of the same sign and the largest there is, so that a
    sum reaches 2^30 under powers of 2^-102 and 2^-49, whose product is 0 in fp32."""
    K = 256
    x = torch.full((rows, K), 1.3125 * 2.0 ** -91, dtype=torch.bfloat16)
    w = torch.full((1, N, K), 1.3125 * 2.0 ** -38, dtype=torch.bfloat16)
    Y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_gemm_fp4(made(x), None, made(w), Y)
    torch.cuda.synchronize()
    X, W = numbers(x), numbers(w[0])
    assert (X @ W.T > 2.0 ** -122).all()
    assert_gemm_exact(Y, X, W.T, "Y")


@pytest.mark.parametrize("counts", [[3, 0, 200], [700, 130]])
def test_experts_between_powers_out_of_range(counts):
    """The forward and dA and dU, with rows of 2^100 and weights of 2^-100 in every other expert, and the
    other way round in the rest."""
    d, f, E = 256, 128, len(counts)
    ro = padded_offsets(counts)
    rows, ro_d = int(ro[-1]), dev(torch.from_numpy(ro))
    g = torch.Generator().manual_seed(sum(counts))
    sign = [100 if e % 2 else -100 for e in range(E)]
    X, dY = torch.zeros(rows, d, dtype=torch.bfloat16), torch.zeros(rows, d, dtype=torch.bfloat16)
    A, U = torch.zeros(rows, f, dtype=torch.bfloat16), torch.zeros(rows, f, dtype=torch.bfloat16)
    segs = [(int(ro[e]), int(ro[e]) + c) for e, c in enumerate(counts)]
    for (lo, hi), s in zip(segs, sign):
        X[lo:hi] = scaled(randn_bf16((hi - lo, d), g), [s] * (hi - lo))
        dY[lo:hi] = scaled(randn_bf16((hi - lo, d), g), [s] * (hi - lo))
        A[lo:hi], U[lo:hi] = randn_bf16((hi - lo, f), g), randn_bf16((hi - lo, f), g)
    W = {n: torch.stack([scaled(randn_bf16((a, d), g, d ** -0.5), [-s] * a) for s in sign])
         for n, a in (("W_g", f), ("W_u", f), ("W_dT", f))}
    Wd_fwd = randn_bf16((E, d, f), g, f ** -0.5)
    Xm, Hc = made(X), ops.fp4_empty((rows, f), NV)
    new = lambda c: torch.empty(rows, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Ak, Uk, H, Y, dA, dU = new(f), new(f), new(f), new(d), new(f), new(f)
    ops.moe_expert_fwd_fp4(Xm, ro_d, made(W["W_g"]), made(W["W_u"]), made(Wd_fwd), Ak, Uk, H, Hc, Y)
    ops.moe_expert_bwd_fp4(made(dY), None, None, dev(A), dev(U), None, ro_d, made(W["W_dT"]), None, None, dA, dU,
                           None, None, None, None, None, parts=ops.BWD_DH)
    torch.cuda.synchronize()
    for e, (lo, hi) in enumerate(segs):
        if lo == hi:
            continue
        x, wg, wu, wd = numbers(X[lo:hi]), numbers(W["W_g"][e]), numbers(W["W_u"][e]), numbers(W["W_dT"][e])
        assert_gemm_exact(Ak[lo:hi], x, wg.T, f"A e{e}")
        assert_gemm_exact(Uk[lo:hi], x, wu.T, f"U e{e}")
        a, u = x @ wg.T, x @ wu.T
        assert_close(H[lo:hi], a / (1 + np.exp(-a)) * u, f"H e{e}", atol=1e-5, rtol=2.0 ** -8 + 1e-5)
        r = numbers(dY[lo:hi]) @ wd.T
        da, du = O.swiglu_backward(r, h64(A[lo:hi]), h64(U[lo:hi]))
        assert_close(dA[lo:hi], da, f"dA e{e}", atol=1e-5, rtol=2.0 ** -8 + 1e-5)
        assert_close(dU[lo:hi], du, f"dU e{e}", atol=1e-5, rtol=2.0 ** -8 + 1e-5)
