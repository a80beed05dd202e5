"""Microscaled 4-bit operands without a GPU: the oracle's codes and scales against the formats' lists of
numbers, and the refusals of the entry points and of their bindings (on the host, before any device
work)."""
import math
import os
import shutil
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from pretraining_sigmoid_softmax_gb300 import _lib, build, layer, ops

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not installed")
P = 4096       # a stand-in device address (never dereferenced on the host), 16-byte aligned
BAD = P + 2    # not 16-byte aligned
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
MX, NV = ops.FP4_MX, ops.FP4_NV


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return _lib.load()


# ------------------------------------------------------------------ the oracle's definition

GRID = [Fraction(v) for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]
E4M3 = sorted({Fraction(m * 2 ** max(e, 1), 8) * Fraction(2) ** (-7) if e == 0 else
               Fraction(8 + m, 8) * Fraction(2) ** (e - 7) for e in range(16) for m in range(8)
               if not (e == 15 and m == 7)})


def nearest(v, grid):
    """Index of the nearest of a sorted list; a tie goes to the even index."""
    best = min(range(len(grid)), key=lambda i: (abs(grid[i] - v), i % 2))
    return best


def rows_in(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.pow(2.0, torch.randint(-20, 20, (rows, 1), generator=g).float())
    x[:, ::37] *= 30
    x[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0])
    x[1] = 0
    return x.to(torch.bfloat16).double().numpy()


def test_e4m3_list_is_the_types():
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert [float(e) for e in E4M3] == sorted(set(v.tolist()))


@pytest.mark.parametrize("nv", [False, True])
def test_oracle_codes_are_the_nearest_numbers(nv):
    """Every scale and code by exact fractions: the scale as the format defines it, the code the nearest
    number of the list (ties to the even code)."""
    X = rows_in(6, 128, 3)
    code, S, g = O.quantize_rows_fp4(X, nv)
    b = 16 if nv else 32
    for r in range(X.shape[0]):
        row = [Fraction(v) for v in X[r]]
        top = max(abs(v) for v in row)
        if nv and top > 0:
            want = Fraction(2) ** -126
            while top > 2688 * want:
                want *= 2
            assert Fraction(g[r]) == want and (top <= 2688 * want and top > 1344 * want)
        for j in range(len(row) // b):
            block = row[j * b:(j + 1) * b]
            amax = max(abs(v) for v in block)
            if nv:
                s = E4M3[nearest(amax / Fraction(g[r]) / 6, E4M3)]
            elif amax == 0:
                s = Fraction(2) ** -127
            else:
                s = Fraction(2) ** (math.frexp(float(amax))[1] - 3)
            assert Fraction(S[r, j]) == s
            for i, v in enumerate(block):
                c = int(code[r, j * b + i])
                if s == 0:
                    assert c == 0
                    continue
                assert (c & 7) == nearest(abs(v) / (s * Fraction(g[r])), GRID)
                assert (c >= 8) == (math.copysign(1.0, X[r, j * b + i]) < 0)


@pytest.mark.parametrize("nv", [False, True])
def test_oracle_numbers_are_within_a_step_of_the_input(nv):
    """MX scales saturate by up to a quarter (amax below 8 scales, 6 representable), NV ones by the
    scale's own rounding (1/16); below that a number is off by at most half of the widest gap, 1."""
    X = rows_in(8, 256, 5)[2:]
    Y = O.fp4_dequant_rows(X, nv)
    b = 16 if nv else 32
    amax = np.repeat(np.abs(X).reshape(X.shape[0], -1, b).max(-1), b, axis=1)
    code, S, g = O.quantize_rows_fp4(X, nv)
    full = np.repeat(S * g[:, None], b, axis=1)
    ok = np.abs(Y - X) <= np.maximum(full, np.abs(X) / 4 if not nv else 0.0626 * amax)
    assert ok[full > 0].all()
    assert np.array_equal(O.fp4_dequant_cols(X.T, nv), Y.T)


# ------------------------------------------------------------------------- entry points

@needs_nvcc
def test_scale_bytes(lib):
    assert ops.moe_fp4_scale_bytes(1, 128, MX) == 512
    assert ops.moe_fp4_scale_bytes(128, 256, NV) == 128 * 16
    assert ops.moe_fp4_scale_bytes(129, 256, NV) == 256 * 16
    for bad in ((0, 128, MX), (1, 64, MX), (1, 128, 2), (-1, 128, NV)):
        assert ops.moe_fp4_scale_bytes(*bad) == 0


@needs_nvcc
def test_quantisation_refusals(lib):
    def rows(X=P, X1=None, n=4, cols=256, fmt=MX, q=P, s=P, g=None):
        return lib.moe_quantize_rows_fp4(X, X1, None, n, cols, fmt, q, s, g, None)
    assert {rows(X=None), rows(q=None), rows(s=None), rows(fmt=2), rows(fmt=-1)} == {INVALID}
    assert rows(g=P) == rows(fmt=NV) == INVALID                # powers of two: NV has them, MX has none
    assert rows(n=0) == rows(cols=0) == rows(n=-5) == INVALID
    assert rows(cols=192) == rows(cols=32896) == rows(X1=P, cols=16512) == UNSUPPORTED
    assert {rows(X=BAD), rows(X1=BAD), rows(q=BAD), rows(s=BAD), rows(fmt=NV, g=P + 1)} == {INVALID}

    def cols(X0=P, X1=None, E=2, K0=256, N=128, fmt=NV, q=P, s=P, g=P):
        return lib.moe_quantize_cols_fp4(X0, X1, E, K0, N, fmt, q, s, g, None)
    assert {cols(X0=None), cols(q=None), cols(s=None), cols(g=None), cols(fmt=MX), cols(fmt=7)} == {INVALID}
    assert cols(E=0) == cols(K0=0) == cols(N=0) == INVALID
    assert cols(K0=192) == cols(N=64) == cols(E=65536) == cols(N=32896) == UNSUPPORTED
    assert {cols(X0=BAD), cols(X1=BAD), cols(q=BAD), cols(s=BAD), cols(g=P + 2)} == {INVALID}

    def deq(q=P, s=P, g=None, n=4, cols=128, fmt=MX, out=P):
        return lib.moe_dequantize_fp4(q, s, g, None, n, cols, fmt, out, None)
    assert {deq(q=None), deq(s=None), deq(out=None), deq(g=P), deq(fmt=NV), deq(fmt=3)} == {INVALID}
    assert deq(n=0) == deq(cols=0) == INVALID and deq(cols=130) == UNSUPPORTED
    assert {deq(q=BAD), deq(s=BAD), deq(out=BAD)} == {INVALID}

    def perm(xq=P, sx=P, gx=None, s2r=P, tok=P, ro=P, T=4, R=512, d=128, E=4, k=2, fmt=MX, X=P, sX=P, gX=None):
        return lib.moe_permute_fp4(xq, sx, gx, s2r, tok, ro, T, R, d, E, k, fmt, X, sX, gX, None)
    assert {perm(xq=None), perm(sx=None), perm(s2r=None), perm(tok=None), perm(ro=None), perm(X=None),
            perm(sX=None), perm(gx=P), perm(gX=P), perm(fmt=NV, gx=P), perm(fmt=9)} == {INVALID}
    assert perm(T=0) == perm(R=0) == perm(E=0) == perm(k=0) == perm(d=0) == INVALID
    assert perm(E=257) == perm(k=5) == perm(d=160) == perm(E=64, k=33) == perm(R=1 << 31) == UNSUPPORTED
    assert {perm(xq=BAD), perm(sx=BAD), perm(X=BAD), perm(sX=BAD)} == {INVALID}


@needs_nvcc
def test_product_and_expert_refusals(lib):
    def gemm(x=P, sx=P, gx=None, ro=P, E=4, rows=512, K=256, N=128, w=P, sw=P, gw=None, fmt=MX, Y=P):
        return lib.moe_grouped_gemm_fp4(x, sx, gx, ro, E, rows, K, N, w, sw, gw, fmt, Y, None)
    assert {gemm(x=None), gemm(sx=None), gemm(w=None), gemm(sw=None), gemm(Y=None), gemm(gx=P), gemm(gw=P),
            gemm(fmt=NV), gemm(fmt=NV, gx=P), gemm(fmt=2)} == {INVALID}
    assert gemm(ro=None) == gemm(E=0) == gemm(rows=0) == INVALID   # no layout for four experts
    assert gemm(E=257) == gemm(K=192) == gemm(N=200) == gemm(K=0) == UNSUPPORTED
    assert gemm(rows=1 << 31) == gemm(E=256, N=1 << 24) == UNSUPPORTED  # counted in 32 bits
    assert {gemm(x=BAD), gemm(sx=BAD), gemm(w=BAD), gemm(sw=BAD), gemm(Y=BAD),
            gemm(fmt=NV, gx=BAD, gw=P)} == {INVALID}

    def fwd(fmt=MX, g=None, ro=P, E=4, rows=512, d=256, f=128, A=P, U=P, H=P, hq=P, Y=P, w=P):
        return lib.moe_expert_fwd_fp4(P, P, g, ro, E, rows, d, f, w, P, g, P, P, g, P, P, g, fmt, A, U, H, hq,
                                      P, g, Y, None, None)
    assert {fwd(w=None), fwd(A=None), fwd(U=None), fwd(H=None), fwd(hq=None), fwd(Y=None), fwd(g=P),
            fwd(fmt=NV), fwd(fmt=5)} == {INVALID}
    assert fwd(ro=None) == fwd(E=0) == fwd(rows=0) == INVALID
    assert fwd(E=257) == fwd(d=130) == fwd(f=64) == fwd(f=32896) == fwd(rows=1 << 31) == UNSUPPORTED
    assert {fwd(A=BAD), fwd(U=BAD), fwd(H=BAD), fwd(Y=BAD), fwd(hq=BAD), fwd(w=BAD)} == {INVALID}

    def bwd(parts=7, fmt=MX, dyq=P, dY=P, A=P, H=P, ro=P, E=4, rows=512, d=256, f=128, wd=P, wgu=P, dX=P, dA=P,
            auq=P, dw=P, dl=None, W_r=None, ws=P, wb=1 << 20):
        return lib.moe_expert_bwd_fp4(dyq, P, None, dY, P, A, P, H, ro, E, rows, d, f, wd, P, None, wgu, P,
                                      None, fmt, dX, dA, P, auq, P, None, dw, P, P, parts, dl, W_r, ws, wb,
                                      None)
    assert {bwd(dyq=None), bwd(dY=None), bwd(A=None), bwd(H=None), bwd(wd=None), bwd(wgu=None),
            bwd(dX=None), bwd(dA=None), bwd(auq=None), bwd(dw=None), bwd(fmt=NV)} == {INVALID}
    assert bwd(parts=0) == bwd(parts=8) == bwd(dl=P) == bwd(W_r=P) == INVALID
    assert bwd(dl=P, W_r=BAD) == bwd(dl=P, W_r=P, ro=None, E=1) == INVALID
    assert bwd(f=16512) == bwd(d=192) == bwd(E=257) == UNSUPPORTED
    # what a part does not name may be missing: the next check is the device's
    assert bwd(parts=1, dY=None, H=None, wgu=None, dX=None, auq=None, dw=None, ws=None) == UNSUPPORTED
    assert bwd(parts=2, dyq=None, dY=None, A=None, H=None, wd=None, dw=None, ws=None) == UNSUPPORTED
    assert bwd(parts=4, dyq=None, A=None, wd=None, wgu=None, dX=None, auq=None) == UNSUPPORTED


# ----------------------------------------------------------------------------- bindings

def _operand(*shape, fmt=MX):
    return ops.fp4_empty(shape, fmt, device="cpu")


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@needs_nvcc
def test_bindings_name_what_is_wrong(lib):
    E = ops.MoEError
    with pytest.raises(E, match="no 4-bit operand"):
        _operand(4, 192)
    with pytest.raises(E, match="no 4-bit operand"):
        _operand(0, 128)
    with pytest.raises(E, match="no 4-bit operand"):
        _operand(4, 128, fmt=3)
    m = _operand(4, 256, fmt=NV)
    assert m.q.shape == (4, 128) and m.s.numel() == 128 * 16 and m.g.shape == (4,)
    assert _operand(2, 3, 256).q.shape == (2, 3, 128) and _operand(2, 256).g is None
    for call, match in [
        (lambda: ops.moe_quantize_rows_fp4(None, m), "X must be"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(4, 256), None), "out is missing"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(5, 256), m), "must have shape"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(4, 256), m, X1=_bf(4, 256)), "must have shape"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(4, 256), m._replace(g=None)), "out.g is missing"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(4, 256), m._replace(fmt=MX)), "no powers of two"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(4, 256), m._replace(s=m.s[1:])), "out.s must have shape"),
        (lambda: ops.moe_quantize_rows_fp4(_bf(4, 256), m), "must be a CUDA tensor"),
        (lambda: ops.moe_quantize_cols_fp4(_bf(4, 256), None, m), r"\[E, K0, N\]"),
        (lambda: ops.moe_quantize_cols_fp4(_bf(1, 256, 128), None, None), "out is missing"),
        (lambda: ops.moe_dequantize_fp4(None, _bf(4, 256)), "m is missing"),
        (lambda: ops.moe_dequantize_fp4(m, _bf(4, 128)), "m.q must be a CUDA tensor"),
        (lambda: ops.moe_permute_fp4(None, None, None, None, m), "x is missing"),
        (lambda: ops.moe_permute_fp4(m, torch.zeros(4, 2, dtype=torch.int32), None, None, m), "row_offsets"),
        (lambda: ops.moe_permute_fp4(m, torch.zeros(4, 2, dtype=torch.int32), None,
                                     torch.zeros(5, dtype=torch.int64), m), "the layout takes up to"),
        (lambda: ops.moe_grouped_gemm_fp4(m, None, _operand(2, 128, 256, fmt=NV), _bf(4, 128)),
         "row_offsets is missing"),
        (lambda: ops.moe_grouped_gemm_fp4(m, None, None, _bf(4, 128)), "W is missing"),
        (lambda: ops.moe_grouped_gemm_fp4(m, None, m, _bf(4, 128)), r"\[E, rows, cols / 2\]"),
        (lambda: ops.moe_expert_fwd_fp4(m, None, None, None, None, None, None, None, None, None),
         "W_g is missing"),
        (lambda: ops.moe_expert_bwd_fp4(None, None, None, None, None, None, None, None, None, None, _bf(4, 128),
                                        _bf(4, 128), None, None, None, None, None), "dYc is missing"),
    ]:
        with pytest.raises(E, match=match):
            call()


@needs_nvcc
def test_layer_refusals(lib):
    with pytest.raises(ValueError, match="fp4_format"):
        layer.MoELayer(128, 4, 2, 128, device="cpu", precision="fp4", fp4_format="e2m1")
    with pytest.raises(ValueError, match="precision"):
        layer.MoELayer(128, 4, 2, 128, device="cpu", precision="int4")
    with pytest.raises(ValueError, match="held by a layer"):
        layer.MoELayer(128, 4, 2, 128, device="cpu").hold_weights()
    with pytest.raises(ValueError, match="not both"):
        layer.MoEPlan(layer.MoEShape(64, 128, 4, 2, 128, fp8=True, fp4=True), "cpu")
    block = layer.MoELayer(128, 4, 2, 128, device="cpu", precision="fp4")
    block._held = ()
    with pytest.raises(ValueError, match="held for serving"):
        block(torch.zeros(8, 128, dtype=torch.bfloat16))


def test_configurations_take_the_precision():
    from pretraining_sigmoid_softmax_gb300.configs import C1
    for precision, dgrad in (("fp4", False), ("fp4_dgrad", True)):
        for fmt, code in (("mx", MX), ("nv", NV)):
            s = layer.MoEShape.from_config(C1.with_(precision=precision, fp4_format=fmt))
            assert (s.fp4, s.fp4_dgrad, s.fp4_format, s.fp8) == (True, dgrad, code, False)
