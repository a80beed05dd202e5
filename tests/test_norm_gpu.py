"""The residual addition with the RMS norm (and the FP8 experts' codes), and its backward, against
a plain implementation in 64 bits.

Bounds. u = 2^-24. A kernel sums a row's d terms as chains of at most 32 in a thread, a butterfly
of 5 and at most 32 warps in order: no sum's terms pass more than 69 roundings, and each product
adds one; 80 u bounds the relative error of a sum of squares and, times the sum of magnitudes,
that of the dot product. A stored value is off by half a step of its type more (bf16: 2^-8,
E4M3: 2^-4 of a normal value or 2^-10 of the scale)."""
import numpy as np
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
SUM = 80 * U


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def n64(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, d, rdtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) * scale).to(torch.bfloat16).cuda()
    r = (2 * scale * torch.randn(T, d, generator=g)).to(rdtype).cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    return x, r, w


def _forward(x, r, w, eps=1e-6, codes=True, y=True):
    T, d = x.shape
    o = dict(z=None if r is None else torch.empty_like(r), y=torch.empty_like(x) if y else None,
             rstd=torch.empty(T, device="cuda"), yq=None, sy=None)
    if codes:
        o.update(yq=torch.empty(T, d, dtype=torch.uint8, device="cuda"),
                 sy=torch.empty(T, device="cuda"))
    ops.moe_rms_norm(x, r, w, eps, o["z"], o["y"], o["yq"], o["sy"], o["rstd"])
    torch.cuda.synchronize()
    return o


def _check_forward(x, r, w, o, eps=1e-6):
    z = x if r is None else (x.float() + r.float()).to(r.dtype)
    if r is not None:
        assert torch.equal(o["z"], z)
    z64, w64 = n64(z), n64(w)
    rstd = 1.0 / np.sqrt((z64 ** 2).mean(1) + eps)
    rel = SUM / 2 + 5 * U  # the square root halves the sum's error; five more roundings
    assert (np.abs(n64(o["rstd"]) - rstd) <= rel * rstd).all()
    y = z64 * rstd[:, None] * w64
    rel += 3 * U
    if o["y"] is not None:
        assert (np.abs(n64(o["y"]) - y) <= (2.0 ** -8 * (1 + rel) + rel) * np.abs(y) + 2.0 ** -133).all()
    if o["yq"] is not None:
        sy = np.abs(y).max(1) / 448
        sy[sy == 0] = 1.0
        got_s = n64(o["sy"])
        assert (np.abs(got_s - sy) <= (rel + 2 * U) * sy).all()
        q = n64(o["yq"].view(torch.float8_e4m3fn).float())
        assert np.isfinite(q).all()
        err = np.abs(q * got_s[:, None] - y)
        half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * sy[:, None])
        assert (err <= half * (1 + 1e-5) + (rel + 4 * U) * 1.0625 * np.abs(y)).all()


CASES = [(1, 8), (1, 4096), (3, 16), (7, 248), (2, 256), (9, 264), (33, 384), (129, 1000),
         (64, 1024), (5, 2048), (700, 2056), (3, 4104), (2, 8192), (3, 16384), (2, 32768)]


@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32, None])
@pytest.mark.parametrize("T,d", CASES)
def test_norm_matches_64_bits(T, d, rdtype):
    x, r, w = _inputs(T, d, rdtype or torch.bfloat16, T * 31 + d)
    r = None if rdtype is None else r
    for codes in (False, True):
        _check_forward(x, r, w, _forward(x, r, w, codes=codes))
    _check_forward(x, r, w, _forward(x, r, w, y=False))


def test_norm_of_zero_rows_and_tiny_and_large_values():
    """Zero rows have codes of zero under scale 1; rows near the type's ends keep finite codes."""
    x, r, w = _inputs(6, 512, torch.bfloat16, 3)
    x[0] = 0
    r[0] = 0
    x[1], r[1] = x[1] * 1e-37, r[1] * 1e-37   # squares vanish: rstd = 1/sqrt(eps)
    x[2], r[2] = x[2] * 1e-30, r[2] * 1e-30
    x[3], r[3] = x[3] * 1e15, r[3] * 1e15
    x[4, 1:], r[4, 1:] = 0, 0                 # one value alone
    o = _forward(x, r, w)
    assert (o["yq"][0] == 0).all() and float(o["sy"][0]) == 1.0 and (o["y"][0] == 0).all()
    _check_forward(x[2:], r[2:], w, {k: v[2:] for k, v in o.items()})
    # row 1: values below the normal range keep an absolute precision of 2^-149 only, and the
    # scale, about 1e-37 * 1e3 / 448, is subnormal itself: its codes only have to be finite and of
    # the right sign
    q = o["yq"][1].view(torch.float8_e4m3fn).float()
    assert torch.isfinite(q).all() and (q * (x[1].float() + r[1].float()) >= 0).all()


def test_norm_in_place_matches_out_of_place():
    x, r, w = _inputs(37, 1024, torch.float32, 5)
    want = _forward(x, r, w)
    xi, ri = x.clone(), r.clone()
    yq, sy = torch.empty_like(want["yq"]), torch.empty_like(want["sy"])
    ops.moe_rms_norm(xi, ri, w, 1e-6, ri, xi, yq, sy, None)
    torch.cuda.synchronize()
    assert torch.equal(ri, want["z"]) and torch.equal(xi, want["y"])
    assert torch.equal(yq, want["yq"]) and torch.equal(sy, want["sy"])


def test_norm_non_finite_values_stay_in_their_rows():
    x, r, w = _inputs(8, 256, torch.bfloat16, 6)
    clean = _forward(x, r, w)
    x[2, 5], x[4, 7] = float("nan"), float("inf")
    o = _forward(x, r, w)
    keep = [0, 1, 3, 5, 6, 7]
    assert torch.equal(o["y"][keep], clean["y"][keep]) and torch.equal(o["yq"][keep], clean["yq"][keep])
    assert torch.isnan(o["y"][2]).all() and torch.isnan(o["y"][4, 7])


def _check_backward(dy, dres, z, rstd, w, dz, dx, dw):
    T, d = dy.shape
    dy64, z64, r64, w64 = n64(dy), n64(z), n64(rstd)[:, None], n64(w)
    dr = 0.0 if dres is None else n64(dres)
    h, g = z64 * r64, dy64 * w64
    c = (g * h).mean(1, keepdims=True)
    want = r64 * (g - h * c) + dr
    # dot product, then the products and sums of the formula, each rounded once
    e = (SUM * np.abs(g * h).mean(1, keepdims=True) + 2 * U * np.abs(c)) * np.abs(h) * r64
    e += r64 * 5 * U * (np.abs(g) + np.abs(h * c)) + 2 * U * (np.abs(want) + np.abs(dr))
    half = HALF[dz.dtype]
    assert (np.abs(n64(dz) - want) <= e + half * (np.abs(want) + e)).all()
    if dx is not None:
        assert (np.abs(n64(dx) - want) <= e + 2.0 ** -8 * (np.abs(want) + e)).all()
    prod = dy64 * h
    assert (np.abs(n64(dw) - prod.sum(0)) <= (T + 3) * U * np.abs(prod).sum(0)).all()


@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", CASES + [(609, 256), (1300, 128), (4096, 64)])
def test_norm_bwd_matches_64_bits(T, d, rdtype):
    dy, z, w = _inputs(T, d, rdtype, T * 17 + d)
    g = torch.Generator().manual_seed(T + d)
    dres = torch.randn(T, d, generator=g).to(rdtype).cuda()
    rstd = 1.0 / torch.sqrt(z.float().square().mean(1) + 1e-6)
    for dr in (dres, None):
        dz, dw = torch.empty_like(z), torch.full((d,), float("nan"), device="cuda")
        dx = torch.empty_like(dy) if rdtype is torch.float32 else None
        ws = torch.full((ops.moe_workspace_bytes(T, d, 1, 1),), 255, dtype=torch.uint8, device="cuda")
        ops.moe_rms_norm_bwd(dy, dr, z, rstd, w, dz, dx, dw, ws)
        torch.cuda.synchronize()
        _check_backward(dy, dr, z, rstd, w, dz, dx, dw)
    inplace, dw2 = dres.clone(), torch.empty_like(dw)
    dz = torch.empty_like(z)
    ops.moe_rms_norm_bwd(dy, dres, z, rstd, w, dz, None, dw, ws)
    ops.moe_rms_norm_bwd(dy, inplace, z, rstd, w, inplace, None, dw2, ws)
    torch.cuda.synchronize()
    assert torch.equal(inplace, dz) and torch.equal(dw, dw2)


def test_norm_gradient_against_differences():
    """The 64-bit formula that the kernel is held to, against central differences of the norm."""
    rng = np.random.default_rng(0)
    T, d, eps, h = 3, 16, 1e-3, 1e-5
    z, w, dy, dres = rng.normal(size=(T, d)), rng.normal(size=d), rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(z, w):
        return (z / np.sqrt((z ** 2).mean(1, keepdims=True) + eps) * w * dy).sum() + (z * dres).sum()
    rstd = 1 / np.sqrt((z ** 2).mean(1, keepdims=True) + eps)
    xh, g = z * rstd, dy * w
    dz = rstd * (g - xh * (g * xh).mean(1, keepdims=True)) + dres
    dw = (dy * xh).sum(0)
    for i in np.ndindex(T, d):
        e = np.zeros((T, d))
        e[i] = h
        assert abs((loss(z + e, w) - loss(z - e, w)) / (2 * h) - dz[i]) < 1e-7 * 100
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert abs((loss(z, w + e) - loss(z, w - e)) / (2 * h) - dw[j]) < 1e-7 * 100


def test_norm_on_a_stream_and_in_a_graph():
    """The same bits on another stream, and from a captured graph replayed on new inputs."""
    T, d = 77, 1024
    x, r, w = _inputs(T, d, torch.bfloat16, 9)
    want = _forward(x, r, w)
    s = torch.cuda.Stream()
    z, y, rstd = torch.empty_like(r), torch.empty_like(x), torch.empty(T, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    ops.moe_rms_norm(x, r, w, 1e-6, z, y, None, None, rstd, stream=s)
    s.synchronize()
    assert torch.equal(z, want["z"]) and torch.equal(y, want["y"])
    dz, dw = torch.empty_like(z), torch.empty(d, device="cuda")
    ws = torch.empty(ops.moe_workspace_bytes(T, d, 1, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_rms_norm(x, r, w, 1e-6, z, y, None, None, rstd)
        ops.moe_rms_norm_bwd(y, x, z, rstd, w, dz, None, dw, ws)
    for seed in (10, 11):
        x2, r2, _ = _inputs(T, d, torch.bfloat16, seed)
        x.copy_(x2)
        r.copy_(r2)
        graph.replay()
        o = _forward(x, r, w)
        dz2, dw2 = torch.empty_like(z), torch.empty_like(dw)
        ops.moe_rms_norm_bwd(o["y"], x, o["z"], o["rstd"], w, dz2, None, dw2, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, o["y"]) and torch.equal(dz, dz2) and torch.equal(dw, dw2)


def test_norm_refuses_mismatched_tensors():
    x, r, w = _inputs(4, 64, torch.bfloat16, 1)
    y, rstd, z = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty_like(r)
    bad = [(x, r, w[:32], z, y), (x, r[:3].contiguous(), w, z, y), (x, r, w, z.float(), y),
           (x, r, w, None, y), (x, None, w, z, y), (x, r, w, z, y[:3].contiguous()),
           (x, r.double(), w, z, y), (x, r, w.to(torch.bfloat16), z, y), (x, r, w, z, None)]
    for a in bad:
        with pytest.raises(ops.MoEError):
            ops.moe_rms_norm(a[0], a[1], a[2], 1e-6, a[3], a[4], None, None, rstd)
    off = torch.empty(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 256].view(4, 64)
    with pytest.raises(ops.MoEError, match="invalid argument"):  # 8-byte aligned only
        ops.moe_rms_norm(off, r, w, 1e-6, z, y, None, None, rstd)
