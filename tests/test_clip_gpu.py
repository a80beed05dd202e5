"""The global gradient norm and clipping against a plain implementation in 64 bits.

Bounds, u = 2^-24: squares are summed in fp32 over at most 32 elements (32 roundings and the
products' one, fused), then in 64 bits, so the sum of squares is off by at most 33 u and the norm
by half of that and its own rounding: 18 u. The factor has one more; a clipped gradient is off by
20 u and half a step of its type."""
import numpy as np
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops
from pretraining_sigmoid_softmax_gb300.layer import clip_grad_norm_

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half the smallest step
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _ws():
    return torch.full((ops.moe_workspace_bytes(1, 128, 1, 1),), 255, dtype=torch.uint8, device="cuda")


def _norm64(grads):
    return np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def _check(grads, max_norm, inplace=False):
    before = [g.clone() for g in grads]
    norm = torch.full((2,), float("nan"), device="cuda")
    out = None if inplace else [torch.full_like(g, float("nan")) for g in grads]
    ops.moe_clip_grads(grads, max_norm, out, norm, _ws())
    only = torch.full((2,), float("nan"), device="cuda")
    ops.moe_grad_norm(before, max_norm, only, _ws())
    torch.cuda.synchronize()
    assert torch.equal(norm, only)
    want = _norm64(before)
    assert abs(float(norm[0]) - want) <= 18 * U * want
    coef = max_norm / want if want > max_norm else 1.0
    if want > max_norm * (1 + 40 * U) or want < max_norm * (1 - 40 * U):
        assert abs(float(norm[1]) - coef) <= 19 * U * coef
        assert coef < 1 or float(norm[1]) == 1.0
    for b, o in zip(before, grads if inplace else out):
        w = b.double() * coef
        assert ((o.double() - w).abs() <= (20 * U + HALF[b.dtype] * (1 + 20 * U)) * w.abs() + TINY[b.dtype]).all()
        if coef == 1.0:
            assert torch.equal(o, b)
    if not inplace:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))


def _grads(shapes, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(t).cuda() for s, t in shapes]


SETS = {
    "one element": [((1,), F32)],
    "one bf16 element": [((1,), BF)],
    "around a vector": [((n,), t) for n in (3, 4, 5, 7, 8, 9, 15, 16, 17) for t in (BF, F32)],
    "around a chunk": [((n,), BF) for n in (16383, 16384, 16385, 32767, 32775)]
                      + [((n,), F32) for n in (16383, 16384, 16387)],
    "a layer": [((8, 128, 256), BF)] * 3 + [((8, 256), F32), ((256,), F32), ((257,), BF)],
    "empty ones among them": [((0,), F32), ((5, 7), BF), ((0, 4), BF), ((1000,), F32)],
    "many": [((1 + i % 97,), BF if i % 3 else F32) for i in range(1000)],
    "very many": [((2 + i % 5,), F32) for i in range(2500)],
    "long": [((3_000_001,), BF), ((2_000_003,), F32)],
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
@pytest.mark.parametrize("inplace", [False, True])
def test_clip_matches_64_bits(name, max_norm, inplace):
    _check(_grads(SETS[name], len(name)), max_norm, inplace)


def test_clip_of_only_empty_tensors():
    norm = torch.full((2,), 7.0, device="cuda")
    ops.moe_clip_grads([torch.empty(0, device="cuda")], 1.0, None, norm, _ws())
    assert norm.tolist() == [0.0, 1.0]


def test_clip_at_every_alignment():
    """Slices of flat buffers at every element offset, with outputs at offsets of their own."""
    for dtype, n in ((BF, 8), (F32, 4)):
        flat = torch.randn(24000, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        other = torch.zeros_like(flat)
        for a in range(n):
            for b in (a, (a + 1) % n, 0):
                g, o = flat[a:a + 20011], other[b:b + 20011]
                other.fill_(5.0)
                norm = torch.empty(2, device="cuda")
                ops.moe_clip_grads([g], 1.0, [o], norm, _ws())
                torch.cuda.synchronize()
                want = _norm64([g])
                assert abs(float(norm[0]) - want) <= 18 * U * want
                w = g.double() / want
                assert ((o.double() - w).abs() <= (20 * U + 1.001 * HALF[dtype]) * w.abs() + TINY[dtype]).all()
                assert (other[:b] == 5).all() and (other[b + 20011:] == 5).all()  # nothing beside it


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-17, 1e17, 1e22, 1e30])
def test_clip_of_tiny_and_huge_gradients(scale, dtype):
    """Squares outside fp32's range."""
    g = _grads([((5000,), dtype), ((33,), dtype)], 3, 1.0)
    g = [(t.float() * scale).to(dtype) for t in g]
    g[0][100:2000] = 0
    _check(g, scale)
    _check(g + _grads([((100,), F32)], 4), scale)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_clip_leaves_gradients_of_a_non_finite_norm(bad):
    g = _grads([((5000,), BF), ((70,), F32)], 5)
    g[1][3] = bad
    before = [t.clone() for t in g]
    norm, out = torch.empty(2, device="cuda"), [torch.empty_like(t) for t in g]
    ops.moe_clip_grads(g, 1e-3, out, norm, _ws())
    ops.moe_clip_grads(g, 1e-3, None, norm, _ws())
    torch.cuda.synchronize()
    assert not torch.isfinite(norm[0]) and float(norm[1]) == 1.0
    for a, b, c in zip(g, before, out):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
        assert torch.equal(torch.nan_to_num(c), torch.nan_to_num(b))


def test_clip_to_zero():
    g = _grads([((100,), F32)], 6)
    norm = torch.empty(2, device="cuda")
    ops.moe_clip_grads(g, 0.0, None, norm, _ws())
    assert float(norm[1]) == 0.0 and (g[0] == 0).all()


def test_clip_repeats_bit_for_bit_and_on_a_stream_and_in_graphs():
    """Two captured graphs, each with its own workspace, replayed on new gradients, the second
    on another stream."""
    shapes = SETS["a layer"]
    g = _grads(shapes, 7)
    outs = [[torch.empty_like(t) for t in g] for _ in range(2)]
    norms, wss = [torch.empty(2, device="cuda") for _ in range(2)], [_ws(), _ws()]
    graphs = []
    for o, n, w in zip(outs, norms, wss):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.moe_clip_grads(g, 0.5, o, n, w)
        graphs.append(graph)
    s = torch.cuda.Stream()
    for seed in (8, 9):
        for t, new in zip(g, _grads(shapes, seed)):
            t.copy_(new)
        s.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(s):
            graphs[1].replay()
        torch.cuda.synchronize()
        want, n, w = [torch.empty_like(t) for t in g], torch.empty(2, device="cuda"), _ws()
        ops.moe_clip_grads(g, 0.5, want, n, w)
        torch.cuda.synchronize()
        for o, m in zip(outs, norms):
            assert torch.equal(m, n) and all(torch.equal(a, b) for a, b in zip(o, want))


def test_clip_refuses_mismatched_tensors():
    g, norm = _grads([((8,), F32), ((8,), BF)], 1), torch.empty(2, device="cuda")
    for out in ([g[0]], [g[0], g[0]], [g[1], g[0]], [g[0][:4], g[1]]):
        with pytest.raises(ops.MoEError):
            ops.moe_clip_grads(g, 1.0, out, norm, _ws())
    with pytest.raises(ops.MoEError, match="invalid argument"):
        ops.moe_clip_grads([g[0], g[0]], 1.0, None, norm, _ws())
    with pytest.raises(ops.MoEError, match="invalid argument"):
        ops.moe_clip_grads([], 1.0, None, norm, _ws())
    with pytest.raises(ops.MoEError, match="bf16 or fp32"):
        ops.moe_clip_grads([g[0].half()], 1.0, None, norm, _ws())
    with pytest.raises(ops.MoEError, match="contiguous"):
        ops.moe_clip_grads([torch.zeros(4, 4, device="cuda").t()], 1.0, None, norm, _ws())
    with pytest.raises(ops.MoEError, match="workspace"):
        ops.moe_clip_grads(g, 1.0, None, norm, _ws()[:64])


def _params(shapes, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    ps = [torch.nn.Parameter(torch.zeros(s, device="cuda", dtype=dtype)) for s in shapes]
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g).to(dtype).cuda()
    return ps


@pytest.mark.parametrize("dtype", [BF, F32])
def test_clip_grad_norm_takes_gradients_in_any_order_of_dimensions(dtype):
    """A transposed parameter's gradient is transposed too; its elements still lie side by side."""
    ps = _params([(33, 70), (5, 6, 7), (64,), (1, 40), (4, 3, 5, 2), (0, 3)], dtype, 11)
    ps[0].grad = ps[0].grad.t().contiguous().t()
    ps[1].grad = ps[1].grad.permute(2, 0, 1).contiguous().permute(1, 2, 0)
    ps[4].grad = ps[4].grad.contiguous(memory_format=torch.channels_last)
    assert sum(not p.grad.is_contiguous() for p in ps) == 3
    before, at = [p.grad.clone() for p in ps], [(p.grad.data_ptr(), p.grad.stride()) for p in ps]
    want = _norm64(before)
    norm = clip_grad_norm_(ps, 0.5)
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 18 * U * want
    for p, b, a in zip(ps, before, at):
        assert (p.grad.data_ptr(), p.grad.stride()) == a
        w = b.double() * (0.5 / want)
        assert ((p.grad.double() - w).abs() <= (20 * U + HALF[dtype] * (1 + 20 * U)) * w.abs() + TINY[dtype]).all()


def test_clip_grad_norm_refuses_gradients_with_gaps():
    """Elements of a larger tensor, or one element many times: named, and nothing is clipped."""
    for grad in (torch.randn(8, 16, device="cuda")[:, ::2], torch.randn(8, 1, device="cuda").expand(8, 8)):
        ps = _params([(8, 8), (8, 8)], F32, 12)
        before = ps[0].grad.clone()
        ps[1].grad = grad
        with pytest.raises(ops.MoEError, match=r"gradient 1 .*side by side"):
            clip_grad_norm_(ps, 1e-3)
        torch.cuda.synchronize()
        assert torch.equal(ps[0].grad, before)


def test_clip_grad_norm_without_gradients_is_a_device_zero():
    ps = [torch.nn.Parameter(torch.zeros(4, device="cuda"))]
    norm = clip_grad_norm_(iter(ps), 1.0)
    assert norm.shape == () and norm.is_cuda and norm.dtype == F32 and float(norm) == 0.0
