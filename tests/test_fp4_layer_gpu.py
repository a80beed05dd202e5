"""The layer on 4-bit experts (precision fp4 and fp4_dgrad): a step against the same formulas in 64
bits, held weights for serving, captured and replayed steps, streams, and refusals.

Bound. The codes are taken from the same bf16 numbers in both, up to those that a 32-bit and a 64-bit
result round to different neighbours; so the difference is that of the tensors stored in bf16
between (at most half a step, 2^-8, each): rows of y, out, dY, dA, dU, dX, the shared expert's and
the layer's, at most twelve of them in a row (tests of the block with its norm count the same)."""
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops
from pretraining_sigmoid_softmax_gb300.layer import MoELayer, MoEPlan, MoEShape, weights4

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

REL = 12 * 2.0 ** -8


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm().clamp_min(1e-300))


def bf(t):
    return t.to(torch.bfloat16).double()


def hat(x, nv):
    """The numbers that the codes of x's rows stand for, in 64 bits on the GPU."""
    b = 16 if nv else 32
    v = x.double().unflatten(-1, (-1, b))
    amax = v.abs().amax(-1, keepdim=True)
    p2 = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    if nv:
        top = amax.amax(-2, keepdim=True).clamp(min=2.0 ** -100)
        e = torch.frexp(top).exponent - 12
        g = p2(e + (top > 2688 * p2(e)))
        s = amax / g / 6
        step = p2((torch.frexp(s).exponent - 1).clamp(min=-6) - 3)
        s = g * (torch.round(s / step) * step).clamp(max=448)
    else:
        s = p2(torch.frexp(amax.clamp(min=2.0 ** -100)).exponent - 3)
    z = (v.abs() / torch.where(s > 0, s, 1.0)).clamp(max=6)
    step = p2((torch.frexp(z).exponent - 1).clamp(min=0) - 1)
    return (torch.sign(v) * torch.round(z / step) * step * s).flatten(-2)


def cols_hat(w, nv):
    return hat(w.t().contiguous(), nv).t()


def expert(x, Wg, Wu, Wd, nv):
    xh = hat(x, nv)
    a, u = xh @ hat(Wg, nv).t(), xh @ hat(Wu, nv).t()
    h = bf(torch.nn.functional.silu(a) * u)
    return bf(a), bf(u), h, bf(hat(h, nv) @ hat(Wd, nv).t())


def expert_bwd(dy, x, a, u, h, Wg, Wu, Wd, nv, dgrad):
    r = hat(dy, nv) @ cols_hat(Wd, nv) if dgrad else dy @ Wd
    p = torch.sigmoid(a)
    da, du = bf(r * u * p * (1 + a * (1 - p))), bf(r * a * p)
    if dgrad:
        dx = hat(torch.cat([da, du], 1), nv) @ cols_hat(torch.cat([Wg, Wu]), nv)
    else:
        dx = da @ Wg + du @ Wu
    return bf(dx), da.t() @ x, du.t() @ x, dy.t() @ h


def reference(layer, x, idx, dout):
    """out and all gradients, with the experts `idx` of each token."""
    nv, dg4 = layer.fp4_format == ops.FP4_NV, layer.fp4_dgrad
    p = {n: t.detach().double() for n, t in layer.named_parameters()}
    grads = {n: torch.zeros_like(t) for n, t in p.items()}
    xr, W_r = x.double().requires_grad_(True), p["W_r"].clone().requires_grad_(True)
    l = xr @ W_r.t()
    s = torch.sigmoid(l) if layer.mode == ops.MODE_SIGMOID else torch.softmax(l, 1)
    gate = s.gather(1, idx)
    if layer.mode == ops.MODE_SIGMOID if layer.renorm is None else layer.renorm:
        gate = gate / gate.sum(1, keepdim=True)
    gate = layer.gate_scale * gate
    x64, dout = x.double(), dout.double()
    out, dx, dgate = torch.zeros_like(x64), torch.zeros_like(x64), torch.zeros_like(gate)
    for e in range(layer.E):
        t, i = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        w = [p[n][e] for n in ("W_g", "W_u", "W_d")]
        a, u, h, y = expert(x64[t], *w, nv)
        g = gate[t, i].detach()[:, None]
        out.index_add_(0, t, g * y)
        dgate[t, i] = (dout[t] * y).sum(1)
        dxe, grads["W_g"][e], grads["W_u"][e], grads["W_d"][e] = expert_bwd(
            bf(g * dout[t]), x64[t], a, u, h, *w, nv, dg4)
        dx.index_add_(0, t, dxe)
    if layer.f_shared:
        w = [p[n] for n in ("Ws_g", "Ws_u", "Ws_d")]
        a, u, h, y = expert(x64, *w, nv)
        out += y
        dxe, grads["Ws_g"], grads["Ws_u"], grads["Ws_d"] = expert_bwd(dout, x64, a, u, h, *w, nv, dg4)
        dx += dxe
    (gate * dgate).sum().backward()
    grads["W_r"] = W_r.grad
    return out, dx + xr.grad, grads


CASES = {
    "sigmoid": dict(T=300, d=256, E=8, k=2, f=128),
    "shared": dict(T=515, d=384, E=16, k=4, f=256, f_shared=384),
    "softmax": dict(T=257, d=512, E=24, k=3, f=256, mode="softmax"),
    "groups": dict(T=200, d=256, E=16, k=4, f=128, f_shared=128, n_group=4, topk_group=2, gate_scale=2.5),
    "router term in the rows": dict(T=260, d=256, E=8, k=2, f=768),
    "one token": dict(T=1, d=1024, E=16, k=4, f=256, f_shared=256),
}


def _layer(name, precision, fmt, **kw):
    c = dict(CASES[name])
    T = c.pop("T")
    torch.manual_seed(len(name))
    layer = MoELayer(precision=precision, fp4_format=fmt, **c, **kw)
    x = torch.randn(T, c["d"], device="cuda").to(torch.bfloat16)
    return layer, x


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("precision", ["fp4", "fp4_dgrad"])
@pytest.mark.parametrize("name", CASES)
def test_step_matches_64_bits(name, precision, fmt):
    layer, x = _layer(name, precision, fmt)
    x.requires_grad_(True)
    dout = torch.randn_like(x)
    ops.moe_clear_device_status()
    out = layer(x)
    out.backward(dout)
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)
    want, dx, grads = reference(layer, x.detach(), layer._last_plan.topk_idx.long(), dout)
    assert _off(out, want) <= REL
    assert _off(x.grad, dx) <= REL
    for n, p in layer.named_parameters():
        assert _off(p.grad, grads[n]) <= REL, n


def test_the_two_formats_and_bf16_differ_as_their_steps_do():
    """The layers' outputs are apart by the codes' steps: E2M1 rounds by up to 1/6 of a block's largest
    value (twice in a row), and blocks of 16 with finer scales are nearer to bf16 than blocks of 32."""
    outs = {}
    for precision, fmt in (("bf16", "nv"), ("fp4", "nv"), ("fp4", "mx")):
        layer, x = _layer("shared", precision, fmt)
        with torch.no_grad():
            outs[precision, fmt] = layer(x).double()
    nv, mx = (_off(outs["fp4", f], outs["bf16", "nv"]) for f in ("nv", "mx"))
    assert 0.01 < nv < mx < 0.5


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("name", ["shared", "one token", "groups"])
def test_held_weights_give_the_same_output(name, fmt):
    layer, x = _layer(name, "fp4", fmt)
    with torch.no_grad():
        want = layer(x)
        layer.hold_weights()
        assert torch.equal(layer(x), want)
        plan = layer._last_plan
        assert plan.A is None and not plan.has_backward and plan.W4 is None
        layer.W_g.mul_(2.0)                      # held: not seen until they are quantised again
        assert torch.equal(layer(x), want)
        layer.hold_weights()
        assert not torch.equal(layer(x), want)
        layer.W_g.mul_(0.5)
    with pytest.raises(ValueError, match="held"):
        layer(x)                                 # the parameters require a gradient
    layer.hold_weights(False)
    x.requires_grad_(True)
    out = layer(x)
    assert torch.equal(out, want)
    out.sum().backward()
    assert x.grad is not None


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_captured_forward_follows_weights_held_again(fmt):
    layer, x = _layer("shared", "fp4", fmt)
    layer.hold_weights()
    with torch.no_grad():
        for _ in range(2):
            layer(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x)
        for _ in range(3):
            for w in (layer.W_g, layer.W_d, layer.Ws_u):
                w.copy_(torch.randn_like(w) * 0.1)
            layer.hold_weights()
            graph.replay()
            got = out.clone()
            want = layer(x)
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_plans_refuse_other_weights():
    layer, x = _layer("shared", "fp4", "mx")
    W = [getattr(layer, n).detach() for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")]
    plan = MoEPlan(layer._plan(x.shape[0]).s, backward=False)
    with pytest.raises(ValueError, match="3 operands"):
        plan.forward(x, layer.W_r.detach(), layer.b, *W, weights4=weights4(ops.FP4_MX, *W[:3]))
    with pytest.raises(ops.MoEError, match="format"):
        plan.forward(x, layer.W_r.detach(), layer.b, *W, weights4=weights4(ops.FP4_NV, *W))
    bf16, x = _layer("shared", "bf16", "mx")
    plan = MoEPlan(bf16._plan(x.shape[0]).s, backward=False)
    with pytest.raises(ValueError, match="4-bit"):
        plan.forward(x, layer.W_r.detach(), layer.b, *W, weights4=weights4(ops.FP4_MX, *W))


def test_serving_tokens_one_by_one_equals_the_batch():
    """Rows do not depend on one another: tokens alone give what they give in a batch."""
    layer, x = _layer("sigmoid", "fp4", "mx")
    with torch.no_grad():
        layer.hold_weights()
        want = layer(x[:5].contiguous())
        for i in range(5):
            assert torch.equal(layer(x[i:i + 1]), want[i:i + 1])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_norm_in_front_of_the_layer(fmt):
    """The layer with its norm is the layer on the norm's y."""
    layer, x = _layer("shared", "fp4_dgrad", fmt, norm_eps=1e-6)
    plain, _ = _layer("shared", "fp4_dgrad", fmt)
    plain.load_state_dict({n: t for n, t in layer.state_dict().items() if not n.startswith("norm")})
    res = torch.randn_like(x)
    out, z = layer(x, res)
    y, _ = layer.norm(x, res)
    assert torch.equal(out, plain(y))
    out.sum().backward()
    assert all(torch.isfinite(p.grad).all() for p in layer.parameters())


@pytest.mark.parametrize("precision,fmt", [("fp4", "mx"), ("fp4_dgrad", "nv"), ("fp4_dgrad", "mx")])
def test_captured_step_equals_the_eager_one_and_repeats(precision, fmt):
    layer, x = _layer("shared", precision, fmt)
    dY = torch.randn_like(x)
    shape = layer._plan(x.shape[0]).s
    W = {n: p.detach() for n, p in layer.named_parameters()}
    eager, plan = MoEPlan(shape), MoEPlan(shape)
    eager.forward(x, W["W_r"], layer.b, *(W[n] for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")))
    eager.backward(dY)
    graph = plan.capture_step(x, W, dY, layer.b)
    for _ in range(2):
        plan.out.zero_()
        for g in plan.grads().values():
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out, eager.out)
        for n, g in plan.grads().items():
            assert torch.equal(g, eager.grads()[n]), n
    assert ops.moe_device_status() == (0, 0)


def test_two_plans_on_two_streams_at_once():
    layer, x = _layer("sigmoid", "fp4_dgrad", "nv")
    shape = layer._plan(x.shape[0]).s
    W = [p.detach() for n, p in layer.named_parameters() if n != "W_r"]
    plans = [MoEPlan(shape) for _ in range(3)]
    xs = [x, x.flip(0).contiguous()]
    dY = torch.randn_like(x)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, t, st in zip(plans, xs, streams):
            p.forward(t, layer.W_r.detach(), layer.b, *W, stream=st)
            p.backward(dY, stream=st)
    torch.cuda.synchronize()
    for p, t in zip(plans, xs):
        plans[2].forward(t, layer.W_r.detach(), layer.b, *W)
        plans[2].backward(dY)
        torch.cuda.synchronize()
        assert torch.equal(p.out, plans[2].out)
        for n, g in p.grads().items():
            assert torch.equal(g, plans[2].grads()[n]), n


def test_weights_quantised_on_a_stream_of_their_own():
    layer, x = _layer("shared", "fp4", "nv")
    W = [getattr(layer, n).detach() for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    W4 = weights4(ops.FP4_NV, *W, stream=st)
    st.synchronize()
    with torch.no_grad():
        want = layer(x)
    plan = MoEPlan(layer._plan(x.shape[0]).s, backward=False)
    plan.forward(x, layer.W_r.detach(), layer.b, *W, weights4=W4)
    torch.cuda.synchronize()
    assert torch.equal(plan.out, want)


@pytest.mark.parametrize("precision", ["fp4", "fp4_dgrad"])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("name", ["shared", "router term in the rows"])
def test_launch_count_matches_the_plan(name, fmt, precision):
    from torch.autograd import DeviceType
    from torch.profiler import ProfilerActivity, profile
    layer, x = _layer(name, precision, fmt)
    W = [None if getattr(layer, n) is None else getattr(layer, n).detach()
         for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")]
    plan = MoEPlan(layer._plan(x.shape[0]).s)
    dY = torch.randn_like(x)

    def step():
        plan.forward(x, layer.W_r.detach(), layer.b, *W)
        plan.backward(dY)

    step()
    torch.cuda.synchronize()
    kernels = []
    for _ in range(2):  # the profiler's first session in a process may record no activity
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            step()
            torch.cuda.synchronize()
        kernels = [e.name for e in prof.events() if e.device_type == DeviceType.CUDA]
        if kernels:
            break
    if not kernels:
        pytest.skip("the profiler recorded no CUDA activity on this machine")
    assert len([n for n in kernels if "moe::" in n]) == plan.launches_per_step()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_launch_count_without_a_backward(fmt):
    from torch.autograd import DeviceType
    from torch.profiler import ProfilerActivity, profile
    layer, x = _layer("shared", "fp4", fmt)
    W = [getattr(layer, n).detach() for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")]
    plan = MoEPlan(layer._plan(x.shape[0]).s, backward=False)
    assert plan.X_perm is None
    plan.forward(x, layer.W_r.detach(), layer.b, *W)
    torch.cuda.synchronize()
    kernels = []
    for _ in range(2):  # the profiler's first session in a process may record no activity
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            plan.forward(x, layer.W_r.detach(), layer.b, *W)
            torch.cuda.synchronize()
        kernels = [e.name for e in prof.events() if e.device_type == DeviceType.CUDA]
        if kernels:
            break
    if not kernels:
        pytest.skip("the profiler recorded no CUDA activity on this machine")
    assert len([n for n in kernels if "moe::" in n]) == plan.launches_per_step(backward=False)


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (700, 16, 4)])
def test_layout_without_its_rows(T, E, k):
    torch.manual_seed(T)
    idx = torch.rand(T, E, device="cuda").topk(k, 1).indices.to(torch.int32)
    gate, R, i32, i64 = torch.rand(T, k, device="cuda"), ops.moe_padded_rows(T, k, E), torch.int32, torch.int64
    ws = torch.empty(ops.moe_workspace_bytes(T, 128, E, k), dtype=torch.uint8, device="cuda")
    x = torch.randn(T, 128, device="cuda").to(torch.bfloat16)
    outs = []
    for rows in (True, False):
        o = [torch.full(n, -7, dtype=t, device="cuda") for n, t in (
            ((E,), i32), ((E + 1,), i64), ((E + 1,), i64), ((R,), i32), ((T, k), i32))]
        g = torch.full((R,), -7.0, device="cuda")
        ops.moe_permute(idx, x if rows else None, E, *o,
                        torch.empty(R, 128, dtype=torch.bfloat16, device="cuda") if rows else None, ws,
                        topk_gate=gate, row_gate=g)
        outs.append(o + [g])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    with pytest.raises(ops.MoEError, match="invalid"):
        ops.moe_permute(idx, x, E, *o, None, ws)


def test_layer_refuses_unknown_formats_and_weights_to_hold():
    with pytest.raises(ValueError, match="fp4_format"):
        MoELayer(128, 4, 2, 128, precision="fp4", fp4_format="e2m1")
    with pytest.raises(ValueError, match="precision"):
        MoELayer(128, 4, 2, 128, precision="int4")
    with pytest.raises(ValueError, match="fp4"):
        MoELayer(128, 4, 2, 128).hold_weights()
    shape = MoEShape(64, 128, 4, 2, 128, fp8=True, fp4=True)
    with pytest.raises(ValueError, match="fp8"):
        MoEPlan(shape)
