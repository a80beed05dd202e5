"""The operators around the layer as a training step uses them: residual addition and RMS norm,
experts chosen within groups, the layer, its backward through the norm, and clipping, against a
64-bit autograd graph of the same formulas on the GPU's choice of experts.

Bounds. Every tensor that a step stores in bf16 is off by at most half a step, 2^-8 of each
value (2^-9 on average over a binade), so by at most 2^-8 of its norm; errors of independent
roundings do not add up coherently in a product, and the map from one stored tensor to the next
(a product with a Gaussian matrix, SwiGLU, a sum) keeps relative norms of errors to within a
small factor. Forward, seven tensors are stored between the inputs and out (z, y, a, u, h, the
experts' rows, out); a gradient has up to five more (the rows of dY, dA, dU, dX, dx). Twelve
times 2^-8 bounds the relative norm of every difference: 4.7e-2. FP8 operands have 2^-4 of each
value instead, twice in a row (the input and h): 2 * 2^-4 on top."""
import numpy as np
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops
from pretraining_sigmoid_softmax_gb300.layer import MoELayer, MoEPlan, MoEShape, RMSNorm, clip_grad_norm_

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

REL = 12 * 2.0 ** -8
REL_FP8 = REL + 2 * 2.0 ** -4


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _off(got, want):
    want = want.double()
    return float((got.double() - want).norm() / want.norm().clamp_min(1e-300))


def _reference(layer, x, residual, idx, dout, dz):
    """out, the stream and all gradients in 64 bits, with the experts `idx` of each token."""
    p = {n: t.detach().double().requires_grad_(True) for n, t in layer.named_parameters()}
    x, r = x.double().requires_grad_(True), residual.double().requires_grad_(True)
    z = x + r
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + layer.norm.eps) * p["norm.w"]
    l = y @ p["W_r"].t()
    s = torch.sigmoid(l) if layer.mode == ops.MODE_SIGMOID else torch.softmax(l, 1)
    g = s.gather(1, idx)
    renorm = layer.mode == ops.MODE_SIGMOID if layer.renorm is None else layer.renorm
    if renorm:
        g = g / g.sum(1, keepdim=True)
    g = layer.gate_scale * g
    out = torch.zeros_like(y)
    for e in range(layer.E):
        t, i = (idx == e).nonzero(as_tuple=True)
        if len(t):
            h = torch.nn.functional.silu(y[t] @ p["W_g"][e].t()) * (y[t] @ p["W_u"][e].t())
            out = out.index_add(0, t, g[t, i][:, None] * (h @ p["W_d"][e].t()))
    if layer.f_shared:
        out = out + (torch.nn.functional.silu(y @ p["Ws_g"].t()) * (y @ p["Ws_u"].t())) @ p["Ws_d"].t()
    loss = (out * dout.double()).sum() + (z * dz.double()).sum()
    if layer.mode == ops.MODE_SOFTMAX and layer.z_coef:
        loss = loss + layer.z_coef * (torch.logsumexp(l, 1) ** 2).mean()
    loss.backward()
    return out, z, x.grad, r.grad, {n: t.grad for n, t in p.items()}


CASES = {
    "sigmoid in groups": dict(T=300, d=256, E=16, k=4, f=128, f_shared=128, mode="sigmoid", n_group=4,
                              topk_group=2, gate_scale=2.5),
    "softmax renormalised": dict(T=257, d=384, E=24, k=3, f=256, mode="softmax", n_group=3, topk_group=2,
                                 group_rule="max", renorm=True),
    "softmax with z-loss": dict(T=200, d=256, E=32, k=4, f=128, mode="softmax", z_coef=1e-2, n_group=8,
                                topk_group=4),
    "many experts": dict(T=150, d=256, E=160, k=6, f=128, mode="sigmoid", n_group=8, topk_group=4,
                         renorm=False),
    "no groups, long experts": dict(T=128, d=256, E=8, k=2, f=768, mode="sigmoid"),
    "fp8": dict(T=256, d=256, E=16, k=4, f=256, f_shared=128, mode="sigmoid", n_group=4, topk_group=2,
                precision="fp8"),
    "fp8 data gradients": dict(T=256, d=256, E=16, k=4, f=256, mode="sigmoid", n_group=4, topk_group=2,
                               precision="fp8_dgrad"),
}


@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", CASES)
def test_block_matches_64_bits(name, rdtype):
    c = dict(CASES[name])
    T, d = c.pop("T"), c["d"]
    torch.manual_seed(len(name))
    layer = MoELayer(norm_eps=1e-5, **c)
    with torch.no_grad():
        layer.norm.w.add_(0.1 * torch.randn(d, device="cuda"))
        if layer.mode == ops.MODE_SIGMOID:
            layer.b.copy_(0.1 * torch.rand(layer.E, device="cuda"))
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16).requires_grad_(True)
    res = torch.randn(T, d, device="cuda").to(rdtype).requires_grad_(True)
    dout = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    dz = torch.randn(T, d, device="cuda").to(rdtype)
    ops.moe_clear_device_status()
    out, z = layer(x, res)
    torch.autograd.backward([out, z], [dout, dz])
    torch.cuda.synchronize()
    assert ops.moe_device_status()[0] == 0
    plan = layer._last_plan
    assert plan.s.selects == (name != "no groups, long experts")
    idx = plan.topk_idx.long()
    per = layer.E // layer.n_group
    assert (torch.stack([(idx // per == g).any(1) for g in range(layer.n_group)]).sum(0)
            <= layer.topk_group).all()
    want_out, want_z, want_dx, want_dr, grads = _reference(layer, x.detach(), res.detach(), idx, dout, dz)
    rel = REL_FP8 if layer.fp8 else REL
    assert out.dtype == torch.bfloat16 and z.dtype == rdtype
    assert torch.equal(z, (x.detach().float() + res.detach().float()).to(rdtype))
    assert _off(out, want_out) <= rel
    assert x.grad.dtype == torch.bfloat16 and res.grad.dtype == rdtype
    assert _off(x.grad, want_dx) <= rel and _off(res.grad, want_dr) <= rel
    for n, p in layer.named_parameters():
        assert p.grad.dtype == p.dtype
        assert _off(p.grad, grads[n]) <= rel, n
    # the step's end: clip what the backward left
    before = {n: p.grad.clone() for n, p in layer.named_parameters()}
    total = float(torch.sqrt(sum((g.double() ** 2).sum() for g in before.values())))
    norm = layer.clip_grads_(0.5)
    assert abs(float(norm) - total) <= 1e-5 * total and total > 0.5
    for n, p in layer.named_parameters():
        assert _off(p.grad, before[n].double() * (0.5 / total)) <= 2.0 ** -8
    assert float(clip_grad_norm_(layer.parameters(), 1.0)) == pytest.approx(0.5, rel=2.0 ** -8)


def test_fp8_block_takes_the_norm_codes():
    """The FP8 layer reads the codes that the norm wrote: the experts' inputs are those codes."""
    torch.manual_seed(0)
    layer = MoELayer(256, 8, 2, 128, precision="fp8", norm_eps=1e-6)
    x = torch.randn(200, 256, device="cuda").to(torch.bfloat16)
    layer(x)
    plan = layer._last_plan
    yq, sy = torch.empty_like(plan.x8), torch.empty_like(plan.sx)
    y, z = layer.norm(x, None, yq, sy)
    torch.cuda.synchronize()
    assert z is x and torch.equal(plan.x8, yq) and torch.equal(plan.sx, sy)
    rows = plan.slot_to_row.reshape(-1).long()
    assert torch.equal(plan.X8[rows], yq.repeat_interleave(2, 0))
    dq = yq.view(torch.float8_e4m3fn).float() * sy[:, None]
    # a code is off by half a step of E4M3, 2^-4 of the value or 2^-10 of the scale, and y itself by
    # half a step of bf16
    half = torch.maximum(2.0 ** -4 * y.float().abs(), 2.0 ** -10 * sy[:, None])
    assert ((dq - y.float()).abs() <= half * (1 + 2.0 ** -7) + 2.0 ** -8 * 1.07 * y.float().abs()).all()


def test_two_blocks_share_a_residual_stream():
    """Two layers in a row on one fp32 stream: gradients meet in it. The stream's own gradient is
    checked against 64-bit autograd of the same two blocks."""
    torch.manual_seed(3)
    T, d = 130, 256
    layers = [MoELayer(d, 16, 4, 128, norm_eps=1e-6, n_group=4, topk_group=2) for _ in range(2)]
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16).requires_grad_(True)
    r = torch.randn(T, d, device="cuda").requires_grad_(True)
    y1, z1 = layers[0](x, r)
    y2, z2 = layers[1](y1, z1)
    dout = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    dz = torch.randn(T, d, device="cuda")
    torch.autograd.backward([y2, z2], [dout, dz])
    torch.cuda.synchronize()
    idx = [l._last_plan.topk_idx.long() for l in layers]
    _, _, gx2, gr2, _ = _reference(layers[1], y1.detach(), z1.detach(), idx[1], dout, dz)
    _, _, gx1, gr1, _ = _reference(layers[0], x.detach(), r.detach(), idx[0], gx2, gr2)
    assert _off(x.grad, gx1) <= 2 * REL and _off(r.grad, gr1) <= 2 * REL


def test_norm_module_alone():
    torch.manual_seed(4)
    norm = RMSNorm(512, eps=1e-5)
    x = torch.randn(33, 512, device="cuda").to(torch.bfloat16).requires_grad_(True)
    y, z = norm(x)
    assert z is x
    dy = torch.randn_like(y)
    y.backward(dy)
    x64, w64 = x.detach().double().requires_grad_(True), norm.w.detach().double().requires_grad_(True)
    y64 = x64 * torch.rsqrt((x64 ** 2).mean(1, keepdim=True) + 1e-5) * w64
    y64.backward(dy.double())
    assert _off(y, y64) <= 2.0 ** -8 and _off(x.grad, x64.grad) <= 2.0 ** -8
    assert _off(norm.w.grad, w64.grad) <= 1e-5
    # a stream that is used alone: its gradient is x's and the residual's
    r = torch.randn(33, 512, device="cuda", requires_grad=True)
    x.grad = None
    _, z = norm(x, r)
    g = torch.randn_like(z)
    z.backward(g)
    assert torch.equal(r.grad, g) and torch.equal(x.grad, g.to(torch.bfloat16))
    with pytest.raises(ValueError):
        norm(x.float())
    with pytest.raises(ValueError):
        norm(x, r[:5])


def test_norm_refuses_a_second_derivative():
    """Its backward is a kernel: autograd cannot go through it again, and says so."""
    norm = RMSNorm(256)
    x = torch.randn(4, 256, device="cuda").to(torch.bfloat16).requires_grad_(True)
    g, = torch.autograd.grad(norm(x)[0].float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().sum().backward()


def test_layer_refuses_what_it_cannot_do():
    for kw in (dict(n_group=3), dict(n_group=4, topk_group=5), dict(n_group=4, topk_group=1, k=5),
               dict(group_rule="sum"), dict(gate_scale=0.0), dict(gate_scale=-1.0)):
        a = dict(d=128, E=16, k=4, f=128)
        a.update(kw)
        with pytest.raises(ValueError):
            MoELayer(**a)
    layer = MoELayer(128, 8, 2, 128)
    x = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="norm_eps"):
        layer(x, x)


@pytest.mark.parametrize("E,mode,T", [(16, ops.MODE_SIGMOID, 260), (16, ops.MODE_SOFTMAX, 260),
                                      (160, ops.MODE_SIGMOID, 260), (32, ops.MODE_SIGMOID, 3000)])
def test_plan_step_in_a_graph_and_launch_count(E, mode, T):
    """A captured step with grouped routing repeats the eager one bit for bit, and runs as many
    kernels as the plan says."""
    from torch.autograd import DeviceType
    from torch.profiler import ProfilerActivity, profile
    torch.manual_seed(E)
    d, f, k = 256, 128, 4
    plan = MoEPlan(MoEShape(T, d, E, k, f, mode=mode, seq_len=T, n_group=4, topk_group=2, gate_scale=1.5))
    dev = dict(device="cuda")
    W = dict(W_r=torch.randn(E, d, **dev) / 16, W_g=torch.randn(E, f, d, **dev).to(torch.bfloat16) / 16,
             W_u=torch.randn(E, f, d, **dev).to(torch.bfloat16) / 16,
             W_d=torch.randn(E, d, f, **dev).to(torch.bfloat16) / 16)
    b = torch.rand(E, **dev) * 0.1
    x, dY = (torch.randn(T, d, **dev).to(torch.bfloat16) for _ in range(2))
    graph = plan.capture_step(x, W, dY, b)
    for _ in range(2):
        x.copy_(torch.randn(T, d, **dev))
        graph.replay()
        torch.cuda.synchronize()
        got = [plan.out.clone(), plan.topk_idx.clone(), *(t.clone() for t in plan.grads().values())]

        def step():
            plan.forward(x, W["W_r"], b, W["W_g"], W["W_u"], W["W_d"])
            plan.backward(dY)
        step()
        torch.cuda.synchronize()
        for a, t in zip(got, [plan.out, plan.topk_idx, *plan.grads().values()]):
            assert torch.equal(a, t)
    kernels = []
    for _ in range(2):
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            step()
            torch.cuda.synchronize()
        kernels = [e.name for e in prof.events() if e.device_type == DeviceType.CUDA]
        if kernels:
            break
    if kernels:
        assert len([n for n in kernels if "moe::" in n]) == plan.launches_per_step()
    # the plan's gradients clipped into buffers of an optimiser's own
    g = {n: t.clone() for n, t in plan.grads().items() if n != "dx"}
    out = {n: torch.full_like(t, float("nan")) for n, t in g.items()}
    norm = plan.clip_grads(1e-3, out)
    torch.cuda.synchronize()
    total = float(torch.sqrt(sum((t.double() ** 2).sum() for t in g.values())))
    assert abs(float(norm[0]) - total) <= 1e-5 * total
    for n, t in g.items():
        assert torch.equal(plan.grads()[n], t)  # untouched
        assert _off(out[n], t.double() * (1e-3 / total)) <= 2.0 ** -8
    with pytest.raises(ValueError):
        plan.clip_grads(1.0, {"dW_r": out["dW_r"]})


class _OtherNorm(torch.nn.Module):
    """A norm of the user's own, which knows nothing of codes."""

    def __init__(self, norm):
        super().__init__()
        self.norm = norm

    def forward(self, x, residual=None, yq=None, sy=None):
        y, z = self.norm(x, residual)
        return y * 4, z


class _Scaled(RMSNorm):
    """Writes the codes, and returns another y than theirs."""

    def forward(self, x, residual=None, yq=None, sy=None):
        y, z = super().forward(x, residual, yq, sy)
        return y * 4, z


def _in_place(module, args, out):
    with torch.no_grad():
        out[0].mul_(4)


CHANGES = {
    "a hook that returns another y": lambda l: l.norm.register_forward_hook(lambda m, a, o: (o[0] * 4, o[1])),
    "a hook that writes into y": lambda l: l.norm.register_forward_hook(_in_place),
    "a hook that leaves the code buffers out": lambda l: l.norm.register_forward_pre_hook(lambda m, a: a[:2]),
    "another module": lambda l: setattr(l, "norm", _OtherNorm(l.norm)),
    "a subclass": lambda l: setattr(l.norm, "__class__", _Scaled),
    "a hook that only looks": lambda l: l.norm.register_forward_hook(lambda m, a, o: None),
}


@pytest.mark.parametrize("precision", ["fp8", "fp8_dgrad"])
@pytest.mark.parametrize("change", CHANGES)
def test_fp8_block_computes_from_the_y_that_its_norm_returns(change, precision):
    """Whatever a hook or a module in the norm's place makes of y, the experts run on that y: the same
    bits as a layer without a norm that is given it (where the norm's own y comes back, its codes
    are one rounding nearer to the unrounded y than that layer's, two steps of E4M3 at most)."""
    torch.manual_seed(5)
    kw = dict(d=256, E=8, k=2, f=128, f_shared=128, precision=precision)
    layer, plain = MoELayer(norm_eps=1e-6, **kw), MoELayer(**kw)
    plain.load_state_dict({n: t for n, t in layer.state_dict().items() if not n.startswith("norm.")})
    x = torch.randn(200, 256, device="cuda").to(torch.bfloat16)
    layer(x.flip(0))  # the code buffers hold an earlier step's
    CHANGES[change](layer)
    out, z = layer(x)
    y = layer._last_plan.x
    want = plain(y)
    torch.cuda.synchronize()
    assert z is x
    if change == "a hook that only looks":
        yq, sy = torch.empty_like(layer._last_plan.x8), torch.empty_like(layer._last_plan.sx)
        layer.norm(x, None, yq, sy)
        torch.cuda.synchronize()
        assert torch.equal(layer._last_plan.x8, yq) and torch.equal(layer._last_plan.sx, sy)
        assert _off(out, want) <= REL_FP8
    else:
        assert torch.equal(layer._last_plan.x8, plain._last_plan.x8)
        assert torch.equal(layer._last_plan.sx, plain._last_plan.sx)
        assert torch.equal(out, want)


def test_fp8_block_in_inference_mode_computes_from_the_y_of_its_norm():
    torch.manual_seed(6)
    layer = MoELayer(256, 8, 2, 128, precision="fp8", norm_eps=1e-6)
    plain = MoELayer(256, 8, 2, 128, precision="fp8")
    plain.load_state_dict({n: t for n, t in layer.state_dict().items() if not n.startswith("norm.")})
    x = torch.randn(64, 256, device="cuda").to(torch.bfloat16)
    own, _ = layer(x)
    plain(x)  # (the plans have their buffers)
    with torch.inference_mode():  # the norm's codes, as in training
        assert torch.equal(layer(x)[0], own)
    layer.norm.register_forward_hook(_in_place)
    with torch.inference_mode():
        out, _ = layer(x)
        want = plain(layer._last_plan.x)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("scale", [2.5, -2.5])
def test_plan_with_fp8_data_gradients_and_gates_of_either_sign(scale):
    """The codes that the expert backward reads are those of the rows, for small gradients too."""
    torch.manual_seed(7)
    T, d, E, k, f = 300, 256, 16, 4, 128
    plan = MoEPlan(MoEShape(T, d, E, k, f, seq_len=T, fp8=True, fp8_dgrad=True, n_group=4, topk_group=2,
                            gate_scale=scale))
    dev = dict(device="cuda")
    bf = dict(dtype=torch.bfloat16)
    W = (torch.randn(E, d, **dev) / 16, torch.rand(E, **dev) * 0.1, torch.randn(E, f, d, **dev).to(**bf) / 16,
         torch.randn(E, f, d, **dev).to(**bf) / 16, torch.randn(E, d, f, **dev).to(**bf) / 16)
    x, dY = torch.randn(T, d, **dev).to(**bf), (torch.randn(T, d, **dev) * 2.0 ** -12).to(**bf)
    plan.forward(x, *W)
    plan.backward(dY)
    n = int(plan.row_offsets[-1])
    q, s = torch.empty_like(plan.dYq), torch.empty_like(plan.sdY)
    ops.moe_quantize_rows_fp8(plan.dY_perm, plan.row_offsets[E:], q, s)
    torch.cuda.synchronize()
    assert (plan.topk_gate * scale > 0).all()
    assert torch.equal(plan.sdY[:n], s[:n]) and torch.equal(plan.dYq[:n], q[:n])


def _view(t, byte):
    """The same values in a contiguous view that starts `byte` bytes past an allocation's start."""
    flat = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
    at = byte // t.element_size()
    v = flat[at:at + t.numel()].view(t.shape)
    v.copy_(t.detach())
    assert v.is_contiguous() and v.data_ptr() % 512 == byte
    return v


@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32, None])
@pytest.mark.parametrize("byte", [4, 16, 48])
def test_norm_module_takes_views_that_start_anywhere(byte, rdtype):
    """Inputs, gradients and the weight as slices of larger buffers: the same bits as from their own."""
    torch.manual_seed(8)
    T, d = 21, 264
    norm, other = RMSNorm(d), RMSNorm(d)
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    norm.w.data = w
    other.w.data = _view(w, byte)
    x, dy = (torch.randn(T, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    r, dz = ((None, None) if rdtype is None else
             (torch.randn(T, d, device="cuda").to(rdtype) for _ in range(2)))
    got = []
    for n, put in ((norm, lambda t: t.clone()), (other, lambda t: _view(t, byte))):
        xi = put(x).requires_grad_(True)
        ri = None if r is None else put(r).requires_grad_(True)
        y, z = n(xi, ri)
        if r is None:
            y.backward(put(dy))
        else:
            torch.autograd.backward([y, z], [put(dy), put(dz)])
        got.append([y.detach(), z.detach(), xi.grad, n.w.grad] + ([] if r is None else [ri.grad]))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_plan_clips_on_a_stream_with_a_norm_of_that_stream():
    """The norm's buffer comes from the stream that writes it, not from the current one, whose
    allocator may hand out memory that the current stream's kernels still use."""
    torch.manual_seed(9)
    T, d, E, f = 128, 128, 4, 128
    plan = MoEPlan(MoEShape(T, d, E, 2, f, seq_len=T))
    g = [t for n, t in plan.grads().items() if n != "dx"]
    for t in g:
        t.copy_(torch.randn(t.shape, device="cuda"))
    total = float(torch.sqrt(sum((t.double() ** 2).sum() for t in g)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm = plan.clip_grads(1.0, stream=s)
    s.synchronize()
    assert abs(float(norm[0]) - total) <= 1e-5 * total
    at = [seg["stream"] for seg in torch.cuda.memory_snapshot()
          if seg["address"] <= norm.data_ptr() < seg["address"] + seg["total_size"]]
    assert at == [s.cuda_stream]
