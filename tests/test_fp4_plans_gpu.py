"""Plans that a layer of 4-bit experts is made of: their backward's branches, and how long they live."""
import copy
import threading

import pytest
import torch

from oracle import moe_oracle as O
from pretraining_sigmoid_softmax_gb300 import ops
from pretraining_sigmoid_softmax_gb300.layer import MoELayer, MoEPlan, MoEShape

from gpu_common import require_gpu
from test_fp4_layer_gpu import REL, _off
from test_fp4_layer_gpu import reference as step_in_64_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _inputs(layer, T):
    W = [None if getattr(layer, n) is None else getattr(layer, n).detach()
         for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")]
    x = torch.randn(T, layer.d, device="cuda").to(torch.bfloat16)
    return x, torch.randn_like(x), W


def test_a_backward_forms_every_gradient_whatever_the_flags():
    """fp8_dgrad alone leaves the experts in bf16 and their backward with them, also where the router's
    term joins the rows (d_ff 768): the gradients are the bf16 plan's, bit for bit."""
    torch.manual_seed(1)
    layer = MoELayer(256, 8, 2, 768)
    x, dY, W = _inputs(layer, 130)
    got = {}
    for flag in (False, True):
        plan = MoEPlan(MoEShape(130, 256, 8, 2, 768, fp8_dgrad=flag))
        for g in plan.grads().values():
            g.fill_(float("nan"))
        plan.forward(x, layer.W_r.detach(), layer.b, *W)
        plan.backward(dY)
        torch.cuda.synchronize()
        got[flag] = plan.grads()
    for n, g in got[False].items():
        assert torch.isfinite(g).all() and torch.equal(got[True][n], g), n
    assert ops.moe_device_status() == (0, 0)


# ----------------------------------------------------------------- plans of held weights

def _serving(f_shared=128, **kw):
    torch.manual_seed(2)
    layer = MoELayer(256, 8, 2, 128, f_shared, precision="fp4", **kw)
    layer.hold_weights()
    return layer


def _x(T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(100 * seed + T)
    return torch.randn(T, 256, generator=g, device="cuda").to(torch.bfloat16)


def _bytes(plan):
    return sum(t.untyped_storage().nbytes() for t in plan.buffers())


@torch.no_grad()
def test_a_plan_owns_what_it_allocates():
    """buffers() are all of a plan's memory, and neither the inputs nor the weights."""
    layer = _serving()
    before = torch.cuda.memory_allocated()
    plan = MoEPlan(layer._plan(40).s, backward=False)
    del layer._plans[40, "held"]
    torch.cuda.synchronize()
    grown = torch.cuda.memory_allocated() - before
    assert _bytes(plan) <= grown <= _bytes(plan) + 512 * len(plan.buffers())  # allocations are of 512 bytes
    x, W = _x(40), [getattr(layer, n).detach() for n in ("W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")]
    n = len(plan.buffers())
    plan.forward(x, layer.W_r.detach(), layer.b, *W, weights4=layer._held)
    assert len(plan.buffers()) == n
    assert not any(t is u for t in plan.buffers() for u in [x, *W])


@torch.no_grad()
def test_batches_of_every_size_keep_a_bounded_number_of_plans():
    layer = _serving()
    want = {T: layer(_x(T)).clone() for T in (1, 2, 3)}
    one = _bytes(layer._plans[3, "held"])
    layer.HELD_PLAN_BYTES = 4 * one + one // 2
    kept = []
    for T in list(range(4, 40)) + [1, 2, 3, 2, 1]:
        out = layer(_x(T))
        if T in want:
            assert torch.equal(out, want[T])
        held = layer._held_plans()
        kept.append(len(held))
        assert held[-1][0] == (T, "held") and layer._last_plan is held[-1][1]
        assert sum(_bytes(p) for _, p in held[:-1]) <= layer.HELD_PLAN_BYTES
    assert max(kept) <= 5 and kept[-1] >= 4
    assert [k for k, _ in layer._held_plans()][-3:] == [(3, "held"), (2, "held"), (1, "held")]
    layer.HELD_PLAN_BYTES = 0
    layer(_x(50))
    assert len(layer._held_plans()) == 1


@torch.no_grad()
def test_released_weights_leave_no_plans_and_no_memory():
    layer = _serving(mode="softmax", z_coef=1e-3)
    layer.hold_weights(False)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    layer.hold_weights()
    for T in (3, 300, 5):
        layer(_x(T))
    z = layer.z_loss().clone()
    assert torch.cuda.memory_allocated() > before + _bytes(layer._plans[300, "held"])
    layer.hold_weights(False)
    torch.cuda.synchronize()
    assert layer._held is None and not layer._held_plans()
    assert torch.cuda.memory_allocated() <= before + 4096     # the losses and counts of the last forward
    assert torch.equal(layer.z_loss(), z) and layer.aux_loss() is None
    layer.hold_weights(False)                                 # nothing more to release
    layer.hold_weights()
    assert torch.equal(layer(_x(5)), layer(_x(5)))


@torch.no_grad()
def test_the_last_counts_move_the_bias_after_the_release():
    a, b = _serving(), _serving()
    a(_x(70)), b(_x(70))
    a.update_bias()
    b.hold_weights(False)
    b.update_bias()
    assert a.b.any() and torch.equal(a.b, b.b)


@torch.no_grad()
def test_captured_plans_stay():
    """A graph's buffers are not given to others while the weights are held, however many plans follow."""
    layer = _serving()
    layer.HELD_PLAN_BYTES = 0
    x = _x(9)
    layer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    for T in (1, 2, 3, 200):
        torch.full((4 << 20,), float("nan"), device="cuda")
        layer(_x(T))
    assert [k[0] for k, _ in layer._held_plans()] == [9, 200]
    for seed in (1, 2):
        x.copy_(_x(9, seed))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, layer(_x(9, seed)))
    layer.hold_weights(False)
    assert not layer._held_plans()


@torch.no_grad()
def test_dropped_plans_of_another_stream_are_not_given_away_early():
    """A forward waits on its stream while its plan is dropped and others ask for memory: its output is that
    of a forward left alone. So with its weights' codes, released meanwhile."""
    layer = _serving(f_shared=0)
    want = layer(_x(33)).clone()
    layer.HELD_PLAN_BYTES = 0
    side, x = torch.cuda.Stream(), _x(33)
    layer(_x(34))                                             # the plan of 33 is gone
    plan = layer._plan(33)                                    # made on this stream, used on another
    sizes = [t.untyped_storage().nbytes() for t in plan.buffers() + list(layer._held[0][:2])]
    del plan
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                        # 0.1 s of clock cycles
        out = layer(x)
    layer(_x(35))
    assert [k[0] for k, _ in layer._held_plans()] == [35]
    layer.hold_weights(False)
    assert not side.query()                                   # the forward is still under way
    noise = [torch.full((n,), 0x77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(noise) == 2 * len(sizes)
    assert ops.moe_device_status() == (0, 0)


def test_threads_with_batches_of_their_own_share_a_layer():
    """Four threads, each on its stream with its token counts, while plans come and go."""
    layer = _serving(f_shared=0)
    layer.HELD_PLAN_BYTES = 0
    with torch.no_grad():
        want = {T: layer(_x(T)).clone() for T in range(1, 25)}
    torch.cuda.synchronize()
    wrong = []

    def serve(first):
        try:
            with torch.no_grad(), torch.cuda.stream(torch.cuda.Stream()):
                for i in range(60):
                    T = first + 4 * (i % 6)
                    out = layer(_x(T))
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(out, want[T]):
                        wrong.append(T)
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=serve, args=(n,)) for n in (1, 2, 3, 4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert len(layer._held_plans()) == 1 and ops.moe_device_status() == (0, 0)


@torch.no_grad()
def test_a_copied_layer_has_its_own_held_weights():
    layer = _serving(f_shared=0)
    want = layer(_x(6)).clone()
    other = copy.deepcopy(layer)
    layer.hold_weights(False)
    torch.full((1 << 20,), float("nan"), device="cuda")
    assert other._held is not None and torch.equal(other(_x(6)), want)
    other.hold_weights(False)
    assert torch.equal(other(_x(6)), want)


# ------------------------------------------------------- branches of the step in 4 bits

@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("precision", ["fp4", "fp4_dgrad"])
@pytest.mark.parametrize("kw", [dict(mode="softmax", z_coef=10.0, aux_switch=100.0),
                                dict(aux_switch=100.0, aux_seq=50.0, seq_len=64, f=768),
                                dict(mode="softmax", z_coef=10.0, aux_seq=100.0, seq_len=128, f_shared=128)])
def test_router_losses_beside_4_bit_experts(kw, precision, fmt):
    """The z-loss and the balancing losses enter the router's gradient and x's, as in 64 bits; the bound
    is that of the step without them (test_fp4_layer_gpu)."""
    T, kw = 256, {"f": 128, **kw}
    torch.manual_seed(4)
    layer = MoELayer(256, 8, 2, precision=precision, fp4_format=fmt, **kw)
    x = _x(T).requires_grad_(True)
    dout = 0.02 * torch.randn_like(x)
    layer(x).backward(dout)
    torch.cuda.synchronize()
    idx = layer._last_plan.topk_idx.long()
    want, dx, grads = step_in_64_bits(layer, x.detach(), idx, dout)
    x64, W_r = x.detach().double(), layer.W_r.detach().double()
    l = x64 @ W_r.t()
    mode = O.SOFTMAX if layer.mode == ops.MODE_SOFTMAX else O.SIGMOID
    dl = torch.from_numpy(O.aux_losses_backward(l.cpu().numpy(), idx.cpu().numpy(), mode, layer.seq_len or T,
                                                layer.aux_switch, layer.aux_seq)).cuda()
    if layer.z_coef:
        dl = dl + layer.z_coef * 2 / T * torch.logsumexp(l, 1, keepdim=True) * torch.softmax(l, 1)
    alone = dl.t() @ x64
    assert alone.norm() > 4 * REL * grads["W_r"].norm()        # left out, it would be seen
    assert _off(x.grad, dx + dl @ W_r) <= REL
    grads["W_r"] = grads["W_r"] + alone
    for n, p in layer.named_parameters():
        assert _off(p.grad, grads[n]) <= REL, n


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("precision", ["fp4", "fp4_dgrad"])
def test_shared_expert_on_one_stream_or_two(precision, fmt):
    """The shared expert beside the routed ones (small layers) or behind them (large ones): the same bits."""
    torch.manual_seed(5)
    layer = MoELayer(384, 8, 2, 256, 384, precision=precision, fp4_format=fmt)
    x, dY, W = _inputs(layer, 515)
    got = []
    for overlap in (False, True):
        plan = MoEPlan(layer._plan(515).s, overlap_shared=overlap)
        assert (plan.ws_side is plan.ws) is not overlap
        for g in plan.grads().values():
            g.fill_(float("nan"))
        for _ in range(2):
            plan.forward(x, layer.W_r.detach(), layer.b, *W)
            plan.backward(dY)
        torch.cuda.synchronize()
        got.append({"out": plan.out, **plan.grads()})
    for n, t in got[0].items():
        assert torch.isfinite(t).all() and torch.equal(t, got[1][n]), n
    held = MoEPlan(layer._plan(515).s, backward=False, overlap_shared=False)
    held.forward(x, layer.W_r.detach(), layer.b, *W)
    torch.cuda.synchronize()
    assert torch.equal(held.out, got[0]["out"])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("d,f,f_shared", [(3328, 128, 0), (3456, 128, 128), (128, 1792, 0), (128, 1664, 1792)])
def test_launch_count_with_long_columns(d, f, f_shared, fmt):
    """NV columns of more than 3328 elements take three kernels each."""
    from torch.autograd import DeviceType
    from torch.profiler import ProfilerActivity, profile
    torch.manual_seed(6)
    layer = MoELayer(d, 4, 2, f, f_shared, precision="fp4_dgrad", fp4_format=fmt)
    x, dY, W = _inputs(layer, 60)
    plan = MoEPlan(layer._plan(60).s)

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
