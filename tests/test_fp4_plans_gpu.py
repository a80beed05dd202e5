"""Plans that a layer of 4-bit experts is made of: their backward's branches, and how long they live."""
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops
from pretraining_sigmoid_softmax_gb300.layer import MoELayer, MoEPlan, MoEShape

from gpu_common import require_gpu

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
