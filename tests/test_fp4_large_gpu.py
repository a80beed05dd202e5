"""A step of the largest layer on 4-bit experts: sampled tokens' outputs and input gradients, and sampled
experts' weight gradients, in 64 bits.

Bounds. Tokens: as the small layers' (test_fp4_layer_gpu). Weight gradients against products of the stored
bf16 tensors: the rounding of the result (2^-9 of it in the mean, 2^-8 at most) and, with fp32 sums over n
rows, n 2^-24 of the sum of magnitudes, whose norm is at most sqrt(n) times that of sums of random sign."""
import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import ops
from pretraining_sigmoid_softmax_gb300.configs import C4
from pretraining_sigmoid_softmax_gb300.layer import MoEPlan, MoEShape, weights4

from gpu_common import require_gpu
from test_fp4_layer_gpu import REL, _off, bf, expert, expert_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_step_of_the_largest_layer(fmt):
    s, nv = MoEShape.from_config(C4.with_(precision="fp4_dgrad", fp4_format=fmt)), fmt == "nv"
    g = torch.Generator(device="cuda").manual_seed(7)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(std=std, generator=g)

    x, dY = randn(s.T, s.d), randn(s.T, s.d)
    W_r, b = randn(s.E, s.d, std=s.d ** -0.5, dtype=torch.float32), torch.zeros(s.E, device="cuda")
    W = [randn(s.E, s.f, s.d, std=s.d ** -0.5), randn(s.E, s.f, s.d, std=s.d ** -0.5),
         randn(s.E, s.d, s.f, std=s.f ** -0.5)]
    Ws = [randn(s.f_shared, s.d, std=s.d ** -0.5), randn(s.f_shared, s.d, std=s.d ** -0.5),
          randn(s.d, s.f_shared, std=s.f_shared ** -0.5)]
    ops.moe_clear_device_status()
    plan = MoEPlan(s)
    assert not plan.overlap and plan.router_rows
    plan.forward(x, W_r, b, *W, *Ws)
    plan.backward(dY)
    torch.cuda.synchronize()
    assert ops.moe_device_status() == (0, 0)

    tokens = torch.randperm(s.T, generator=torch.Generator().manual_seed(1))[:40].cuda()
    tokens[:2] = torch.tensor([0, s.T - 1])
    idx, xt, dout = plan.topk_idx[tokens].long(), x[tokens].double(), dY[tokens].double()
    xr = xt.clone().requires_grad_(True)
    score = torch.sigmoid(xr @ W_r.double().t()).gather(1, idx)
    gate = score / score.sum(1, keepdim=True)
    w = [t.double() for t in Ws]
    a, u, h, out = expert(xt, *w, nv)
    dx = expert_bwd(dout, xt, a, u, h, *w, nv, True)[0]
    dgate = torch.zeros_like(gate)
    for e in range(s.E):
        t, i = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        w = [m[e].double() for m in W]
        a, u, h, y = expert(xt[t], *w, nv)
        ge = gate[t, i].detach()[:, None]
        out.index_add_(0, t, ge * y)
        dgate[t, i] = (dout[t] * y).sum(1)
        dx.index_add_(0, t, expert_bwd(bf(ge * dout[t]), xt[t], a, u, h, *w, nv, True)[0])
    (gate * dgate).sum().backward()
    assert _off(plan.out[tokens], out) <= REL
    assert _off(plan.dx[tokens], dx + xr.grad) <= REL

    for e in (0, s.E - 1):
        lo, hi = plan.row_offsets[e:e + 2].tolist()
        bound = 2.0 ** -8 + (hi - lo) ** 1.5 * 2.0 ** -24
        X, H, dYp, dA, dU = (t[lo:hi].double() for t in (plan.X_perm, plan.H, plan.dY_perm, plan.dA, plan.dU))
        assert _off(plan.dW_d[e], dYp.t() @ H) <= bound
        assert _off(plan.dW_g[e], dA.t() @ X) <= bound
        assert _off(plan.dW_u[e], dU.t() @ X) <= bound

    held = MoEPlan(s, backward=False)  # the same without what a backward needs, on weights made once
    held.forward(x, W_r, b, *W, *Ws, weights4=weights4(s.fp4_format, *W, *Ws))
    torch.cuda.synchronize()
    assert torch.equal(held.out, plan.out)
    assert ops.moe_device_status() == (0, 0)
    del plan, held
    torch.cuda.empty_cache()
