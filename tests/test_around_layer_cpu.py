"""The argument checks of the operators around the layer (norm, router logits, choice of
experts, gradient clipping): what they refuse, they refuse on the host, before any device work,
so the checks hold without a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from pretraining_sigmoid_softmax_gb300 import _lib, build, layer, ops

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not installed")
P = 4096       # a stand-in device address (never dereferenced on the host), 16-byte aligned
BAD = P + 2    # not 16-byte aligned
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return _lib.load()


@needs_nvcc
def test_norm_refusals(lib):
    def fwd(x=P, res=P, rt=0, w=P, eps=1e-6, T=4, d=256, z=P, y=P, yq=None, sy=None, rstd=P):
        return lib.moe_rms_norm(x, res, rt, w, eps, T, d, z, y, yq, sy, rstd, None)
    assert fwd(x=None) == fwd(w=None) == INVALID
    assert fwd(y=None) == INVALID                                # neither y nor codes
    assert fwd(res=None) == fwd(z=None) == INVALID               # residual and z come together
    assert fwd(yq=P) == fwd(sy=P) == INVALID                     # codes and scales come together
    assert fwd(T=0) == fwd(d=0) == fwd(T=-1) == INVALID
    assert fwd(eps=-1.0) == fwd(eps=float("nan")) == INVALID
    assert fwd(rt=2) == INVALID
    assert fwd(d=260) == fwd(d=32776) == fwd(T=1 << 31) == UNSUPPORTED
    assert fwd(x=BAD) == fwd(res=BAD) == fwd(w=BAD) == fwd(z=BAD) == fwd(y=BAD) == INVALID
    assert fwd(yq=P + 4, sy=P) == INVALID

    def bwd(dy=P, dres=P, z=P, rt=0, rstd=P, w=P, T=4, d=256, dz=P, dx=None, dw=P, ws=P,
            wb=1 << 20):
        return lib.moe_rms_norm_bwd(dy, dres, z, rt, rstd, w, T, d, dz, dx, dw, ws, wb, None)
    assert {bwd(dy=None), bwd(z=None), bwd(rstd=None), bwd(w=None), bwd(dz=None),
            bwd(dw=None)} == {INVALID}
    assert bwd(T=0) == bwd(d=0) == bwd(rt=-1) == INVALID
    assert bwd(d=12) == bwd(d=32776) == UNSUPPORTED
    assert {bwd(dy=BAD), bwd(dres=BAD), bwd(z=BAD), bwd(w=BAD), bwd(dz=BAD), bwd(dx=BAD)} == {INVALID}
    assert bwd(ws=None) == bwd(ws=BAD) == bwd(wb=4 * 256 * 4 - 1) == WORKSPACE


@needs_nvcc
def test_router_logits_and_weight_gradient_refusals(lib):
    def logits(x=P, W=P, T=16, d=256, E=8, out=P, ws=P, wb=1 << 20):
        return lib.moe_router_logits(x, W, T, d, E, 0.0, out, None, None, ws, wb, None)
    assert logits(x=None) == logits(W=None) == logits(out=None) == INVALID
    assert logits(T=0) == logits(d=0) == logits(E=0) == INVALID
    assert logits(E=257) == logits(d=200) == UNSUPPORTED
    assert logits(x=BAD) == logits(W=BAD) == INVALID
    assert logits(ws=None) == logits(wb=64) == WORKSPACE

    def dw(dl=P, x=P, T=16, d=256, E=8, out=P, ws=P, wb=1 << 20):
        return lib.moe_router_dw(dl, x, T, d, E, out, ws, wb, None)
    assert dw(dl=None) == dw(x=None) == dw(out=None) == INVALID
    assert dw(T=0) == dw(d=0) == dw(E=0) == INVALID
    assert dw(E=257) == dw(d=200) == UNSUPPORTED
    assert dw(x=BAD) == dw(out=BAD) == INVALID
    assert dw(ws=None) == dw(wb=64) == WORKSPACE


@needs_nvcc
def test_choice_refusals(lib):
    def sel(l=P, b=None, T=4, E=64, k=8, mode=0, G=8, tg=4, rule=1, idx=P, gate=P, score=P):
        return lib.moe_select_experts(l, b, T, E, k, mode, G, tg, rule, 1, 1.0, idx, gate, score,
                                      None, None)
    assert sel(l=None) == sel(idx=None) == sel(gate=None) == sel(score=None) == INVALID
    assert sel(T=0) == sel(E=0) == sel(k=0) == sel(G=0) == sel(tg=0) == INVALID
    assert sel(mode=2) == sel(rule=2) == INVALID
    assert sel(tg=9) == INVALID                        # more groups kept than there are
    assert sel(E=60, G=8) == INVALID                   # groups of unequal size
    assert sel(k=9, G=8, tg=1) == INVALID              # fewer experts left than chosen
    assert sel(E=264, G=8) == UNSUPPORTED              # too many experts
    assert sel(E=4, k=5, G=1, tg=1) == UNSUPPORTED     # more chosen than there are
    assert sel(E=256, k=33, G=1, tg=1) == UNSUPPORTED
    assert sel(E=64, k=8, G=64, tg=32) == UNSUPPORTED  # too many groups

    def bwd(dg=P, idx=P, score=P, l=P, lse=P, T=4, E=64, k=8, mode=0, renorm=1, z=0.0, out=P):
        return lib.moe_select_experts_bwd(dg, idx, score, l, lse, None, T, E, k, mode, renorm, 1.0,
                                          z, out, None)
    assert bwd(dg=None) == bwd(idx=None) == bwd(score=None) == bwd(out=None) == INVALID
    assert bwd(T=0) == bwd(E=0) == bwd(k=0) == bwd(mode=5) == INVALID
    assert bwd(z=1e-3) == INVALID                                   # a z-loss needs softmax scores
    assert bwd(mode=1, renorm=0, l=None) == bwd(mode=1, renorm=0, lse=None) == INVALID
    assert bwd(mode=1, z=1e-3, lse=None) == INVALID
    assert bwd(E=257) == bwd(E=4, k=5) == bwd(k=33) == UNSUPPORTED


def _arrays(ptrs, numel, types):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int * n)(*types))


@needs_nvcc
def test_clip_refusals(lib):
    def clip(grads=(P,), out=None, numel=(64,), types=(1,), count=None, max_norm=1.0, norm=P, ws=P,
             wb=1 << 20):
        g, n, t = _arrays(grads, numel, types)
        o = g if out is None else _arrays(out, numel, types)[0]
        c = len(grads) if count is None else count
        return lib.moe_clip_grads(g, o, n, t, c, max_norm, norm, ws, wb, None)
    assert clip(count=0) == clip(count=-1) == INVALID
    assert clip(norm=None) == clip(max_norm=-1.0) == clip(max_norm=float("nan")) == INVALID
    assert clip(types=(2,)) == clip(numel=(-1,)) == INVALID
    assert clip(grads=(None,)) == INVALID
    assert clip(grads=(P + 2,)) == INVALID                          # fp32 off its own alignment
    assert clip(grads=(P + 1,), types=(0,)) == INVALID
    assert clip(grads=(P,), out=(None,)) == INVALID
    assert clip(ws=None) == clip(ws=BAD) == clip(wb=128) == WORKSPACE
    two = dict(numel=(64, 64), types=(1, 1))
    assert clip(grads=(P, P), **two) == INVALID                     # the same tensor twice, in place
    assert clip(grads=(P, P + 128), **two) == INVALID               # tensors that overlap
    far = 1 << 20
    assert clip(grads=(P, far), out=(2 * far, 2 * far), **two) == INVALID      # one output twice
    assert clip(grads=(P, far), out=(far, 2 * far), **two) == INVALID          # another's gradient
    assert clip(grads=(P, far), out=(P + 64, 2 * far), **two) == INVALID       # shifted in place
    assert lib.moe_clip_grads(*_arrays((P,), (4,), (1,))[:1], None, *_arrays((P,), (4,), (1,))[1:],
                              1, 1.0, P, P, 1 << 20, None) == INVALID
    # what only reads may name a tensor twice: the refusal then comes from the missing device
    g, n, t = _arrays((P, P), (64, 64), (1, 1))
    assert lib.moe_grad_norm(g, n, t, 2, 1.0, P, P, 128, None) == WORKSPACE


@needs_nvcc
def test_workspace_covers_the_operators(lib):
    for T, d in [(1, 8), (5, 1000), (65536, 4096), (700, 32768)]:
        assert lib.moe_workspace_bytes(T, d, 1, 1) >= min(T, 608) * d * 4


def test_binding_refuses_wrong_tensors():
    """Types, shapes, layouts and devices are checked before the library is called."""
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x, w = torch.zeros(4, 16, dtype=bf), torch.ones(16)
    y = torch.empty_like(x)
    bad = [
        (lambda: ops.moe_rms_norm(x, None, w, 1e-6, None, y), "CUDA tensor"),
        (lambda: ops.moe_rms_norm(x.float(), None, w, 1e-6, None, y), "x must be torch.bfloat16"),
        (lambda: ops.moe_rms_norm(x.t(), None, w, 1e-6, None, y), "contiguous"),
        (lambda: ops.moe_rms_norm(x[0], None, w, 1e-6, None, y), "2-D"),
        (lambda: ops.moe_rms_norm(x[:0], None, w, 1e-6, None, y), "at least one row"),
    ]
    for call, says in bad:
        with pytest.raises(ops.MoEError, match=says):
            call()
    with pytest.raises(ops.MoEError, match="CUDA tensor"):
        ops.moe_select_experts(torch.zeros(4, 8), None, 2, ops.MODE_SIGMOID, 1, 1, ops.GROUP_MAX,
                               True, 1.0, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2),
                               torch.zeros(4, 2))
    with pytest.raises(ops.MoEError, match="CUDA tensor"):
        ops.moe_select_experts_bwd(torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32),
                                   torch.zeros(4, 2), None, None, ops.MODE_SIGMOID, True, 1.0,
                                   torch.zeros(4, 8))
    ws, norm = torch.zeros(16384, dtype=u8), torch.zeros(2)
    with pytest.raises(ops.MoEError, match="CUDA tensor"):
        ops.moe_clip_grads([torch.zeros(4)], 1.0, None, norm, ws)
    with pytest.raises(ops.MoEError, match="bf16 or fp32"):
        ops.moe_grad_norm([torch.zeros(4, dtype=torch.float64)], 1.0, norm, ws)
    with pytest.raises(ops.MoEError, match="CUDA tensor"):
        ops.moe_router_logits(x, torch.zeros(2, 16), torch.zeros(4, 2), ws)
    with pytest.raises(ops.MoEError, match="CUDA tensor"):
        ops.moe_router_dw(torch.zeros(4, 2), x, torch.zeros(2, 16), ws)
    with pytest.raises(ops.MoEError, match="CUDA tensor"):
        ops.moe_rms_norm_bwd(x, None, x, torch.zeros(4), w, y, None, torch.zeros(16), ws)


@needs_nvcc
def test_router_entries_refuse_a_misaligned_workspace(lib):
    """Their sums and pieces are read as whole vectors."""
    assert lib.moe_router_logits(P, P, 16, 256, 8, 0.0, P, None, None, BAD, 1 << 20, None) == WORKSPACE
    assert lib.moe_router_dw(P, P, 16, 256, 8, P, BAD, 1 << 20, None) == WORKSPACE


def test_binding_names_the_missing_tensor():
    """The first wrong argument is the one that is named, whatever the workspace is."""
    with pytest.raises(ops.MoEError, match="norm is missing"):
        ops.moe_clip_grads([torch.zeros(4)], 1.0, None, None, torch.zeros(16384, dtype=torch.uint8))
    with pytest.raises(ops.MoEError, match="norm is missing"):
        ops.moe_grad_norm([torch.zeros(4)], 1.0, None, torch.zeros(16384, dtype=torch.uint8))
    x, ws = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(16384, dtype=torch.uint8)
    with pytest.raises(ops.MoEError, match="dy must be a CUDA tensor"):
        ops.moe_rms_norm_bwd(x, None, x, torch.zeros(4), torch.ones(16), x, None, torch.zeros(16), ws)
    with pytest.raises(ops.MoEError, match="x must be a CUDA tensor"):
        ops.moe_router_logits(x, torch.zeros(2, 16), torch.zeros(4, 2), ws)
    with pytest.raises(ops.MoEError, match="dlogits must be a CUDA tensor"):
        ops.moe_router_dw(torch.zeros(4, 2), x, torch.zeros(2, 16), ws)


KEYS_CPP = r"""
#include <stdio.h>
#include <string.h>
#include "select_key.h"
using namespace moe;
int main() {
    int last = INT_MIN;
    for (long u = 0; u < 8388608; u += u < 64 || u > 8388544 ? 1 : 4093) {
        const float v = (float)(1.0 + (double)u / kUnits);
        uint32_t bits;
        memcpy(&bits, &v, 4);
        for (int e = 0; e < 256; e += 51) {
            const int key = key_of(bits, INT_MIN + 1 + e);
            if (key <= last || units_of(key) != u || expert_of(key) != e) return printf("%ld %d %d\n", u, e, key), 1;
            last = key;
        }
    }
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_choice_keys_are_defined_arithmetic(tmp_path):
    """The keys order values and hold value and expert, in arithmetic that C++ defines throughout."""
    src, exe = tmp_path / "keys.cpp", tmp_path / "keys"
    src.write_text(KEYS_CPP)
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", csrc,
                    str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr


@needs_nvcc
def test_clip_grad_norm_hands_over_runs_of_memory(lib, monkeypatch):
    """Gradients whose dimensions lie in another order are handed over as the memory they are; ones
    with gaps, or with one element many times, are refused before anything is launched."""
    seen = []
    monkeypatch.setattr(layer.ops, "moe_clip_grads", lambda grads, *a: seen.append(grads))

    def clip(*grads):
        ps = [torch.nn.Parameter(torch.zeros(g.shape)) for g in grads]
        for p, g in zip(ps, grads):
            p.grad = g
        layer.clip_grad_norm_(ps, 1.0)
    base = torch.arange(210.0)
    orders = [base.view(14, 15).t(), base.view(5, 6, 7).permute(2, 0, 1), base.view(2, 3, 5, 7).permute(0, 3, 1, 2),
              base.view(14, 1, 15).permute(2, 1, 0), base[3:203].view(10, 20).t(), base.view(210, 1)]
    clip(*orders)
    for got, g in zip(seen[0], orders):
        assert got.is_contiguous() and got.data_ptr() == g.data_ptr() and got.numel() == g.numel()
        assert sorted(got.flatten().tolist()) == sorted(g.flatten().tolist())
    seen.clear()
    for g in (base.view(14, 15)[:, ::2], base.view(14, 15)[:, :5], base[:8].expand(4, 8),
              base.as_strided((4, 5), (3, 1)), base.as_strided((4, 5), (1, 6))):
        with pytest.raises(ops.MoEError, match=r"gradient 1 .*side by side"):
            clip(base, g)
    assert not seen


@needs_nvcc
def test_clip_grad_norm_runs_on_the_gradients_device(lib, monkeypatch):
    """The library's call is made with the gradients' device as the current one, whichever was."""
    current = [0]

    class DeviceOf:
        def __init__(self, t):
            self.to = 1  # where these stand-ins for gradients are said to lie
            assert t.shape == (2,)

        def __enter__(self):
            self.was, current[0] = current[0], self.to

        def __exit__(self, *a):
            current[0] = self.was
    calls = []
    monkeypatch.setattr(torch.cuda, "device_of", DeviceOf)
    monkeypatch.setattr(layer.ops, "moe_clip_grads", lambda g, m, out, norm, ws: (calls.append(current[0]), norm.fill_(3)))
    p = torch.nn.Parameter(torch.zeros(4))
    p.grad = torch.ones(4)
    assert float(layer.clip_grad_norm_(p, 1.0)) == 3.0
    assert calls == [1] and current == [0]


class _Returns(torch.nn.Module):
    def __init__(self, change):
        super().__init__()
        self.change = change

    def forward(self, x, residual=None, yq=None, sy=None):
        return self.change(x), x


@needs_nvcc
@pytest.mark.parametrize("precision", ["bf16", "fp8"])
@pytest.mark.parametrize("change", [lambda x: x.float(), lambda x: x[:4], lambda x: x[:, :128], lambda x: x[0],
                                    lambda x: x.half(), lambda x: x.to("meta")])
def test_layer_refuses_another_kind_of_y_from_its_norm(lib, change, precision):
    """The kernels read [T, d] bf16 at the address they are given, whatever lies there."""
    block = layer.MoELayer(256, 4, 2, 128, norm_eps=1e-6, device="cpu", precision=precision)
    block.norm = _Returns(change)
    with pytest.raises(ValueError, match="the norm must return"):
        block(torch.zeros(8, 256, dtype=torch.bfloat16))
