"""The gated products, the codes and their product together, as
examples/gated_block.py uses them: one training step against float64 autograd.

With what is kept in bf16 a gradient passes at most six roundings of 2^-8 on its
way (n, gu, y, dz, dGU, dn), over sums whose terms partly cancel: by norm 2^-8
sqrt(6) is 1 %, and 3 % is allowed.  In 8 bits three of them are of 2^-4 at most
(n, G and U; the backward pass reads none of the down product's codes): by norm
2^-4 sqrt(3) is 11 %, and bf16's 3 % on top.  The forward's output, beside the
stream, passes the codes of y and Wd: 2^-4 sqrt(2) is 9 %, and 3 % on top."""

import os
import sys

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api
from optimizer_tcgen05_dw_gb300.build import build

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def _off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("T,H,F", [(333, 256, 720), (20, 128, 208), (515, 512, 1408)])
def test_one_step_against_autograd(T, H, F, act, eight):
    import gated_block as gb
    # one step of AdamW from zero moments: m = (1 - beta1) g, so the moments give the gradients back
    hp = dict(lr=0.0, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0)
    block = gb.GatedBlock(T, H, F, act, eight, seed=3, hp=hp)
    torch.manual_seed(1)
    x, dout = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda")
    w, wd, norm, xd = (t.double().requires_grad_() for t in (block.w, block.wd, block.norm, x))
    out = block.forward(x)
    n = xd * (xd.square().mean(1, keepdim=True) + gb.EPS).rsqrt() * norm
    gu = n @ w.t()
    gate = torch.nn.functional.silu(gu[:, :F]) if act == "silu" else torch.nn.functional.gelu(gu[:, :F], approximate="tanh")
    z = (gate * gu[:, F:]) @ wd.t()
    ref = xd + z
    assert _off(out - x.float(), z.detach()) < (0.12 if eight else 0.03)
    ref.backward(dout.double())
    before = block.w.clone(), block.wd.clone()
    dx = block.backward_step(dout)
    api.forge_get_device_status()
    assert torch.equal(block.w, before[0]) and torch.equal(block.wd, before[1])  # lr 0
    g, room = 1.0 / (1.0 - hp["beta1"]), 0.14 if eight else 0.03
    assert _off(block.md * g, wd.grad) < room
    assert _off(block.m * g, w.grad) < room
    assert _off(block.d_norm, norm.grad) < room
    assert _off(dx, xd.grad) < room


@pytest.mark.parametrize("eight", [False, True])
def test_the_step_captured_in_a_graph(eight):
    """Forward and backward captured and replayed give the direct calls' gradients (lr 0: the weights stay)."""
    import gated_block as gb
    hp = dict(lr=0.0, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0)  # the moments are the gradients
    a, b = (gb.GatedBlock(130, 256, 336, "silu", eight, seed=3, hp=hp) for _ in range(2))
    x, dout = torch.randn(130, 256, device="cuda").bfloat16(), torch.randn(130, 256, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = a.forward(x)
        a.backward_step(dout)
    for _ in range(2):
        x.copy_(torch.randn(130, 256, device="cuda").bfloat16())
        dout.copy_(torch.randn(130, 256, device="cuda"))
        graph.replay()
        want = b.forward(x)
        b.backward_step(dout)
        torch.cuda.synchronize()
        for s, t in ((out, want), (a.dx, b.dx), (a.m, b.m), (a.md, b.md), (a.d_norm, b.d_norm)):
            assert torch.equal(s, t)


@pytest.mark.parametrize("eight", [False, True])
def test_the_example_runs(eight):
    import gated_block as gb
    losses = gb.train(steps=3, tokens=200, hidden=128, ff=272, eight=eight)
    assert len(losses) == 3 and all(v == v and v < 1e6 for v in losses)
