"""The operators together, as examples/expert_block.py uses them: one training
step of a block with experts against float64 autograd, and a short run.

The block rounds every activation and gradient it hands on to bf16 (2^-8 each);
the reference is differentiated in float64 at the block's own bf16 activations'
inputs.  A gradient passes at most six such roundings on its way (down, up,
mid, d_down, d_up, d_in, d_n), relative to sums whose terms partly cancel:
compared by norm, 2^-8 sqrt(6) is 1 %, and 3 % is allowed."""

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


def test_one_step_against_autograd():
    import expert_block as eb
    T, H, F, E = 333, 256, 200, 5
    # one step of AdamW from zero moments: m = (1 - beta1) g, so the moments give the gradients back
    hp = dict(lr=0.0, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0)
    block = eb.ExpertBlock(T, H, F, E, seed=3, hp=hp)
    torch.manual_seed(1)
    x, res = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
    dout = torch.randn(T, H, device="cuda")
    w1, w2, norm, router = (t.double().requires_grad_() for t in (block.w1, block.w2, block.norm, block.router))
    out = block.forward(x, res)
    stream = block.h.double().requires_grad_()
    n = stream * (stream.square().mean(1, keepdim=True) + eb.EPS).rsqrt() * norm
    probs = (n @ router.t()).softmax(1)
    share = probs.gather(1, block.chosen)
    ref = stream
    for k in range(eb.TOP):
        e = block.chosen[:, k]
        up = torch.einsum("th,tfh->tf", n, w1[e])
        ref = ref + share[:, k:k + 1] * torch.einsum("tf,thf->th", torch.nn.functional.silu(up), w2[e])
    assert _off(out, ref.detach()) < 0.03
    ref.backward(dout.double())
    before = block.w1.clone(), block.w2.clone()
    dx = block.backward_step(dout)
    api.forge_get_device_status()
    assert torch.equal(block.w1, before[0]) and torch.equal(block.w2, before[1])  # lr 0
    g = 1.0 / (1.0 - hp["beta1"])
    assert _off(block.m2.float() * g, w2.grad) < 0.03
    assert _off(block.m1.float() * g, w1.grad) < 0.03
    assert _off(block.d_norm, norm.grad) < 0.03
    assert _off(block.d_router, router.grad) < 0.03
    assert _off(dx, stream.grad) < 0.03


def test_the_loss_falls():
    import expert_block as eb
    losses = eb.train(steps=25, tokens=515, hidden=256, ff=128, experts=6)
    assert losses[-1] < 0.5 * losses[0], losses
