"""One block with experts, trained step by step on the library's kernels.

    x, residual --forge_rmsnorm_fwd--> h (the stream), n
    n --router--> each token's two experts and their shares (torch)
    n, gathered by expert --forge_grouped_linear(W1)--> silu --forge_grouped_linear(W2)--> added back by share
    loss = mean((h + experts - target)^2)

and back: forge_grouped_bwd_step updates W2, then W1 (each gives dX from its
weights before the update), forge_rmsnorm_bwd adds the stream's gradient, and
forge_multi_opt_step steps what is left: the norm's weight and the router's.
The experts' weight gradients never exist as tensors.

    python examples/expert_block.py [--steps 30] [--tokens 1000] [--hidden 512] [--ff 384] [--experts 8]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from optimizer_tcgen05_dw_gb300 import api  # noqa: E402

EPS = 1e-6
TOP = 2  # experts a token


class ExpertBlock:
    """Weights, AdamW moments (bf16 for the experts) and buffers for `tokens` rows."""

    def __init__(self, tokens, hidden, ff, experts, seed=0, hp=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.T, self.E, self.seed, self.step_no = tokens, experts, seed, 0
        self.hp = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0) if hp is None else hp
        draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        b16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.w1 = (draw(experts, ff, hidden) * hidden ** -0.5).bfloat16()
        self.w2 = (draw(experts, hidden, ff) * ff ** -0.5).bfloat16()
        self.norm = torch.ones(hidden, device="cuda").bfloat16()
        self.router = (draw(experts, hidden) * hidden ** -0.5).bfloat16()
        self.m1, self.v1 = torch.zeros_like(self.w1), torch.zeros_like(self.w1)
        self.m2, self.v2 = torch.zeros_like(self.w2), torch.zeros_like(self.w2)
        # everything that is not an expert's: one table, built once
        self.d_norm, self.d_router = torch.zeros(hidden, device="cuda"), torch.zeros(experts, hidden, device="cuda")
        moments = [[torch.zeros_like(d) for d in (self.d_norm, self.d_router)] for _ in range(2)]
        self.rest = api.make_tensors([self.norm, self.router], [self.d_norm, self.d_router], *moments)
        self.work = torch.empty(api.forge_rmsnorm_bwd_workspace(tokens, hidden), device="cuda")
        self.h, self.n, self.dx = b16(tokens, hidden), b16(tokens, hidden), b16(tokens, hidden)
        self.rstd = torch.empty(tokens, device="cuda")
        self.up, self.mid, self.d_up = (b16(tokens * TOP, ff) for _ in range(3))
        self.down, self.d_in = b16(tokens * TOP, hidden), b16(tokens * TOP, hidden)

    def forward(self, x, residual):
        api.forge_rmsnorm_fwd(x, self.norm, EPS, residual=residual, h=self.h, rstd=self.rstd, y=self.n)
        self.probs = (self.n.float() @ self.router.float().t()).softmax(1)
        self.share, chosen = self.probs.topk(TOP, dim=1)
        order = chosen.reshape(-1).argsort(stable=True)  # token slots by expert
        self.chosen, self.order, self.token = chosen, order, order // TOP
        counts = torch.bincount(chosen.reshape(-1), minlength=self.E)
        self.offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()  # stays on the device
        self.rows = self.n[self.token]
        api.forge_grouped_linear(self.rows, self.w1, self.offsets, self.up)
        self.mid.copy_(torch.nn.functional.silu(self.up.float()))
        api.forge_grouped_linear(self.mid, self.w2, self.offsets, self.down)
        gate = self.share.reshape(-1)[order]
        return self.h.float().index_add(0, self.token, self.down.float() * gate[:, None])

    def backward_step(self, dout):
        """Gradients of `dout` (float32 [T, hidden]) through the block and one optimizer step; the gradient of x."""
        self.step_no += 1
        gate = self.share.reshape(-1)[self.order]
        d_down = (dout[self.token] * gate[:, None]).bfloat16()
        d_share = torch.zeros_like(self.share).reshape(-1)
        d_share[self.order] = (dout[self.token] * self.down.float()).sum(1)
        api.forge_grouped_bwd_step(self.mid, d_down, self.w2, self.offsets, "adamw", self.hp, self.step_no, self.seed, self.m2,
                                   self.v2, dX=self.d_up)
        up = self.up.float()
        s = torch.sigmoid(up)
        d_up = (self.d_up.float() * s * (1 + up * (1 - s))).bfloat16()
        api.forge_grouped_bwd_step(self.rows, d_up, self.w1, self.offsets, "adamw", self.hp, self.step_no, self.seed + 1,
                                   self.m1, self.v1, dX=self.d_in)
        d_probs = torch.zeros_like(self.probs).scatter(1, self.chosen, d_share.view_as(self.share))
        d_logits = self.probs * (d_probs - (self.probs * d_probs).sum(1, keepdim=True))
        self.d_router.copy_(d_logits.t() @ self.n.float())
        d_n = (d_logits @ self.router.float()).index_add(0, self.token, self.d_in.float()).bfloat16()
        api.forge_rmsnorm_bwd(d_n, self.h, self.norm, self.rstd, self.dx, self.d_norm, self.work, dh=dout.bfloat16())
        api.forge_multi_opt_step(self.rest, "adamw", self.hp, self.step_no, self.seed + 2)
        return self.dx


def train(steps=30, tokens=1000, hidden=512, ff=384, experts=8, seed=0):
    """Losses of `steps` steps toward a fixed random target map."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    block = ExpertBlock(tokens, hidden, ff, experts, seed)
    x, residual = draw(tokens, hidden).bfloat16(), draw(tokens, hidden).bfloat16()
    h = x.float() + residual.float()
    target = h + torch.tanh(h @ draw(hidden, hidden) * hidden ** -0.5)
    losses = []
    for _ in range(steps):
        off = block.forward(x, residual) - target
        losses.append(off.square().mean())
        block.backward_step(off * (2.0 / off.numel()) * 1e3)  # scaled up: AdamW does not mind, bf16 does
    api.forge_get_device_status()
    return [float(v) for v in losses]


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 30), ("tokens", 1000), ("hidden", 512), ("ff", 384), ("experts", 8)):
        a.add_argument("--" + name, type=int, default=value)
    for i, v in enumerate(train(**vars(a.parse_args()))):
        print(f"step {i + 1:3d}  loss {v:.5f}")
