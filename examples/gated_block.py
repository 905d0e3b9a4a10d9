"""One gated feed-forward block, trained step by step on the library's kernels.

    x --forge_rmsnorm_fwd--> n --forge_gated_linear(W)--> y --down projection(Wd)--> out = x + z
    loss = mean((out - target)^2)

and back: forge_gated_dgrad gives the gradients of both projections from what the
forward kept, forge_linear_bwd_step updates Wd, then W (with dn from its weights
before the update), forge_rmsnorm_bwd adds the stream's gradient and
forge_multi_opt_step steps the norm's weight.  No weight gradient ever exists as
a tensor.

With --eight, what is kept between forward and backward is in 8 bits (n and both
projections as E4M3 codes: T (hidden + 2 ff) bytes and their scales, in place of
twice that and y), and the down projection multiplies codes
(forge_linear_e4m3, its weight coded anew every step).

    python examples/gated_block.py [--steps 30] [--tokens 1000] [--hidden 512] [--ff 1408] [--act silu] [--eight]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from optimizer_tcgen05_dw_gb300 import api  # noqa: E402

EPS = 1e-6


class Coded:
    """A tensor's E4M3 codes and scales (rows: 1 for activations, 128 for weights)."""

    def __init__(self, rows, cols, block_rows):
        self.block_rows = block_rows
        self.codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
        scales = rows if block_rows == 1 else -(-rows // block_rows)
        self.scale = torch.empty((scales, -(-cols // api.CODE_BLOCK)), device="cuda")

    def write(self, x):
        api.forge_quantize_e4m3(x, self.codes, self.scale, block_rows=self.block_rows)
        return self

    def read(self, x):
        api.forge_dequantize_e4m3(self.codes, self.scale, x, block_rows=self.block_rows)
        return x


class GatedBlock:
    """Weights, AdamW moments (float32) and buffers for `tokens` rows."""

    def __init__(self, tokens, hidden, ff, act="silu", eight=False, seed=0, hp=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.T, self.F, self.act, self.eight, self.seed, self.step_no = tokens, ff, act, eight, seed, 0
        self.hp = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0) if hp is None else hp
        draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        b16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.w = (draw(2 * ff, hidden) * hidden ** -0.5).bfloat16()  # the gate's rows, then the up projection's
        self.wd = (draw(hidden, ff) * ff ** -0.5).bfloat16()
        self.norm = torch.ones(hidden, device="cuda").bfloat16()
        moments = lambda t: (torch.zeros_like(t, dtype=torch.float32), torch.zeros_like(t, dtype=torch.float32))  # noqa: E731
        self.m, self.v = moments(self.w)
        self.md, self.vd = moments(self.wd)
        self.mn, self.vn = moments(self.norm)
        self.n, self.dn, self.dx, self.z = (b16(tokens, hidden) for _ in range(4))
        self.y, self.d_gu = b16(tokens, ff), b16(tokens, 2 * ff)
        self.rstd, self.d_norm = torch.empty(tokens, device="cuda"), torch.empty(hidden, device="cuda")
        self.work = torch.empty(api.forge_rmsnorm_bwd_workspace(tokens, hidden), device="cuda")
        self.rest = api.make_tensors([self.norm], [self.d_norm], [self.mn], [self.vn])
        if eight:
            self.kept_n, self.coded_y, self.coded_wd = Coded(tokens, hidden, 1), Coded(tokens, ff, 1), Coded(hidden, ff, 128)
            self.kept = dict(gu_codes=torch.empty((tokens, 2 * ff), dtype=torch.float8_e4m3fn, device="cuda"),
                             gu_scale=torch.empty((tokens, 2, -(-ff // api.CODE_BLOCK)), device="cuda"))
        else:
            self.kept = dict(gu=b16(tokens, 2 * ff))
            self.rows = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")

    def forward(self, x):
        """x + the block's output, float32 [T, hidden]."""
        self.x = x
        api.forge_rmsnorm_fwd(x, self.norm, EPS, rstd=self.rstd, y=self.n)
        api.forge_gated_linear(self.n, self.w, self.y, act=self.act, **self.kept)
        if self.eight:
            self.kept_n.write(self.n)
            y, w = self.coded_y.write(self.y), self.coded_wd.write(self.wd)
            api.forge_linear_e4m3(y.codes, y.scale, w.codes, w.scale, self.z)
        else:  # one group of all the rows
            api.forge_grouped_linear(self.y, self.wd[None], self.rows, self.z)
        return x.float() + self.z.float()

    def backward_step(self, dout):
        """Gradients of `dout` (float32 [T, hidden]) through the block and one optimizer step; the gradient of x."""
        self.step_no += 1
        dz = dout.bfloat16()
        if self.eight:  # (y and n are free between forward and backward: other blocks may use their buffers)
            self.kept_n.read(self.n)
        api.forge_gated_dgrad(dz, self.wd, self.d_gu, act=self.act, Y=self.y, **self.kept)
        step = lambda X, dY, W, m, v, seed, **kw: api.forge_linear_bwd_step(  # noqa: E731
            X, dY, W, "adamw", self.hp, self.step_no, self.seed + seed, m, v, **kw)
        step(self.y, dz, self.wd, self.md, self.vd, 0)
        step(self.n, self.d_gu, self.w, self.m, self.v, 1, dX=self.dn)
        api.forge_rmsnorm_bwd(self.dn, self.x, self.norm, self.rstd, self.dx, self.d_norm, self.work, dh=dz)
        api.forge_multi_opt_step(self.rest, "adamw", self.hp, self.step_no, self.seed + 2)
        return self.dx


def train(steps=30, tokens=1000, hidden=512, ff=1408, act="silu", eight=False, seed=0):
    """Losses of `steps` steps toward a fixed random target map."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    block = GatedBlock(tokens, hidden, ff, act, eight, seed)
    x = draw(tokens, hidden).bfloat16()
    target = x.float() + torch.tanh(x.float() @ draw(hidden, hidden) * hidden ** -0.5)
    losses = []
    for _ in range(steps):
        off = block.forward(x) - target
        losses.append(off.square().mean())
        block.backward_step(off * (2.0 / off.numel()) * 1e3)  # scaled up: AdamW does not mind, bf16 does
    api.forge_get_device_status()
    return [float(v) for v in losses]


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 30), ("tokens", 1000), ("hidden", 512), ("ff", 1408)):
        a.add_argument("--" + name, type=int, default=value)
    a.add_argument("--act", choices=list(api.ACT_KINDS), default="silu")
    a.add_argument("--eight", action="store_true")
    for i, v in enumerate(train(**vars(a.parse_args()))):
        print(f"step {i + 1:3d}  loss {v:.5f}")
