"""forge_multi_opt_step against the oracle, bit for bit: the per-element
arithmetic is a fixed sequence of float32 operations, so on equal inputs every
weight, moment, code and scale must be the oracle's.  Tensors of any length
(ragged groups of eight, short last INT8 blocks, empty ones) in one table."""

import numpy as np
import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build
from oracle import linear_step as ls
from oracle import optimizers as opt
from oracle import quant, rounding

pytestmark = pytest.mark.gpu

LENGTHS = [1, 7, 8, 9, 63, 64, 65, 0, 200, 2047, 2048, 2049, 4096 + 13, 70001]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def _bits(t):
    return inputs.bf16_to_bits(t)


class Set:
    """Tensors of the given lengths with random contents, and the oracle's step on them."""

    def __init__(self, lengths, w_dtype, g_dtype, s_dtype, rule, block=64, seed=5):
        self.lengths, self.w_dtype, self.s_dtype, self.block = lengths, w_dtype, s_dtype, block
        self.kind = opt.NAMES.index(rule)
        self.rule, self.hp = rule, dict(inputs.SWEEP_HPARAMS[rule], weight_decay=0.1)
        self.w, self.g, self.s1, self.s2, self.a1, self.a2 = [], [], [], [], [], []
        u1, u2 = opt.USES_S1[self.kind], opt.USES_S2[self.kind]
        for i, n in enumerate(lengths):
            k = seed + 10 * i
            self.w.append(inputs.normal((n,), 0.02, k, torch.bfloat16 if w_dtype == "bf16" else torch.float32))
            self.g.append(inputs.normal((n,), 1e-2, k + 1, torch.bfloat16 if g_dtype == "bf16" else torch.float32))
            m, v = inputs.normal((n,), 1e-3, k + 2, torch.float32), inputs.abs_normal((n,), 1e-5, k + 3)
            if s_dtype == "int8":
                pad = -n % block
                mc, ma = quant.quantize_blocks(np.pad(m.numpy(), (0, pad))[None], True, block)
                vc, va = quant.quantize_blocks(np.pad(v.numpy(), (0, pad))[None], False, block)
                m, v = torch.from_numpy(mc[0, :n].copy()), torch.from_numpy(vc[0, :n].copy())
                self.a1.append(torch.from_numpy(ma[0].copy()) if u1 else None)
                self.a2.append(torch.from_numpy(va[0].copy()) if u2 else None)
            else:
                if s_dtype == "bf16":
                    m, v = m.to(torch.bfloat16), v.to(torch.bfloat16)
                self.a1.append(None)
                self.a2.append(None)
            self.s1.append(m if u1 else None)
            self.s2.append(v if u2 else None)

    def on_gpu(self):
        up = lambda v: [None if t is None else t.cuda() for t in v]  # noqa: E731
        return [up(v) for v in (self.w, self.g, self.s1, self.s2, self.a1, self.a2)]

    def expected(self, step, seed):
        for i, n in enumerate(self.lengths):
            if n == 0:
                yield i, None
                continue
            pad = (lambda a: np.pad(a, (0, -n % self.block))[None]) if self.s_dtype == "int8" else (lambda a: a[None])
            num = lambda t: _bits(t) if t.dtype == torch.bfloat16 else t.numpy()  # noqa: E731
            row = lambda t: None if t is None else t.numpy()[None]  # noqa: E731
            st = lambda t: None if t is None else pad(num(t))  # noqa: E731
            yield i, ls.update_block(self.kind, opt.Hparams(**self.hp), step, seed + i, pad(self.g[i].float().numpy()),
                                     pad(num(self.w[i])), self.w_dtype, st(self.s1[i]), st(self.s2[i]), row(self.a1[i]),
                                     row(self.a2[i]), self.s_dtype, block=self.block)

    def check(self, gpu, step, seed):
        w, _, s1, s2, a1, a2 = gpu
        for i, ref in self.expected(step, seed):
            n = self.lengths[i]
            if ref is None:
                continue
            for name, got in (("W", w[i]), ("s1", s1[i]), ("s2", s2[i])):
                if got is None:
                    continue
                got = _bits(got) if got.dtype == torch.bfloat16 else got.cpu().numpy()
                np.testing.assert_array_equal(got, ref[name][0, :n], err_msg=f"tensor {i} (n={n}) {name}")
            for name, got in (("s1_scale", a1[i]), ("s2_scale", a2[i])):
                if got is not None:
                    np.testing.assert_array_equal(got.cpu().numpy(), ref[name][0], err_msg=f"tensor {i} (n={n}) {name}")


def _step(s, gpu, step=3, seed=77, **kw):
    table = api.make_tensors(*gpu, block=s.block, **kw)
    api.forge_multi_opt_step(table, s.rule, s.hp, step, seed)
    torch.cuda.synchronize()


@pytest.mark.parametrize("s_dtype", ["fp32", "bf16", "int8"])
@pytest.mark.parametrize("w_dtype,g_dtype", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_adamw_every_type_and_ragged_length(w_dtype, g_dtype, s_dtype):
    s = Set(LENGTHS, w_dtype, g_dtype, s_dtype, "adamw")
    gpu = s.on_gpu()
    _step(s, gpu)
    s.check(gpu, 3, 77)


@pytest.mark.parametrize("s_dtype", ["fp32", "int8"])
@pytest.mark.parametrize("rule", opt.NAMES)
def test_every_rule(rule, s_dtype):
    s = Set([5, 64, 1000], "bf16", "fp32", s_dtype, rule)
    gpu = s.on_gpu()
    _step(s, gpu)
    s.check(gpu, 3, 77)


@pytest.mark.parametrize("block", [32, 128, 256])
def test_int8_block_widths(block):
    s = Set([1, block - 1, block, block + 1, 3 * block + 5, 5000], "fp32", "fp32", "int8", "adamw", block)
    gpu = s.on_gpu()
    _step(s, gpu)
    s.check(gpu, 3, 77)


@pytest.mark.parametrize("count", [1, 56, 57, 140, 141, 480, 481, 1000])
@pytest.mark.parametrize("s_dtype", ["fp32", "int8"])
def test_table_sizes_on_either_side_of_a_launch(count, s_dtype):
    s = Set([(37 * i) % 150 if i % 7 else 2048 * (i % 3) + i % 5 for i in range(count - 1)] + [9], "bf16", "bf16", s_dtype, "adamw")
    gpu = s.on_gpu()
    _step(s, gpu)
    s.check(gpu, 3, 77)


def test_one_tensor_steps_as_the_linear_form_does():
    N, K, seed = 48, 320, 123
    s = Set([N * K], "bf16", "fp32", "int8", "adamw")
    a, b = s.on_gpu(), s.on_gpu()
    _step(s, a, seed=seed)
    shape = lambda t, c: t.view(N, c)  # noqa: E731
    w, g, s1, s2, a1, a2 = (v[0] for v in b)
    api.forge_unfused_opt_step(shape(g, K), shape(w, K), "adamw", s.hp, 3, seed, shape(s1, K), shape(s2, K),
                               shape(a1, K // 64), shape(a2, K // 64))
    for x, y in zip(a, b):
        assert torch.equal(x[0], y[0])


def test_missing_gradient_is_zero_and_no_state_rules_need_none():
    s = Set([100, 300], "fp32", "fp32", "fp32", "sgd")
    w, g, *_ = s.on_gpu()
    api.forge_multi_opt_step(api.make_tensors(w, [None, g[1]]), "sgd", dict(lr=0.5), 1, 0)
    assert torch.equal(w[0].cpu(), s.w[0])
    assert torch.equal(w[1].cpu(), s.w[1] - 0.5 * s.g[1])


def test_non_finite_gradients_stay_in_their_elements():
    s = Set([130], "bf16", "fp32", "fp32", "adamw")
    s.g[0][3], s.g[0][70], s.g[0][129] = float("nan"), float("inf"), -float("inf")
    gpu = s.on_gpu()
    _step(s, gpu)
    with np.errstate(all="ignore"):
        s.check(gpu, 3, 77)


def test_elements_past_a_tensors_end_are_left_alone():
    """Neighbours in one buffer: a ragged tensor's last group must not reach into the next one."""
    n, room = 1003, 1008
    flat = torch.full((2 * room,), 7.0, device="cuda")
    m, v = torch.zeros(2 * room, device="cuda"), torch.zeros(2 * room, device="cuda")
    g = torch.ones(2 * room, device="cuda")
    cut = lambda t: [t[:n], t[room:room + n]]  # noqa: E731
    api.forge_multi_opt_step(api.make_tensors(cut(flat), cut(g), cut(m), cut(v)), "adamw", dict(lr=1.0), 1, 0)
    gaps = torch.cat([flat[n:room], flat[room + n:]])
    assert torch.equal(gaps, torch.full_like(gaps, 7.0)) and not m[n:room].any()
    assert (flat[:n] != 7.0).all() and (flat[room:room + n] != 7.0).all()


def test_side_stream_and_graph_replay():
    s = Set([3, 5000], "bf16", "fp32", "fp32", "adamw")
    gpu = s.on_gpu()
    table = api.make_tensors(*gpu)
    side = torch.cuda.Stream()
    api.forge_multi_opt_step(table, s.rule, s.hp, 3, 77, stream=side)
    side.synchronize()
    s.check(gpu, 3, 77)
    again = s.on_gpu()
    table = api.make_tensors(*again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.forge_multi_opt_step(table, s.rule, s.hp, 3, 77)
    graph.replay()
    torch.cuda.synchronize()
    s.check(again, 3, 77)
