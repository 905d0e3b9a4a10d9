"""INT8 optimizer states with absmax blocks of 32, 128 and 256 row elements
on the GPU (block 64, the pages' size, is covered by every other INT8 test).

The explainer's Technical Summary §2 "Precision and Fidelity" sets FORGE's
block of 64 against the 2048 of standard 8-bit optimizers; the widths built
here are those that stay inside one 256-column tile pair, so a tile's
requantisation needs only its own new moments.  Each width is checked bit for
bit on integer-grid inputs (every FP32 sum exact) in every kernel that steps
INT8 states: the fused step with staged weights (T <= 8192) and with direct
weights (T > 8192), the one-launch step with dX, the last-wave column halves,
the E4M3 step, the unfused optimizer kernel and the quantiser helpers; and on
realistic data through the interval oracle.
"""

import numpy as np
import pytest
import torch

from oracle import fp8
from oracle import linear_step as ls
from oracle import quant
from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build

from _helpers import Problem, assert_bitexact, assert_dx_close, oracle_hparams, to_bits

pytestmark = pytest.mark.gpu

BLOCKS = [32, 128, 256]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()
    api.forge_set_wait_limit_ns(200_000_000)
    api.forge_debug_skip_loads(False)
    api.forge_set_step_fusion(True)
    yield
    api.forge_set_wait_limit_ns(0)


def _hp(name):
    hp = dict(inputs.SWEEP_HPARAMS[name])
    hp.setdefault("weight_decay", 0.01)  # the coupled rules' moments then depend on W
    return hp


def _compare_exact(gpu, ref, what=""):
    assert_bitexact(gpu["W"], ref["W"], what + "W")
    for k in ("s1", "s2", "s1_scale", "s2_scale"):
        if ref.get(k) is not None:
            assert_bitexact(gpu[k], ref[k], what + k)


@pytest.mark.parametrize("qb", BLOCKS)
@pytest.mark.parametrize("opt_name", ["adamw", "lion", "rmsprop", "nadam"])
@pytest.mark.parametrize("case", ["staged_w", "one_launch", "direct_w"])
def test_int8_blocks_bitexact_on_integer_grid(case, opt_name, qb):
    """Two steps from pre-warmed INT8 moments; K spans several blocks and
    ragged tiles (N % 256, K % 256 != 0 where the width allows)."""
    K = {32: 320, 128: 384, 256: 768}[qb]
    T = 8256 if case == "direct_w" else 200  # above 8192 the epilogue reads W directly
    N = 136 if case == "direct_w" else 320
    prob = Problem(T=T, N=N, K=K, w_dtype="bf16", s_dtype="int8", opt_name=opt_name,
                   hp=_hp(opt_name), grid=True, steps=2, seed=31 + qb, qblock=qb)
    want_dx = case == "one_launch"
    gpu, gdx = prob.run_gpu(fused=True, want_dx=want_dx)
    ref, _, _ = prob.run_oracle()
    _compare_exact(gpu, ref)
    if want_dx:
        assert_dx_close(gdx[0], to_bits(prob.dY[0]), prob.state0["W"], "dX")


@pytest.mark.parametrize("qb", [32, 128])
def test_int8_blocks_split_last_wave_bitexact(qb):
    """80 pair tiles on 76 pairs: the last wave runs as 128-column halves (a
    128-column block is whole in a half; 256 disables the split)."""
    prob = Problem(T=144, N=2560, K=2048, w_dtype="bf16", s_dtype="int8", opt_name="adamw",
                   hp=_hp("adamw"), grid=True, steps=1, seed=41, qblock=qb)
    gpu, _ = prob.run_gpu(fused=True)
    ref, _, _ = prob.run_oracle()
    _compare_exact(gpu, ref)


@pytest.mark.parametrize("qb", BLOCKS)
@pytest.mark.parametrize("opt_name", ["adamw", "sgd_momentum", "adagrad"])
def test_int8_blocks_unfused_and_zero_tokens_bitexact(opt_name, qb):
    """The separate optimizer kernel (the unfused schedule, and the T = 0
    step) shares a block's absmax over qb/8 lanes."""
    prob = Problem(T=200, N=264, K=512, w_dtype="bf16", s_dtype="int8", opt_name=opt_name,
                   hp=_hp(opt_name), grid=True, steps=2, seed=51 + qb, qblock=qb)
    gpu, _ = prob.run_gpu(fused=False)
    ref, _, _ = prob.run_oracle()
    _compare_exact(gpu, ref)
    # T = 0: the rule on a zero gradient through forge_linear_bwd_step
    st = prob.gpu_state()
    X0 = torch.empty((0, prob.K), dtype=torch.bfloat16, device="cuda")
    dY0 = torch.empty((0, prob.N), dtype=torch.bfloat16, device="cuda")
    api.forge_linear_bwd_step(X0, dY0, st["W"], opt_name, prob.hp, 1, prob.seed, st.get("s1"),
                              st.get("s2"), st.get("s1_scale"), st.get("s2_scale"))
    api.forge_get_device_status()
    s0 = prob.state0
    ref0 = ls.update_block(prob.kind, oracle_hparams(prob.hp), 1, prob.seed,
                           np.zeros((prob.N, prob.K), np.float32), s0["W"], "bf16", s0.get("s1"),
                           s0.get("s2"), s0.get("s1_scale"), s0.get("s2_scale"), "int8", 0, 0,
                           prob.K, block=qb)
    _compare_exact(st, ref0, "T=0 ")


@pytest.mark.parametrize("qb", BLOCKS)
def test_int8_blocks_fp8_step_bitexact(qb):
    """The E4M3 step's staged epilogue with each block width."""
    T, N, K = 208, 320, {32: 384, 128: 384, 256: 512}[qb]
    prob = Problem(T=T, N=N, K=K, w_dtype="bf16", s_dtype="int8", opt_name="adamw", hp=_hp("adamw"),
                   steps=1, seed=61, qblock=qb)
    xts = [inputs.e4m3_integer_grid((K, T), -4, 4, inputs.layer_seed(61, 0, s, 11)) for s in range(2)]
    dyts = [inputs.e4m3_integer_grid((N, T), -4, 4, inputs.layer_seed(61, 0, s, 12)) for s in range(2)]
    sx, sdy = 2.0 ** -3, 2.0 ** -12
    g = prob.gpu_state()
    for s in range(2):
        api.forge_linear_bwd_step_fp8(xts[s].cuda(), dyts[s].cuda(), sx, sdy, g["W"], "adamw", prob.hp,
                                      s + 1, prob.seed, g["s1"], g["s2"], g["s1_scale"], g["s2_scale"])
    api.forge_get_device_status()
    st = dict(prob.state0)
    for s in range(2):
        gr = fp8.weight_gradient_fp8(xts[s].numpy().astype(np.uint8), dyts[s].numpy().astype(np.uint8),
                                     sx, sdy)
        out = ls.update_block(prob.kind, oracle_hparams(prob.hp), s + 1, prob.seed, gr, st["W"], "bf16",
                              st["s1"], st["s2"], st["s1_scale"], st["s2_scale"], "int8", 0, 0, K,
                              block=qb)
        st.update({k: out[k] for k in ("W", "s1", "s2", "s1_scale", "s2_scale")})
    _compare_exact(g, st)


@pytest.mark.parametrize("qb", BLOCKS + [64])
@pytest.mark.parametrize("signed", [True, False])
def test_quantiser_helpers_per_block_bitexact(signed, qb):
    rows, cols = 37, 1024
    x = inputs.normal((rows, cols), 1e-3, 71 + qb, torch.float32)
    if not signed:
        x = x.abs()
    x[3, :qb] = 0.0  # a zero block
    codes = torch.empty((rows, cols), dtype=torch.int8 if signed else torch.uint8, device="cuda")
    amax = torch.empty((rows, cols // qb), dtype=torch.float32, device="cuda")
    api.forge_quantize_state(x.cuda(), codes, amax, signed, block=qb)
    back = torch.empty((rows, cols), dtype=torch.float32, device="cuda")
    api.forge_dequantize_state(codes, amax, back, signed, block=qb)
    api.forge_get_device_status()
    rc, ra = quant.quantize_blocks(x.numpy(), signed=signed, block=qb)
    assert_bitexact(codes, rc, "codes")
    assert_bitexact(amax, ra, "absmax")
    assert_bitexact(back, quant.dequantize_blocks(rc, ra, signed, block=qb), "dequantised")


@pytest.mark.parametrize("qb", BLOCKS)
@pytest.mark.parametrize("T", [512, 8448], ids=["staged_w", "direct_w"])
def test_int8_blocks_realistic_interval(T, qb):
    """Realistic data (N(0,1) activations, N(0,1e-3) gradients), each step from
    the oracle's state: every output in the oracle's interval for the
    tensor-core summation error."""
    prob = Problem(T=T, N=256, K=512, w_dtype="bf16", s_dtype="int8", opt_name="adamw",
                   hp=_hp("adamw"), steps=2, seed=81 + qb, qblock=qb)
    prob.per_step_from_common_state()


@pytest.mark.parametrize("qb", BLOCKS + [64])
@pytest.mark.parametrize("signed", [True, False])
def test_quantiser_of_any_values(signed, qb):
    """Either sign in both codes (the unsigned one gives 0 to a negative value,
    whatever its neighbours are), values that are not finite, tiny blocks."""
    rows, cols = 64, 1024
    x = inputs.normal((rows, cols), 1e-3, 171 + qb, torch.float32)
    steps = torch.arange(cols, dtype=torch.float32) % 512 - 255  # x / s of -255 .. 256, halves on odd rows
    x[0], x[1], x[2] = steps / 256, (steps + 0.5) / 256, -steps.abs()
    x[3], x[4] = x[3] * 2.0 ** -130, x[4] * 2.0 ** -139  # blocks whose step is denormal, its reciprocal infinite
    x[5, ::7], x[6, ::9], x[7, ::11] = float("nan"), float("inf"), float("-inf")
    x[8] = float("nan")
    codes = torch.empty((rows, cols), dtype=torch.int8 if signed else torch.uint8, device="cuda")
    amax = torch.empty((rows, cols // qb), dtype=torch.float32, device="cuda")
    api.forge_quantize_state(x.cuda(), codes, amax, signed, block=qb)
    api.forge_get_device_status()
    rc, ra = quant.quantize_blocks(x.numpy(), signed=signed, block=qb)
    assert_bitexact(codes, rc, "codes")
    assert_bitexact(amax, ra, "absmax")
