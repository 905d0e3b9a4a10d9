"""Linears grouped by expert: the forward product, dX and the backward step.

Integer-grid operands make every float32 partial sum exact, so products must be
the correctly rounded bf16 of the exact sums, and the step must be the oracle's
bit for bit, whatever the groups' lengths.  On normal data a product lies within
one rounding to bf16 (2^-8) plus the float32 sum's bound of tests/_helpers: one
rounding per 16-term instruction of a partial sum at most three times its
random-walk scale."""

import math

import numpy as np
import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build
from oracle import linear_step as ls
from oracle import optimizers as opt
from oracle import quant

pytestmark = pytest.mark.gpu

GROUPS = [
    ([1], 256, 64), ([0, 1, 0, 2], 264, 200), ([5, 0, 33, 257, 300, 16], 512, 320), ([1300], 256, 256),
    ([2049, 3, 0], 128, 72), ([0, 0, 0], 64, 64), ([63, 64, 65, 31, 32, 33], 520, 136), ([17] * 70, 136, 264),
    ([1] * 300 + [0] * 700, 8, 8), ([700, 1, 900], 1024, 1096),
    # 32 rows or fewer in all take the forward product's own kernel: tiles of 8, 16 and 32 tokens, ragged K and N
    ([8], 16, 32), ([9, 0, 23], 200, 328), ([16, 16], 24, 40), ([32], 264, 1032), ([1] * 32, 8, 8), ([0, 17, 15, 0], 72, 264),
    ([33], 264, 1032),
]
IDS = [f"{len(c)}groups_T{sum(c)}_N{n}_K{k}_{max(c)}most" for c, n, k in GROUPS]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()
    api.forge_set_wait_limit_ns(200_000_000)
    api.forge_debug_skip_loads(False)
    yield
    api.forge_set_wait_limit_ns(0)


def _offsets(counts, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _slices(counts, lead=0):
    at = lead
    for e, c in enumerate(counts):
        yield e, slice(at, at + c)
        at += c


def _nan(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def _grid(shape, scale, seed):
    return inputs.integer_grid(shape, -4, 4, scale, seed, device="cuda")


def _round(exact64):
    """bf16 of exact float64 sums: they fit float32 here, so one rounding."""
    assert torch.equal(exact64.float().double(), exact64)
    return exact64.float().to(torch.bfloat16)


@pytest.mark.parametrize("counts,N,K", GROUPS, ids=IDS)
def test_products_are_exact_on_integer_grids(counts, N, K):
    E, T = len(counts), sum(counts)
    W, X, dY = _grid((E, N, K), -3, 1), _grid((T, K), 0, 2), _grid((T, N), -6, 3)
    Y, dX, off = _nan(T, N), _nan(T, K), _offsets(counts)
    api.forge_grouped_linear(X, W, off, Y)
    api.forge_grouped_dgrad(dY, W, off, dX)
    api.forge_get_device_status()
    for e, r in _slices(counts):
        assert torch.equal(Y[r], _round(X[r].double() @ W[e].double().t())), f"Y of group {e}"
        assert torch.equal(dX[r], _round(dY[r].double() @ W[e].double())), f"dX of group {e}"


@pytest.mark.parametrize("counts,N,K", [([3, 0, 900, 40], 1024, 2048), ([2000, 150], 328, 4096)])
def test_products_on_normal_data(counts, N, K):
    E, T = len(counts), sum(counts)
    W = inputs.normal((E, N, K), 0.02, 1, device="cuda")
    X, dY = inputs.normal((T, K), 1.0, 2, device="cuda"), inputs.normal((T, N), 1e-3, 3, device="cuda")
    Y, dX, off = _nan(T, N), _nan(T, K), _offsets(counts)
    api.forge_grouped_linear(X, W, off, Y)
    api.forge_grouped_dgrad(dY, W, off, dX)
    api.forge_get_device_status()

    def near(got, a, b, terms):
        ref = a.double() @ b.double()
        walk = (a.double().square() @ b.double().square()).sqrt()
        tol = ref.abs() * 2.0 ** -8 + 2.0 ** -24 * (math.ceil(terms / 16) * 3 * walk + 4 * ref.abs())
        assert ((got.double() - ref).abs() <= tol).all()

    for e, r in _slices(counts):
        near(Y[r], X[r], W[e].t(), K)
        near(dX[r], dY[r], W[e], N)


@pytest.mark.parametrize("counts,lead,tail", [([40, 0, 7], 13, 29), ([5, 0, 7], 3, 9)])
def test_rows_of_no_group_become_zero(counts, lead, tail):
    N, K = 72, 136
    T = lead + sum(counts) + tail
    W, X, dY = _grid((3, N, K), -3, 1), _grid((T, K), 0, 2), _grid((T, N), -6, 3)
    X[:lead], X[-tail:] = float("nan"), float("inf")
    Y, dX, off = _nan(T, N), _nan(T, K), _offsets(counts, lead)
    api.forge_grouped_linear(X, W, off, Y)
    api.forge_grouped_dgrad(dY, W, off, dX)
    for out in (Y, dX):
        assert not out[:lead].any() and not out[-tail:].any()
    for e, r in _slices(counts, lead):
        assert torch.equal(Y[r], _round(X[r].double() @ W[e].double().t()))
        assert torch.equal(dX[r], _round(dY[r].double() @ W[e].double()))


@pytest.mark.parametrize("counts", [[30, 45, 70, 3], [10, 5, 9, 3]], ids=["tiles", "few"])
@pytest.mark.parametrize("N,K", [(200, 328), (256, 320)])
def test_values_that_are_not_finite_stay_in_their_group(N, K, counts):
    T = sum(counts)
    W, X, dY = _grid((4, N, K), -3, 1), _grid((T, K), 0, 2), _grid((T, N), -6, 3)
    rows = dict(_slices(counts))
    bad = rows[1]
    X[bad], dY[bad] = float("nan"), float("inf")
    W[2] = float("nan")
    Y, dX, off = _nan(T, N), _nan(T, K), _offsets(counts)
    api.forge_grouped_linear(X, W, off, Y)
    api.forge_grouped_dgrad(dY, W, off, dX)
    for e in (0, 3):
        assert torch.equal(Y[rows[e]], _round(X[rows[e]].double() @ W[e].double().t()))
        assert torch.equal(dX[rows[e]], _round(dY[rows[e]].double() @ W[e].double()))
    for e in (1, 2):
        assert torch.isnan(Y[rows[e]].float()).all() and torch.isnan(dX[rows[e]].float()).all()
    # the step: the tokens after a group's last stage are another group's
    W = _grid((4, N, K), -3, 1)
    m = torch.zeros((4, N, K), device="cuda")
    api.forge_grouped_bwd_step(X, dY, W, off, "sgd_momentum", dict(lr=0.0), 1, 0, m)
    api.forge_get_device_status()
    for e in (0, 2, 3):
        assert torch.equal(m[e].double(), dY[rows[e]].double().t() @ X[rows[e]].double()), e
    assert torch.isnan(m[1]).all()


def _state(E, N, K, s_dtype, kind, block, seed):
    """Random states [E, N, K] on the CPU in the oracle's form, by name."""
    u1, u2 = opt.USES_S1[kind], opt.USES_S2[kind]
    m = inputs.normal((E * N, K), 1e-3, seed, torch.float32).numpy()
    v = inputs.abs_normal((E * N, K), 1e-6, seed + 1).numpy()
    st = dict(s1=None, s2=None, s1_scale=None, s2_scale=None)
    if s_dtype == "int8":
        st["s1"], st["s1_scale"] = quant.quantize_blocks(m, True, block) if u1 else (None, None)
        st["s2"], st["s2_scale"] = quant.quantize_blocks(v, False, block) if u2 else (None, None)
    elif s_dtype == "bf16":
        to = lambda a: inputs.bf16_to_bits(torch.from_numpy(a).to(torch.bfloat16))  # noqa: E731
        st["s1"], st["s2"] = to(m) if u1 else None, to(v) if u2 else None
    else:
        st["s1"], st["s2"] = m if u1 else None, v if u2 else None
    return st


def _step_case(counts, N, K, s_dtype, rule, block=64, with_dx=True, seed=91):
    E, T, kind = len(counts), sum(counts), opt.NAMES.index(rule)
    hp = dict(inputs.SWEEP_HPARAMS[rule], weight_decay=0.1)
    X, dY = _grid((T, K), 0, 2), _grid((T, N), -12, 3)
    W0 = _grid((E, N, K), -6, 1)
    st = _state(E, N, K, s_dtype, kind, block, 7)
    up = {}
    for name, a in st.items():
        if a is None:
            up[name] = None
            continue
        t = inputs.bits_to_bf16(a) if a.dtype == np.uint16 else torch.from_numpy(a.copy())
        up[name] = t.cuda().view(E, N, -1)
    W, dX, off = W0.clone(), _nan(T, K), _offsets(counts)
    api.forge_grouped_bwd_step(X, dY, W, off, rule, hp, 3, seed, up["s1"], up["s2"], up["s1_scale"], up["s2_scale"],
                               dX=dX if with_dx else None)
    api.forge_get_device_status()
    xb, yb, wb = inputs.bf16_to_bits(X), inputs.bf16_to_bits(dY), inputs.bf16_to_bits(W0)
    for e, r in _slices(counts):
        g = ls.weight_gradient(xb[r], yb[r]) if counts[e] else np.zeros((N, K), np.float32)
        rows = slice(e * N, (e + 1) * N)
        part = {k: None if a is None else a[rows] for k, a in st.items()}
        ref = ls.update_block(kind, opt.Hparams(**hp), 3, seed, g, wb[e], "bf16", part["s1"], part["s2"],
                              part["s1_scale"], part["s2_scale"], s_dtype, e * N, 0, K, block)
        np.testing.assert_array_equal(inputs.bf16_to_bits(W[e]), ref["W"], err_msg=f"W of expert {e}")
        for name in ("s1", "s2", "s1_scale", "s2_scale"):
            if up[name] is not None:
                got = up[name][e]
                got = inputs.bf16_to_bits(got) if got.dtype == torch.bfloat16 else got.cpu().numpy()
                np.testing.assert_array_equal(got, ref[name], err_msg=f"{name} of expert {e}")
        if with_dx:
            assert torch.equal(dX[r], _round(dY[r].double() @ W0[e].double())), f"dX of expert {e}"


@pytest.mark.parametrize("s_dtype", ["fp32", "bf16", "int8"])
@pytest.mark.parametrize("counts,N,K", [([1], 128, 64), ([0, 64, 1, 65, 0], 320, 384), ([200, 3, 130, 63], 72, 192),
                                        ([0, 0], 136, 320), ([5] * 20, 264, 128)],
                         ids=["one_row", "stage_edges", "narrow", "no_tokens_but_rows", "many"])
def test_step_equals_the_oracle(counts, N, K, s_dtype):
    _step_case(counts, N, K, s_dtype, "adamw")


@pytest.mark.parametrize("s_dtype", ["fp32", "int8"])
@pytest.mark.parametrize("rule", opt.NAMES)
def test_step_every_rule(rule, s_dtype):
    _step_case([70, 0, 9], 200, 256, s_dtype, rule)


@pytest.mark.parametrize("block", [32, 128, 256])
def test_step_int8_block_widths(block):
    _step_case([70, 0, 9], 320, 512, "int8", "adamw", block)


def test_step_with_ragged_widths_and_no_dx():
    _step_case([33, 90, 0, 128], 200, 136, "fp32", "adamw", with_dx=False)
    _step_case([33, 90, 0, 128], 8, 72, "bf16", "adamw")


def test_more_tiles_than_pairs():
    _step_case([40, 90, 0, 128], 1040, 1280, "fp32", "adamw")


@pytest.mark.parametrize("s_dtype", ["fp32", "bf16", "int8"])
@pytest.mark.parametrize("counts", [[1535], [1536], [3583], [3584], [5000, 900], [9001, 0, 1800]],
                         ids=lambda c: "_".join(map(str, c)))
def test_step_of_longer_groups(counts, s_dtype):
    """Means on either side of each change of the kernel's layout (1536 and 3584 tokens), ragged ends."""
    _step_case(counts, 136, 192, s_dtype, "adamw")


@pytest.mark.parametrize("rule", ["lion", "rmsprop", "sgd", "sgd_momentum"])
@pytest.mark.parametrize("tokens", [1700, 4000])
def test_step_of_longer_groups_other_rules(rule, tokens):
    _step_case([tokens], 264, 320, "fp32", rule)


@pytest.mark.parametrize("s_dtype", ["fp32", "int8"])
def test_one_group_steps_as_the_linear_step(s_dtype):
    # whole 64-token stages: a ragged last stage holds its rows after the zeros here, before them there, which
    # gives the instructions' 16-row sums other members
    T, N, K = 320, 384, 512
    X, dY = inputs.normal((T, K), 1.0, 2, device="cuda"), inputs.normal((T, N), 1e-3, 3, device="cuda")
    W0 = inputs.normal((N, K), 0.02, 1, device="cuda")

    def states():
        if s_dtype == "int8":
            return [torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros((N, K), dtype=torch.uint8, device="cuda"),
                    torch.zeros((N, K // 64), device="cuda"), torch.zeros((N, K // 64), device="cuda")]
        return [torch.zeros((N, K), device="cuda"), torch.zeros((N, K), device="cuda")]

    a, b, Wa, Wb = states(), states(), W0.clone(), W0.clone().view(1, N, K)
    dxa, dxb = _nan(T, K), _nan(T, K)
    hp = dict(lr=1e-3, weight_decay=0.1)
    api.forge_linear_bwd_step(X, dY, Wa, "adamw", hp, 1, 5, *a, dX=dxa)
    api.forge_grouped_bwd_step(X, dY, Wb, _offsets([T]), "adamw", hp, 1, 5, *[t.view(1, N, -1) for t in b], dX=dxb)
    api.forge_get_device_status()
    assert torch.equal(Wa, Wb[0])
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    near = (dxa.double() - dxb.double()).abs()  # the sums run in another order
    assert (near <= 2.0 ** -7 * dxa.double().abs() + 1e-9).all()


def test_gradient_of_the_products_against_differences():
    """With y = W x: dX and the step's dW against central differences of the loss sum(y dy) in float64."""
    counts, N, K = [3, 4], 16, 24
    T = sum(counts)
    W, X, dY = _grid((2, N, K), -3, 1), _grid((T, K), 0, 2), _grid((T, N), -6, 3)
    off, dX = _offsets(counts), _nan(T, K)
    g, W2 = torch.zeros((2, N, K), device="cuda"), W.clone()
    api.forge_grouped_bwd_step(X, dY, W2, off, "sgd_momentum", dict(lr=0.0), 1, 0, g, dX=dX)
    api.forge_get_device_status()

    def loss(w, x):
        return sum(float(((x[r] @ w[e].t()) * dY[r].double()).sum()) for e, r in _slices(counts))

    w, x, step = W.double(), X.double(), 2.0 ** -10  # the loss is bilinear: differences are exact
    for e, n, k in [(0, 0, 0), (1, 15, 23), (1, 7, 11)]:
        d = torch.zeros_like(w)
        d[e, n, k] = step
        assert abs((loss(w + d, x) - loss(w - d, x)) / (2 * step) - float(g[e, n, k])) <= 1e-9
    for t, k in [(0, 0), (2, 5), (3, 5), (6, 23)]:
        d = torch.zeros_like(x)
        d[t, k] = step
        slope = (loss(w, x + d) - loss(w, x - d)) / (2 * step)
        assert abs(slope - float(dX[t, k])) <= 2.0 ** -8 * abs(slope) + 1e-9


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 10, 20, 90], [0, 10, 200, 300], [2 ** 31 - 1, 0, -2 ** 31, 7], [0, 5, 5, 91]])
@pytest.mark.parametrize("T", [90, 20])
def test_offsets_out_of_order_or_range_are_clamped_and_reported(offsets, T):
    N, K = 64, 64
    W, X, dY = _grid((3, N, K), -3, 1), _grid((T, K), 0, 2), _grid((T, N), -6, 3)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    guard = torch.zeros((3 * T, N), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: api.forge_grouped_linear(X, W, off, guard[T:2 * T]),
                 lambda: api.forge_grouped_dgrad(dY, W, off, guard[T:2 * T]),
                 lambda: api.forge_grouped_bwd_step(X, dY, W, off, "sgd", dict(lr=0.0), 1, 0)):
        call()
        with pytest.raises(api.ForgeError, match="offsets"):
            api.forge_get_device_status()
        api.forge_get_device_status()  # reported once
    assert not guard[:T].any() and not guard[2 * T:].any()


def test_side_stream_and_graph_replay_read_the_offsets_when_they_run():
    counts, N, K = [20, 50], 128, 192
    T = 70
    W, X = _grid((2, N, K), -3, 1), _grid((T, K), 0, 2)
    Y, off = _nan(T, N), _offsets(counts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.forge_grouped_linear(X, W, off, Y, stream=side)
    side.synchronize()
    ref = torch.cat([_round(X[r].double() @ W[e].double().t()) for e, r in _slices(counts)])
    assert torch.equal(Y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.forge_grouped_linear(X, W, off, Y)
    off.copy_(_offsets([65, 5]))
    graph.replay()
    torch.cuda.synchronize()
    ref = torch.cat([_round(X[r].double() @ W[e].double().t()) for e, r in _slices([65, 5])])
    assert torch.equal(Y, ref)


@pytest.mark.parametrize("s_dtype", ["fp32", "int8"])
def test_the_captured_step_replays_with_its_dx(s_dtype):
    """dX and the step that starts under its tail, replayed: the same bits as the direct calls, step after step."""
    counts, N, K, hp = [300, 0, 70], 328 if s_dtype == "fp32" else 320, 384, dict(lr=1e-2, weight_decay=0.1)
    T, off = sum(counts), _offsets(counts)
    X, dY = inputs.normal((T, K), 1.0, 2, device="cuda"), inputs.normal((T, N), 1e-2, 3, device="cuda")

    def fresh():
        W = inputs.normal((3, N, K), 0.02, 1, device="cuda")
        if s_dtype == "fp32":
            return W, [torch.zeros((3, N, K), device="cuda") for _ in range(2)], _nan(T, K)
        return W, [torch.zeros((3, N, K), dtype=torch.int8, device="cuda"), torch.zeros((3, N, K), dtype=torch.uint8, device="cuda"),
                   torch.zeros((3, N, K // 64), device="cuda"), torch.zeros((3, N, K // 64), device="cuda")], _nan(T, K)

    (Wa, sa, da), (Wb, sb, db) = fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.forge_grouped_bwd_step(X, dY, Wb, off, "adamw", hp, 1, 5, *sb, dX=db)
    for _ in range(3):
        api.forge_grouped_bwd_step(X, dY, Wa, off, "adamw", hp, 1, 5, *sa, dX=da)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([Wa, da, *sa], [Wb, db, *sb]):
            assert torch.equal(a, b)
    api.forge_get_device_status()


def test_a_wait_that_runs_out_is_reported():
    W, X = _grid((2, 64, 64), -3, 1), _grid((20, 64), 0, 2)
    Y, off = _nan(20, 64), _offsets([10, 10])
    m = torch.zeros((2, 64, 64), device="cuda")
    api.forge_set_wait_limit_ns(20_000_000)
    api.forge_debug_skip_loads(True)
    try:
        for call in (lambda: api.forge_grouped_linear(X, W, off, Y),
                     lambda: api.forge_grouped_bwd_step(X, Y, W, off, "sgd_momentum", dict(lr=0.0), 1, 0, m)):
            call()
            with pytest.raises(api.ForgeError, match="TIMEOUT"):
                api.forge_get_device_status()
    finally:
        api.forge_debug_skip_loads(False)
        api.forge_set_wait_limit_ns(200_000_000)
    api.forge_grouped_linear(X, W, off, Y)
    api.forge_get_device_status()
    assert torch.equal(Y[:10], _round(X[:10].double() @ W[0].double().t()))


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 10, 20, 90], [0, 10, 200, 300], [2 ** 31 - 1, 0, -2 ** 31, 7],
                                     [30, 5, 60, 40], [0, 5, 5, 91]])
@pytest.mark.parametrize("T", [90, 20, 5000, 11000])
def test_clamped_offsets_give_every_kernel_the_same_rows(offsets, T):
    """Expert e's rows run from the largest offset up to e to the largest up to e + 1, all clamped to [0, T]:
    in Y (both forward kernels), dX and dW, in each layout of the step."""
    if T > 90:  # the same order over longer groups
        offsets = [min(o * (T // 90), 2 ** 31 - 1) if o > 0 else o for o in offsets]
    N, K = 72, 64
    W, X, dY = _grid((3, N, K), -3, 1), _grid((T, K), 0, 2), _grid((T, N), -6, 3)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    Y, dX, dX2, m = _nan(T, N), _nan(T, K), _nan(T, K), torch.zeros((3, N, K), device="cuda")
    W0 = W.clone()
    for call in (lambda: api.forge_grouped_linear(X, W, off, Y), lambda: api.forge_grouped_dgrad(dY, W, off, dX),
                 lambda: api.forge_grouped_bwd_step(X, dY, W, off, "sgd_momentum", dict(lr=0.0), 1, 0, m, dX=dX2)):
        call()
        with pytest.raises(api.ForgeError, match="offsets"):
            api.forge_get_device_status()
    edges = np.maximum.accumulate(np.clip(offsets, 0, T))
    own = torch.zeros(T, dtype=torch.bool, device="cuda")
    for e in range(3):
        r = slice(int(edges[e]), int(edges[e + 1]))
        own[r] = True
        assert torch.equal(Y[r], _round(X[r].double() @ W0[e].double().t())), f"Y of group {e}"
        assert torch.equal(dX[r], _round(dY[r].double() @ W0[e].double())), f"dX of group {e}"
        assert torch.equal(m[e].double(), dY[r].double().t() @ X[r].double()), f"dW of group {e}"
    assert torch.equal(dX2, dX)
    for out in (Y, dX):
        assert not out[~own].any()
