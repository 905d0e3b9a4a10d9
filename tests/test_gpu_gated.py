"""The gated feed-forward products: forward, what they keep, and the gradient.

Bounds (u = 2^-23): a float32 sum of K products is off by (K / 16 + 8) u of the
sum of magnitudes (one rounding for each instruction of 16 terms, were it a
truncation); the gate's slope is at most 1.2, its float32 evaluation off by
2^-17 at |g| < 8 (1 - sigma is off by 2^-24 and meets g d, at most 2^7 there);
then bf16's 2^-8 or the codes' 2^-4 (2^-10 of the scale below their smallest
normal).  Integer-grid operands make the sums exact, and what is kept of them is
then exact too."""

import math

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_codes import B16, E4M3, F32, blocks, scales, spread

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh"]
KEEPS = ["none", "bf16", "e4m3"]
U = 2.0 ** -23
# tokens, gated features, reduction
SHAPES = [(1, 8, 8), (1, 4096, 256), (2, 128, 64), (7, 136, 200), (32, 264, 520), (33, 264, 520), (24, 2056, 1032),
          (128, 384, 128), (129, 1000, 72), (256, 128, 64), (257, 2056, 136), (300, 640, 1024), (2049, 520, 264),
          (1000, 9216, 64)]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()
    api.forge_set_wait_limit_ns(200_000_000)
    api.forge_debug_skip_loads(False)
    yield
    api.forge_set_wait_limit_ns(0)


def act(kind, g):
    """The gate and its slope, in g's type: g s, s + g s (1 - s) d."""
    if kind == "silu":
        s, d = torch.sigmoid(g), 1.0
    else:
        c = 2 * math.sqrt(2 / math.pi)
        s, d = torch.sigmoid(c * (g + 0.044715 * g ** 3)), c * (1 + 3 * 0.044715 * g ** 2)
    return g * s, s + g * s * (1 - s) * d


def guarded(T, width, dtype=B16):
    """[T, width] of NaN with a row of sevens behind."""
    t = torch.full((T + 1, width), float("nan"), dtype=F32, device="cuda")
    t[T] = 7
    return t.to(dtype)


def forward(X, W, kind, keep):
    T, F = X.shape[0], W.shape[0] // 2
    Y = guarded(T, F)
    gu = guarded(T, 2 * F) if keep == "bf16" else None
    codes = guarded(T, 2 * F, E4M3) if keep == "e4m3" else None
    scale = guarded(T, 2 * blocks(F), F32).view(T + 1, 2, blocks(F)) if keep == "e4m3" else None
    cut = lambda t: None if t is None else t[:T]  # noqa: E731
    api.forge_gated_linear(X, W, Y[:T], act=kind, gu=cut(gu), gu_codes=cut(codes), gu_scale=cut(scale))
    api.forge_get_device_status()
    for t in (Y, gu, codes, scale):
        assert t is None or (t[T].float() == 7).all()
    return Y[:T], cut(gu), cut(codes), cut(scale)


def decoded(codes, scale):
    T, F = codes.shape[0], codes.shape[1] // 2
    return (codes.double().view(2 * T, F) * spread(scale.double().reshape(2 * T, -1), (2 * T, F), 1)).view(T, 2 * F)


def exact(X, W, kind):
    """G and U side by side, Y, and their bounds before the last rounding."""
    F, K = W.shape[0] // 2, X.shape[1]
    gu = X.double() @ W.double().t()
    off = (X.double().abs() @ W.double().abs().t()) * ((K / 16 + 8) * U)
    a, _ = act(kind, gu[:, :F])
    og, ou = off[:, :F], off[:, F:]
    y = a * gu[:, F:]
    return gu, off, y, 1.2 * og * (gu[:, F:].abs() + ou) + a.abs() * ou + y.abs() * 2.0 ** -18


@pytest.mark.parametrize("keep", KEEPS)
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("T,F,K", SHAPES)
def test_forward(T, F, K, kind, keep):
    X, W = inputs.normal((T, K), 1.0, 1, device="cuda"), inputs.normal((2 * F, K), 1.3 * K ** -0.5, 2, device="cuda")
    Y, gu, codes, scale = forward(X, W, kind, keep)
    want, off, y, oy = exact(X, W, kind)
    assert ((Y.double() - y).abs() <= oy + y.abs() * 2.0 ** -8 + 1e-38).all()
    if keep == "bf16":
        assert ((gu.double() - want).abs() <= off + want.abs() * 2.0 ** -8).all()
    if keep == "e4m3":
        s = scale.double().view(2 * T, -1)
        most = scales(want.float().view(2 * T, F), 1).double()
        room = scales(off.float().view(2 * T, F), 1).double()  # (the largest bound over 448)
        assert ((s - most).abs() <= room + most * 2.0 ** -22).all()
        wide = spread(s, (2 * T, F), 1).reshape(T, 2 * F)
        assert ((decoded(codes, scale) - want).abs() <= off + want.abs() * (2.0 ** -4 + 2.0 ** -20) + wide * 2.0 ** -10).all()


@pytest.mark.parametrize("T,F,K", [(5, 136, 64), (33, 264, 520), (300, 640, 1024), (600, 4096, 72)])
def test_kept_projections_of_exact_sums(T, F, K):
    """Whole numbers: G and U are exact, so is their bf16, and the codes are the quantiser's."""
    X, W = inputs.integer_grid((T, K), -4, 4, 0, 3, device="cuda"), inputs.integer_grid((2 * F, K), -4, 4, -6, 4, device="cuda")
    want = (X.double() @ W.double().t()).float()
    outs = [forward(X, W, "silu", keep) for keep in KEEPS]
    assert torch.equal(outs[1][1], want.to(B16))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][0], outs[2][0])  # Y whatever is kept
    codes, scale = torch.empty((2 * T, F), dtype=E4M3, device="cuda"), torch.empty((2 * T, blocks(F)), device="cuda")
    api.forge_quantize_e4m3(want.view(2 * T, F), codes, scale)
    assert torch.equal(outs[2][3].reshape(-1), scale.view(-1))
    assert torch.equal(outs[2][2].view(torch.uint8).reshape(-1), codes.view(torch.uint8).view(-1))


def test_scales_of_long_sums():
    """Scales are float32, so their sums are cut: 768 terms an instruction of 16 at a time (48 u, were each a
    truncation), the cuts added with half a u each and the division half of one.  Terms of one sign lose most."""
    T, F, K = 33, 264, 8200
    X, W = inputs.normal((T, K), 1.0, 1, device="cuda").abs(), inputs.normal((2 * F, K), 0.02, 2, device="cuda").abs()
    scale = forward(X, W, "silu", "e4m3")[3].double().view(2 * T, -1)
    sums = (X.double() @ W.double().t()).view(2 * T, F)
    most = torch.stack([c.amax(1) for c in sums.split(128, 1)], 1) / 448
    assert ((scale - most).abs() <= most * ((48 + K / 768 + 2) * U)).all()


def gradient(dY, Wd, kind, gu=None, codes=None, scale=None, want_y=True, inplace=False):
    T, F = dY.shape[0], Wd.shape[1]
    dGU = gu if inplace else guarded(T, 2 * F)
    Y = guarded(T, F) if want_y else None
    api.forge_gated_dgrad(dY, Wd, dGU[:T], act=kind, gu=gu, gu_codes=codes, gu_scale=scale, Y=Y[:T] if want_y else None)
    api.forge_get_device_status()
    assert inplace or (dGU[T] == 7).all()
    assert not want_y or (Y[T] == 7).all()
    return dGU[:T], Y[:T] if want_y else None


def check_gradient(dY, Wd, kind, gu, got, y):
    """gu: the kept values in 64 bits."""
    N, F = Wd.shape
    da = dY.double() @ Wd.double()
    off = (dY.double().abs() @ Wd.double().abs()) * ((N / 16 + 8) * U)
    g, u = gu[:, :F], gu[:, F:]
    a, slope = act(kind, g)
    dg, du = da * u * slope, da * a
    room = off * u.abs() * 1.2 + da.abs() * u.abs() * 2.0 ** -17
    assert ((got[:, :F].double() - dg).abs() <= room + dg.abs() * 2.0 ** -8 + 1e-38).all()
    assert ((got[:, F:].double() - du).abs() <= off * a.abs() + du.abs() * (2.0 ** -8 + 2.0 ** -18) + 1e-38).all()
    if y is not None:
        assert ((y.double() - a * u).abs() <= (a * u).abs() * (2.0 ** -8 + 2.0 ** -18) + 1e-38).all()


def kept(T, F, keep, seed=5):
    gu = inputs.normal((T, 2 * F), 1.3, seed, device="cuda")
    if keep == "bf16":
        return dict(gu=gu), gu.double()
    codes, scale = torch.empty((2 * T, F), dtype=E4M3, device="cuda"), torch.empty((2 * T, blocks(F)), device="cuda")
    api.forge_quantize_e4m3(gu.view(2 * T, F), codes, scale)
    codes, scale = codes.view(T, 2 * F), scale.view(T, 2, -1)
    return dict(codes=codes, scale=scale), decoded(codes, scale)


@pytest.mark.parametrize("keep", KEEPS[1:])
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("T,F,N", SHAPES)
def test_gradient(T, F, N, kind, keep):
    dY, Wd = inputs.normal((T, N), 1e-2, 6, device="cuda"), inputs.normal((N, F), 0.05, 7, device="cuda")
    args, gu = kept(T, F, keep)
    check_gradient(dY, Wd, kind, gu, *gradient(dY, Wd, kind, **args))
    alone, _ = gradient(dY, Wd, kind, want_y=False, **args)
    again, _ = gradient(dY, Wd, kind, **args)
    assert torch.equal(alone, again)


@pytest.mark.parametrize("T,F,N", [(7, 136, 200), (300, 640, 64), (600, 2056, 264)])
def test_gradient_over_what_was_kept(T, F, N):
    dY, Wd = inputs.normal((T, N), 1e-2, 6, device="cuda"), inputs.normal((N, F), 0.05, 7, device="cuda")
    gu = kept(T, F, "bf16")[0]["gu"]
    want, y = gradient(dY, Wd, "silu", gu=gu)
    got, y2 = gradient(dY, Wd, "silu", gu=gu, inplace=True)
    assert got.data_ptr() == gu.data_ptr() and torch.equal(got, want) and torch.equal(y, y2)


@pytest.mark.parametrize("kind", ACTS)
def test_gradient_against_differences(kind):
    """dGU is the slope of sum(dY * (Y Wd^T)) in G and U: central differences in 64 bits."""
    T, F, N = 5, 24, 40
    dY, Wd = inputs.normal((T, N), 1.0, 6, device="cuda"), inputs.normal((N, F), 0.2, 7, device="cuda")
    args, gu = kept(T, F, "bf16")
    got, _ = gradient(dY, Wd, kind, **args)

    def loss(v):
        return ((act(kind, v[:, :F])[0] * v[:, F:]) @ Wd.double().t() * dY.double()).sum()

    h, want = 2.0 ** -13, torch.empty_like(gu)
    for t in range(T):
        for j in range(2 * F):
            e = torch.zeros_like(gu)
            e[t, j] = h
            want[t, j] = (loss(gu + e) - loss(gu - e)) / (2 * h)
    # differences: h^2 / 6 of the third derivative (below 20 here), bf16, and the sum's bound
    assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + 20 * h * h / 6 + 2.0 ** -16).all()


@pytest.mark.parametrize("kind", ACTS)
def test_gates_far_from_zero(kind):
    """Saturated gates give g or 0, slopes 1 or 0; what is not finite gives what the formula does."""
    big = torch.tensor([0.0, -0.0, 20, -20, 60, -60, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38, -90, -100, 8, -8], device="cuda")
    T, F = 16, 16
    gu = torch.ones((T, 2 * F), dtype=B16, device="cuda")
    gu[:, :F] = big.to(B16)
    dY = torch.ones((T, 8), dtype=B16, device="cuda")
    Wd = torch.full((8, F), 0.125, dtype=B16, device="cuda")
    dGU, Y = gradient(dY, Wd, kind, gu=gu)  # dA = 1
    g = gu[:, :F].double()
    s = torch.sigmoid(g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    d = 1.0 if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    slope = s + g * s * (1 - s) * d
    assert torch.isfinite(dGU.float()).all() and torch.isfinite(Y.float()).all()
    for got, want in ((dGU[:, F:], g * s), (Y, g * s), (dGU[:, :F], slope)):
        assert ((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -15) + 1e-37).all()
    gu[3, 2], gu[5, F + 4], gu[6, 1] = float("nan"), float("nan"), float("inf")
    dGU, Y = gradient(dY, Wd, kind, gu=gu)
    bad = torch.zeros((T, F), dtype=torch.bool, device="cuda")
    bad[3, 2] = bad[5, 4] = True
    assert torch.equal(torch.isnan(Y), bad) and torch.isinf(Y[6, 1])
    assert torch.isnan(dGU[3, 2]) and torch.isnan(dGU[3, F + 2]) and torch.isnan(dGU[5, 4]) and not torch.isnan(dGU[5, F + 4])


def test_values_that_are_not_finite_stay_in_their_row():
    X, W = inputs.normal((40, 136), 1.0, 1, device="cuda"), inputs.normal((2 * 264, 136), 0.1, 2, device="cuda")
    X[3, 7] = float("nan")
    Y, _, codes, scale = forward(X, W, "silu", "e4m3")
    rows = torch.isnan(Y).any(1)
    assert rows[3] and rows.sum() == 1 and torch.isnan(Y[3]).all()
    assert torch.isnan(scale[3]).all() and torch.isnan(codes[3].float()).all() and not torch.isnan(scale[:3]).any()


def test_nothing_to_sum_and_nothing_to_do():
    e = lambda *s, d=B16: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    Y, gu = torch.full((3, 16), 5.0, dtype=B16, device="cuda"), torch.full((3, 32), 5.0, dtype=B16, device="cuda")
    codes, scale = torch.full((3, 32), 5.0, device="cuda").to(E4M3), torch.full((3, 2, 1), 5.0, device="cuda")
    api.forge_gated_linear(e(3, 0), e(32, 0), Y, gu=gu)
    assert (Y == 0).all() and (gu == 0).all()
    api.forge_gated_linear(e(3, 0), e(32, 0), Y, gu_codes=codes, gu_scale=scale)
    assert (codes.float() == 0).all() and (scale == 0).all()
    api.forge_gated_linear(e(0, 16), e(32, 16), e(0, 16), gu=e(0, 32))
    api.forge_gated_linear(e(3, 16), e(0, 16), e(3, 0))
    api.forge_gated_dgrad(e(0, 16), e(16, 8), e(0, 16), gu=e(0, 16))
    api.forge_gated_dgrad(e(3, 16), e(16, 0), e(3, 0), gu=e(3, 0))
    api.forge_get_device_status()


@pytest.mark.parametrize("keep", KEEPS)
def test_a_wait_that_runs_out_is_reported(keep):
    X, W = inputs.normal((300, 136), 1.0, 1, device="cuda"), inputs.normal((2 * 264, 136), 0.1, 2, device="cuda")
    args, gu = kept(300, 264, "bf16" if keep == "none" else keep)
    dY, Wd = inputs.normal((300, 64), 1e-2, 6, device="cuda"), inputs.normal((64, 264), 0.05, 7, device="cuda")
    api.forge_set_wait_limit_ns(20_000_000)
    api.forge_debug_skip_loads(True)
    try:
        with pytest.raises(api.ForgeError, match="TIMEOUT"):
            forward(X, W, "silu", keep)
        with pytest.raises(api.ForgeError, match="TIMEOUT"):
            gradient(dY, Wd, "silu", **args)
    finally:
        api.forge_debug_skip_loads(False)
        api.forge_set_wait_limit_ns(200_000_000)
    check_gradient(dY, Wd, "silu", gu, *gradient(dY, Wd, "silu", **args))
    _, _, y, oy = exact(X, W, "silu")
    assert ((forward(X, W, "silu", keep)[0].double() - y).abs() <= oy + y.abs() * 2.0 ** -8).all()


@pytest.mark.parametrize("T", [9, 200])
def test_captured_two_streams(T):
    """Forward and gradient captured twice, in flight together, replayed on new values."""
    F, K = 264, 136
    made = []
    for i in range(2):
        t = dict(X=inputs.normal((T, K), 1.0, i, device="cuda"), W=inputs.normal((2 * F, K), 0.1, 2 + i, device="cuda"),
                 dY=inputs.normal((T, K), 0.1, 4 + i, device="cuda"), Wd=inputs.normal((K, F), 0.1, 6 + i, device="cuda"))
        out = [torch.empty((T, n), dtype=B16, device="cuda") for n in (F, 2 * F, 2 * F, F)]
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            api.forge_gated_linear(t["X"], t["W"], out[0], gu=out[1])
            api.forge_gated_dgrad(t["dY"], t["Wd"], out[2], gu=out[1], Y=out[3])
        made.append((t, out, stream, graph))
    for seed in (20, 30):
        for i, (t, out, stream, graph) in enumerate(made):
            t["X"].copy_(inputs.normal((T, K), 1.0, seed + i, device="cuda"))
            t["dY"].copy_(inputs.normal((T, K), 0.1, seed + 5 + i, device="cuda"))
        torch.cuda.synchronize()
        for t, out, stream, graph in made:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for t, out, stream, graph in made:
            Y, gu, _, _ = forward(t["X"], t["W"], "silu", "bf16")
            dGU, Y2 = gradient(t["dY"], t["Wd"], "silu", gu=gu)
            for a, b in zip(out, (Y, gu, dGU, Y2)):
                assert torch.equal(a, b)
