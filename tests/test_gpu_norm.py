"""The norm and its gradient against the formulas in float64.

Bounds (u = 2^-24, half a float32 ulp): a row's sum of squares is K positive
terms added in at most D sequential steps (D below: one thread's elements, then
the warp's and the block's trees), so it is within D u of itself relatively and
rstd within D u / 2 plus three roundings.  y and dx are rounded to bf16 once
(2^-8 relative, its unit roundoff), codes to E4M3 once (2^-4 relative, 2^-10 absolute below the
smallest normal).  dw adds at most S terms in sequence.  A factor 2 on the
float32 parts covers the second-order terms."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
SHAPES = [(1, 8), (1, 4096), (2, 16), (3, 264), (17, 1000), (153, 5120), (305, 2048), (700, 128), (1300, 4104),
          (64, 8200), (33, 16384), (4099, 4096)]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def _steps(K):
    """Sequential float32 additions behind a row's sum, at most."""
    return max(32, K // 32) + 8 + 32


def _inputs(T, K, seed=1):
    x = inputs.normal((T, K), 1.0, seed, device="cuda")
    res = inputs.normal((T, K), 2.0, seed + 1, device="cuda")
    w = (1 + inputs.normal((K,), 0.3, seed + 2, torch.float32, "cuda")).to(torch.bfloat16)
    return x, res, w


def _empty(*shape, dtype=torch.bfloat16):
    # filled with NaN (0xFF in every byte), so that an element never written shows
    return torch.full(shape, 255, dtype=torch.uint8, device="cuda").view(dtype) if dtype == torch.uint8 else \
        torch.full((*shape[:-1], shape[-1] * dtype.itemsize), 255, dtype=torch.uint8, device="cuda").view(dtype)


def _formula(h, w):
    h = h.double()
    r = (h.square().mean(1) + EPS).rsqrt()
    return r, h * r[:, None] * w.double()


def _check_y(y, ref, K):
    tol = ref.abs() * (2.0 ** -8 + 2 * (_steps(K) / 2 + 6) * U) + 1e-38
    assert ((y.double() - ref).abs() <= tol).all()


def _check_codes(q, ref, K):
    ref = ref.clamp(-448, 448)
    tol = ref.abs() * (2.0 ** -4 + 2 * (_steps(K) + 12) * U) + 2.0 ** -10 * 1.001
    assert ((q.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_forward_bf16_and_token_codes(T, K, residual):
    x, res, w = _inputs(T, K)
    h, y, q = _empty(T, K), _empty(T, K), _empty(T, K, dtype=torch.float8_e4m3fn)
    rstd, scale = _empty(T, dtype=torch.float32), _empty(T, dtype=torch.float32)
    api.forge_rmsnorm_fwd(x, w, EPS, residual=res if residual else None, h=h, rstd=rstd, y=y, yq=q, yq_scale=scale)
    want = (x.float() + res.float()).to(torch.bfloat16) if residual else x
    assert torch.equal(h, want)
    r, ref = _formula(h, w)
    near = 2 * (_steps(K) / 2 + 3) * U
    assert ((rstd.double() - r).abs() <= near * r).all()
    _check_y(y, ref, K)
    s = ref.abs().amax(1) / 448
    assert ((scale.double() - s).abs() <= 2 * (_steps(K) / 2 + 8) * U * s).all()
    _check_codes(q, ref / s[:, None], K)
    alone = torch.empty_like(y)
    api.forge_rmsnorm_fwd(h, w, EPS, y=alone)  # the outputs do not depend on which are asked for
    assert torch.equal(alone, y)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,K", [(16, 8), (16, 4096), (48, 520), (160, 5120), (1296, 2048), (32, 16384), (112, 5128), (80, 8192), (48, 136)])
def test_forward_token_contiguous_codes(T, K, residual):
    x, res, w = _inputs(T, K)
    h, qt, y = _empty(T, K), _empty(K, T, dtype=torch.float8_e4m3fn), _empty(T, K)
    rstd, amax = _empty(T, dtype=torch.float32), _empty(1, dtype=torch.float32)
    out = dict(residual=res if residual else None, h=h, rstd=rstd, yt=qt, yt_scale=2.0 ** -6, amax=amax)
    api.forge_rmsnorm_fwd(x, w, EPS, **out)
    r, ref = _formula(h, w)
    assert torch.equal(h, (x.float() + res.float()).to(torch.bfloat16) if residual else x)
    assert ((rstd.double() - r).abs() <= 2 * (_steps(K) / 2 + 3) * U * r).all()
    _check_codes(qt, ref.t() * 64, K)
    top = ref.abs().max()
    assert (amax.double() - top).abs() <= 2 * (_steps(K) / 2 + 8) * U * top
    first = qt.view(torch.uint8).clone()
    api.forge_rmsnorm_fwd(x, w, EPS, **dict(out, h=h.clone(), y=y))  # with y beside them
    _check_y(y, ref, K)
    # the two ways to a row's sum may round a code apart only where it lies between two
    assert ((qt.double() - first.view(torch.float8_e4m3fn).double()).abs() <= 2.0 ** -3 * qt.double().abs() + 2.0 ** -9).all()
    # saturation: a scale so small that most values pass the largest code
    api.forge_rmsnorm_fwd(x, w, EPS, **dict(out, yt_scale=2.0 ** -12))
    _check_codes(qt, ref.t() * 4096, K)


def test_zero_rows_and_non_finite_rows_stay_to_themselves():
    T, K = 64, 512
    x, _, w = _inputs(T, K)
    x[3] = 0
    x[5, 100] = float("nan")
    x[9, 511] = float("inf")
    y, q = _empty(T, K), _empty(T, K, dtype=torch.float8_e4m3fn)
    scale, qt, amax = _empty(T, dtype=torch.float32), _empty(K, T, dtype=torch.float8_e4m3fn), _empty(1, dtype=torch.float32)
    api.forge_rmsnorm_fwd(x, w, EPS, y=y, yq=q, yq_scale=scale)
    api.forge_rmsnorm_fwd(x, w, EPS, yt=qt, yt_scale=0.125, amax=amax)
    fine = [t for t in range(T) if t not in (5, 9)]
    _, ref = _formula(x, w)
    _check_y(y[fine], ref[fine], K)
    assert not y[3].any() and scale[3] == 0 and not q.float()[3].any() and not qt.float()[:, 3].any()
    assert torch.isfinite(scale[fine]).all() and torch.isfinite(q.float()[fine]).all()
    assert torch.isfinite(qt.float()[:, fine]).all()
    for t in (5, 9):
        assert torch.isnan(scale[t]) and torch.isnan(q.float()[t]).all()
    assert torch.isnan(qt.float()[:, 5]).all() and torch.isnan(qt.float()[511, 9])
    assert torch.isnan(amax).all()


def _gradient(dy, h, w, r, dh):
    dy, h, w, r = dy.double(), h.double(), w.double(), r.double()[:, None]
    n, g = h * r, dy * w
    mean = (g * n).mean(1, keepdim=True)
    dx = r * (g - n * mean)
    size = r * (g.abs() + n.abs() * ((g * n).abs().mean(1, keepdim=True)))
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return dx, size, (dy * n).sum(0), (dy * n).abs().sum(0)


@pytest.mark.parametrize("stream_grad", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_gradient(T, K, stream_grad):
    h, dh, w = _inputs(T, K, 11)
    dy = inputs.normal((T, K), 1e-2, 21, device="cuda")
    dh = dh if stream_grad else None
    rstd = (h.float().square().mean(1) + EPS).rsqrt()
    dx, dw = _empty(T, K), _empty(K, dtype=torch.float32)
    work = _empty(api.forge_rmsnorm_bwd_workspace(T, K), dtype=torch.float32)
    api.forge_rmsnorm_bwd(dy, h, w, rstd, dx, dw, work, dh=dh)
    ref, size, wref, wsize = _gradient(dy, h, w, rstd, dh)
    assert ((dx.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 2 * (_steps(K) + 8) * U * size + 1e-38).all()
    blocks = work.numel() // K
    steps = -(-T // blocks) + blocks // 8 + 8 + 3
    assert ((dw.double() - wref).abs() <= 2 * steps * U * wsize).all()
    again, same = torch.empty_like(dw), dy.clone()
    api.forge_rmsnorm_bwd(same, h, w, rstd, same, again, work, dh=dh)  # dx over dy; the same bits again
    assert torch.equal(again, dw) and torch.equal(same, dx)


@pytest.mark.parametrize("T,K", [(5, 64), (3, 1000)])
def test_gradient_against_differences_of_the_forward_formula(T, K):
    x, dy, w = _inputs(T, K, 31)
    w64 = w.double()
    rstd = (x.float().square().mean(1) + EPS).rsqrt()
    dx, dw = _empty(T, K), _empty(K, dtype=torch.float32)
    work = torch.empty(api.forge_rmsnorm_bwd_workspace(T, K), device="cuda")
    api.forge_rmsnorm_bwd(dy, x, w, rstd, dx, dw, work)
    loss = lambda h, ww: float(((h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * ww) * dy.double()).sum())  # noqa: E731
    step = 1e-5  # central differences: error step^2 / 6 times a third derivative below 1e3, and 1e-16 / step of rounding
    for t, k in [(0, 0), (T - 1, K - 1), (1, K // 2), (2, 7)]:
        d = torch.zeros_like(x, dtype=torch.float64)
        d[t, k] = step
        slope = (loss(x.double() + d, w64) - loss(x.double() - d, w64)) / (2 * step)
        assert abs(float(dx[t, k]) - slope) <= 2.0 ** -8 * abs(slope) + 1e-5
        e = torch.zeros_like(w64)
        e[k] = step
        slope = (loss(x.double(), w64 + e) - loss(x.double(), w64 - e)) / (2 * step)
        assert abs(float(dw[k]) - slope) <= 1e-5 * (1 + abs(slope))


def test_no_tokens():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dw, amax = _empty(64, dtype=torch.float32), _empty(1, dtype=torch.float32)
    api.forge_rmsnorm_bwd(e, e, w, torch.empty(0, device="cuda"), e, dw, torch.empty(0, device="cuda"))
    assert not dw.any()
    api.forge_rmsnorm_fwd(e, w, EPS, y=e)
    api.forge_rmsnorm_fwd(e, w, EPS, yt=torch.empty((64, 0), dtype=torch.float8_e4m3fn, device="cuda"), amax=amax)
    assert amax == 0


def test_residual_stream_in_place_and_side_stream():
    T, K = 300, 1024
    x, res, w = _inputs(T, K)
    h, y = _empty(T, K), _empty(T, K)
    api.forge_rmsnorm_fwd(x, w, EPS, residual=res, h=h, y=y)
    side, over, y2 = torch.cuda.Stream(), res.clone(), _empty(T, K)
    side.wait_stream(torch.cuda.current_stream())
    api.forge_rmsnorm_fwd(x, w, EPS, residual=over, h=over, y=y2, stream=side)
    side.synchronize()
    assert torch.equal(over, h) and torch.equal(y2, y)


def test_graph_replay_of_the_gradient_and_the_codes():
    """Two launches (the second starts under the first's end) and a cleared maximum, replayed on new values."""
    T, K = 320, 2048
    x, dy, w = _inputs(T, K)
    rstd, dx, dw = torch.empty(T, device="cuda"), _empty(T, K), _empty(K, dtype=torch.float32)
    yt, amax = _empty(K, T, dtype=torch.float8_e4m3fn), _empty(1, dtype=torch.float32)
    work = torch.empty(api.forge_rmsnorm_bwd_workspace(T, K), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.forge_rmsnorm_fwd(x, w, EPS, rstd=rstd, yt=yt, yt_scale=0.125, amax=amax)
        api.forge_rmsnorm_bwd(dy, x, w, rstd, dx, dw, work)
    for scale in (1.0, 0.25):  # the second maximum is smaller: it must not keep the first
        x.copy_(inputs.normal((T, K), 1.0, 77, device="cuda"))
        w.copy_((w.float() * scale).bfloat16())
        graph.replay()
        got = [t.clone() for t in (rstd, yt.view(torch.uint8), amax, dx, dw)]
        api.forge_rmsnorm_fwd(x, w, EPS, rstd=rstd, yt=yt, yt_scale=0.125, amax=amax)
        api.forge_rmsnorm_bwd(dy, x, w, rstd, dx, dw, work)
        for a, b in zip(got, (rstd, yt.view(torch.uint8), amax, dx, dw)):
            assert torch.equal(a, b)


def test_codes_feed_the_e4m3_step():
    """yt and its scale are what forge_linear_bwd_step_fp8 takes as X: the step's gradient is that of the dequantised y."""
    T, K, N = 64, 128, 256
    x, _, w = _inputs(T, K)
    yt, scale = _empty(K, T, dtype=torch.float8_e4m3fn), 2.0 ** -5
    api.forge_rmsnorm_fwd(x, w, EPS, yt=yt, yt_scale=scale)
    dYt = inputs.e4m3_integer_grid((N, T), -4, 4, 9, "cuda")
    W = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    mom = torch.zeros((N, K), device="cuda")
    api.forge_linear_bwd_step_fp8(yt, dYt, scale, 2.0 ** -4, W, "sgd_momentum", dict(lr=0.0), 1, 0, mom)
    api.forge_get_device_status()
    ref = (dYt.view(torch.float8_e4m3fn).double() * 2.0 ** -4) @ (yt.double() * scale).t()
    size = (dYt.view(torch.float8_e4m3fn).double() * 2.0 ** -4).abs() @ (yt.double() * scale).abs().t()
    # two 32-token instructions, each at most one rounding or truncation (2 u) of a partial sum below `size`
    assert ((mom.double() - ref).abs() <= 2 * (T // 32) * 2 * U * size).all()
