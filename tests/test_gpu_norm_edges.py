"""The norm where its arithmetic or its buffers meet an edge: eps = 0, rows and
weights far from one, values that are not finite, outputs over inputs.

Bounds as in test_gpu_norm.py (u = 2^-24): a row's sum carries D u of itself,
rstd half of that and three roundings, y and dx one rounding to bf16 (2^-8),
codes one to E4M3 (2^-4, 2^-10 below the smallest normal)."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def _steps(K):
    """Sequential float32 additions behind a row's sum, at most."""
    return max(32, K // 32) + 8 + 32


def _inputs(T, K, seed=1):
    x, res = inputs.normal((T, K), 1.0, seed, device="cuda"), inputs.normal((T, K), 2.0, seed + 1, device="cuda")
    return x, res, (1 + inputs.normal((K,), 0.3, seed + 2, torch.float32, "cuda")).to(B16)


def _nan(*shape, dtype=B16):
    """Filled with 0xFF, a NaN of every type, so that an element never written shows."""
    return torch.full((*shape[:-1], shape[-1] * dtype.itemsize), 255, dtype=torch.uint8, device="cuda").view(dtype)


def test_a_wait_for_the_cluster_that_runs_out_is_reported():
    """No block sends its rows' shares: each gives up, writes no codes, rstd or maximum, and the next call works."""
    T, K = 80, 4096  # three tiles of eight blocks
    x, res, w = _inputs(T, K)
    args = lambda: dict(residual=res, h=_nan(T, K), rstd=_nan(T, dtype=torch.float32), yt=_nan(K, T, dtype=E4M3),  # noqa: E731
                        yt_scale=2.0 ** -5, amax=_nan(1, dtype=torch.float32))
    a = args()
    api.forge_set_wait_limit_ns(20_000_000)
    api.forge_debug_skip_loads(True)
    try:
        api.forge_rmsnorm_fwd(x, w, 1e-6, **a)
        with pytest.raises(api.ForgeError, match="TIMEOUT"):
            api.forge_get_device_status()
    finally:
        api.forge_debug_skip_loads(False)
        api.forge_set_wait_limit_ns(0)
    assert torch.isnan(a["rstd"]).all() and (a["yt"].view(torch.uint8) == 255).all() and a["amax"] == 0
    a, b = args(), args()
    api.forge_rmsnorm_fwd(x, w, 1e-6, **a)
    api.forge_rmsnorm_fwd(x, w, 1e-6, **dict(b, yt=None, amax=None))
    api.forge_get_device_status()
    assert torch.equal(a["h"], b["h"]) and torch.isfinite(a["yt"].float()).all() and a["amax"] > 1
    assert torch.allclose(a["rstd"], b["rstd"], rtol=1e-5)


def _gradient(dy, h, w, rstd, dh=None):
    T, K = h.shape
    dx, dw = _nan(T, K), _nan(K, dtype=torch.float32)
    api.forge_rmsnorm_bwd(dy, h, w, rstd, dx, dw, _nan(api.forge_rmsnorm_bwd_workspace(T, K), dtype=torch.float32), dh=dh)
    return dx, dw


@pytest.mark.parametrize("stream_grad", [False, True])
@pytest.mark.parametrize("T,K", [(9, 512), (9, 4104), (9, 9000)])
def test_gradient_of_rows_far_from_one(T, K, stream_grad):
    """rstd of 2^66 has no square in float32, dx is 2^66 times an ordinary number and has its value."""
    h, dh, w = _inputs(T, K)
    dy = inputs.normal((T, K), 1e-2, 21, device="cuda")
    for t, e in enumerate((-66, -60, -40, 0, 40, 60)):
        h[t] *= 2.0 ** e
    dh = dh if stream_grad else None
    rstd = h.double().square().mean(1).rsqrt().float()
    dx, _ = _gradient(dy, h, w, rstd, dh)
    r = rstd.double()[:, None]
    n, g = h.double() * r, dy.double() * w.double()
    ref = r * (g - n * (g * n).mean(1, keepdim=True))
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if stream_grad:
        ref, size = ref + dh.double(), size + dh.double().abs()
    assert torch.isfinite(dx).all()
    assert ((dx.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 2 * (_steps(K) + 8) * U * size + 1e-38).all()


@pytest.mark.parametrize("T,K", [(3, 264), (700, 128), (64, 8200)])
def test_codes_of_tiny_rows_are_those_of_the_stored_scale(T, K):
    """y near 2^-126: 448 / max|y| is past the largest float, max|y| / 448 a denormal; code * scale is y all the same.
    A product's denormal rounding is 2^-150, far below a code's 2^-10 of the scale (2^-134 and more)."""
    x, _, w = _inputs(T, K)
    w = (w.float() * 2.0 ** -126).to(B16)
    y, q, scale = _nan(T, K), _nan(T, K, dtype=E4M3), _nan(T, dtype=torch.float32)
    api.forge_rmsnorm_fwd(x, w, 1e-6, y=y, yq=q, yq_scale=scale)
    h = x.double()
    ref = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    s = ref.abs().amax(1) / 448
    rel = 2 * (_steps(K) / 2 + 8) * U
    assert ((scale.double() - s).abs() <= rel * s + 2.0 ** -149).all()
    code = (ref / scale.double()[:, None]).clamp(-448, 448)
    assert ((q.double() - code).abs() <= code.abs() * (2.0 ** -4 + 2 * (_steps(K) + 12) * U) + 2.0 ** -10 * 1.01).all()


def test_a_scale_that_is_no_float_is_a_zero_rows():
    """max|y| / 448 below the smallest denormal: scale 0 and zero codes."""
    T, K = 5, 64
    x = torch.full((T, K), 2.0 ** -10, device="cuda").to(B16)
    w = torch.full((K,), 2.0 ** -133, device="cuda").to(B16)
    q, scale = _nan(T, K, dtype=E4M3), _nan(T, dtype=torch.float32)
    api.forge_rmsnorm_fwd(x, w, 1.0, yq=q, yq_scale=scale)
    assert not scale.any() and not q.float().any()


@pytest.mark.parametrize("T,K", [(16, 512), (48, 5120), (640, 264)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_weight_that_is_not_finite_shows_in_scale_and_amax(T, K, bad):
    x, _, w = _inputs(T, K)
    w[K // 2 + 1] = bad
    y, q, scale = _nan(T, K), _nan(T, K, dtype=E4M3), torch.zeros(T, device="cuda")
    qt, amax = _nan(K, T, dtype=E4M3), torch.zeros(1, device="cuda")
    api.forge_rmsnorm_fwd(x, w, 1e-6, y=y, yq=q, yq_scale=scale)
    api.forge_rmsnorm_fwd(x, w, 1e-6, yt=qt, yt_scale=2.0 ** -5, amax=amax)
    assert torch.isnan(scale).all() and torch.isnan(q.float()).all() and torch.isnan(amax).all()
    rest = [k for k in range(K) if k != K // 2 + 1]  # bf16 and the codes of a given scale keep it to its column
    assert torch.isfinite(y[:, rest]).all() and torch.isfinite(qt.float()[rest]).all()
    assert not torch.isfinite(y[:, K // 2 + 1]).any()


@pytest.mark.parametrize("T", [48, 640])
def test_zero_rows_without_eps(T):
    """A row whose mean square plus eps is zero: rstd 0, so y, codes and scale are zero and its gradient is the stream's."""
    K = 512
    x, dh, w = _inputs(T, K)
    x[::5] = 0
    y, q, scale = _nan(T, K), _nan(T, K, dtype=E4M3), _nan(T, dtype=torch.float32)
    qt, amax, rstd = _nan(K, T, dtype=E4M3), _nan(1, dtype=torch.float32), _nan(T, dtype=torch.float32)
    r2 = torch.empty_like(rstd)
    api.forge_rmsnorm_fwd(x, w, 0.0, rstd=rstd, y=y, yq=q, yq_scale=scale)
    api.forge_rmsnorm_fwd(x, w, 0.0, rstd=r2, yt=qt, yt_scale=2.0 ** -5, amax=amax)
    for t in (y[::5], q.float()[::5], scale[::5], qt.float()[:, ::5], rstd[::5], r2[::5]):
        assert not t.any()
    assert all(torch.isfinite(t.float()).all() for t in (y, q, scale, qt, rstd, r2, amax)) and amax > 1
    dx, dw = _gradient(dh, x, w, rstd, dh)
    assert torch.equal(dx[::5], dh[::5]) and torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_token_contiguous_codes_of_a_scale_far_below_the_rows():
    """rstd / yt_scale past the largest float: zeros stay zero codes, the rest saturate."""
    T, K = 32, 512
    x, _, w = _inputs(T, K)
    x = x.clamp(-3, 3) * 2.0 ** -60
    x[:, ::3] = 0
    w = w.abs().clamp(0.125)
    qt = _nan(K, T, dtype=E4M3)
    api.forge_rmsnorm_fwd(x, w, 0.0, yt=qt, yt_scale=2.0 ** -100)
    assert torch.equal(qt.float(), (x.float().sign() * 448).t())


@pytest.mark.parametrize("T,K", [(32, 512), (640, 1024)])
@pytest.mark.parametrize("residual", [False, True])
def test_y_over_x(T, K, residual):
    """y may be x (or the residual): h and the codes are still those of the input."""
    x, res, w = _inputs(T, K)
    kw = dict(residual=res if residual else None)
    h, y, qt, q, scale = _nan(T, K), _nan(T, K), _nan(K, T, dtype=E4M3), _nan(T, K, dtype=E4M3), _nan(T, dtype=torch.float32)
    api.forge_rmsnorm_fwd(x, w, 1e-6, h=h, y=y, **kw)
    api.forge_rmsnorm_fwd(x, w, 1e-6, h=torch.empty_like(h), yt=qt, yt_scale=2.0 ** -5, **kw)
    api.forge_rmsnorm_fwd(x, w, 1e-6, h=torch.empty_like(h), yq=q, yq_scale=scale, **kw)
    for over in ("x", "residual") if residual else ("x",):
        a, b = x.clone(), res.clone()
        to = a if over == "x" else b
        h2, qt2, q2 = _nan(T, K), _nan(K, T, dtype=E4M3), _nan(T, K, dtype=E4M3)
        api.forge_rmsnorm_fwd(a, w, 1e-6, residual=b if residual else None, h=h2, y=to, yt=qt2, yt_scale=2.0 ** -5,
                              yq=q2, yq_scale=torch.empty_like(scale))
        assert torch.equal(h2, h) and torch.equal(to, y)
        # the two kernels sum a row in their own orders: a code may round apart where it lies between two
        assert ((qt2.double() - qt.double()).abs() <= 2.0 ** -3 * qt.double().abs() + 2.0 ** -9).all()
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("T,K", [(48, 1024), (48, 2048), (400, 4104), (700, 5120), (400, 8192), (64, 16384)])
def test_dx_over_dh(T, K):
    """The documented aliasing, in each variant of the kernel (two load a row ahead)."""
    h, dh, w = _inputs(T, K)
    dy = inputs.normal((T, K), 1e-2, 21, device="cuda")
    rstd = (h.float().square().mean(1) + 1e-6).rsqrt()
    dx, dw = _gradient(dy, h, w, rstd, dh)
    over, dw2 = dh.clone(), _nan(K, dtype=torch.float32)
    api.forge_rmsnorm_bwd(dy, h, w, rstd, over, dw2, _nan(api.forge_rmsnorm_bwd_workspace(T, K), dtype=torch.float32), dh=over)
    assert torch.equal(over, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("T,K", [(16, 520), (48, 4096), (112, 5128), (48, 16384), (400, 2048)])
@pytest.mark.parametrize("with_y", [False, True])
def test_h_over_its_inputs_with_token_contiguous_codes(T, K, with_y):
    """h over x and over the residual, T % 32 == 16 (the last tile repeats rows)."""
    x, res, w = _inputs(T, K)
    y = _nan(T, K) if with_y else None

    def call(a, b, h):
        qt, rstd = _nan(K, T, dtype=E4M3), _nan(T, dtype=torch.float32)
        api.forge_rmsnorm_fwd(a, w, 1e-6, residual=b, h=h, rstd=rstd, y=y, yt=qt, yt_scale=2.0 ** -5)
        return h, qt.view(torch.uint8), rstd, y.clone() if with_y else rstd

    want = call(x, res, _nan(T, K))
    assert torch.equal(want[0], (x.float() + res.float()).to(B16))
    a, b = x.clone(), res.clone()
    for got in (call(a, res, a), call(x, b, b)):
        assert all(torch.equal(i, j) for i, j in zip(got, want))
