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
