"""The gated products and the product of codes on tensors of more than 2^31
elements (more than 2^32 bytes): 219 equal batches of 300 rows, each of which has
to come out as one batch alone does.  Whole numbers, so that sums are exact and do
not depend on the tiles they are formed in."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_codes import B16, E4M3, blocks
from test_gpu_product_e4m3 import _powers, _whole

pytestmark = pytest.mark.gpu

T, TIMES, F, K = 300, 219, 32776, 16  # 65700 x 32776: 2.15e9


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def new(rows, cols, dtype=B16):
    return torch.empty((rows, cols), dtype=dtype, device="cuda")


def same(many, one):
    """Every batch of `many` has the bytes of `one`."""
    a, b = many.view(torch.uint8).view(TIMES, -1), one.contiguous().view(torch.uint8).view(-1)
    return all(torch.equal(row, b) for row in a)


def batch():
    return inputs.integer_grid((T, K), -4, 4, 0, 3, device="cuda"), inputs.integer_grid((2 * F, K), -4, 4, -4, 4, device="cuda")


def test_forward_and_gradient_bf16():
    X, W = batch()
    Y, gu = new(T, F), new(T, 2 * F)
    api.forge_gated_linear(X, W, Y, gu=gu)
    Ys, gus = new(T * TIMES, F), new(T * TIMES, 2 * F)
    api.forge_gated_linear(X.repeat(TIMES, 1), W, Ys, gu=gus)
    assert same(Ys, Y) and same(gus, gu)
    dY, Wd = inputs.integer_grid((T, K), -4, 4, 0, 5, device="cuda"), inputs.integer_grid((K, F), -4, 4, -4, 6, device="cuda")
    dGU, Y2 = new(T, 2 * F), new(T, F)
    api.forge_gated_dgrad(dY, Wd, dGU, gu=gu, Y=Y2)
    api.forge_gated_dgrad(dY.repeat(TIMES, 1), Wd, gus, gu=gus, Y=Ys)  # (over what was kept)
    api.forge_get_device_status()
    assert same(gus, dGU) and same(Ys, Y2)


def test_forward_and_gradient_codes():
    X, W = batch()
    kept = lambda n: (new(n, 2 * F, E4M3), torch.empty((n, 2, blocks(F)), device="cuda"))  # noqa: E731
    (codes, scale), (many, scales) = kept(T), kept(T * TIMES)
    Y, Ys = new(T, F), new(T * TIMES, F)
    api.forge_gated_linear(X, W, Y, gu_codes=codes, gu_scale=scale)
    api.forge_gated_linear(X.repeat(TIMES, 1), W, Ys, gu_codes=many, gu_scale=scales)
    assert same(Ys, Y) and same(many, codes) and same(scales, scale)
    dY, Wd = inputs.integer_grid((T, K), -4, 4, 0, 5, device="cuda"), inputs.integer_grid((K, F), -4, 4, -4, 6, device="cuda")
    dGU, dGUs = new(T, 2 * F), new(T * TIMES, 2 * F)
    api.forge_gated_dgrad(dY, Wd, dGU, gu_codes=codes, gu_scale=scale, Y=Y)
    api.forge_gated_dgrad(dY.repeat(TIMES, 1), Wd, dGUs, gu_codes=many, gu_scale=scales, Y=Ys)
    api.forge_get_device_status()
    assert same(dGUs, dGU) and same(Ys, Y)


def test_product():
    xq, xs, wq, ws = _whole((T, K), 1), _powers((T, 1), 2), _whole((F, K), 3), _powers((blocks(F), 1), 4)
    Y, Ys = new(T, F), new(T * TIMES, F)
    api.forge_linear_e4m3(xq, xs, wq, ws, Y)
    api.forge_linear_e4m3(xq.view(torch.uint8).repeat(TIMES, 1).view(E4M3), xs.repeat(TIMES, 1), wq, ws, Ys)
    api.forge_get_device_status()
    x, w = xq.double() * xs.double(), wq.double() * ws.double().repeat_interleave(128, 0)[:F]
    assert torch.equal(Y, (x @ w.t()).to(B16)) and same(Ys, Y)
