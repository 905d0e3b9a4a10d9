"""The gated products and the product of codes at every width of their tiles.

The host chooses a width (128, 64 or 32) by the shape; each one is a kernel of
its own, with rings of shared-memory stages of its own depth, for up to 32 token
rows another one.  Here every form does more stages a CTA pair than its ring
holds, so that stages are reused, with several tiles a pair and ends of rows and
columns that cut a tile.  Whole-number operands make the sums exact: what is kept
of them has to be right to the bit, and gate and gradient within the gate's own
error (2^-17 of a value, see test_gpu_gated) and one rounding to bf16."""

import ctypes

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build, lib_path
from test_gpu_codes import B16, E4M3, blocks
from test_gpu_gated import ACTS, act, forward, gradient, kept
from test_gpu_product_e4m3 import _exact, _powers, _product, _whole

pytestmark = pytest.mark.gpu

# width for 76 pairs; tokens, features, reduction
FORWARD = [(128, 2049, 520, 1032), (128, 2049, 2456, 520), (64, 1100, 2056, 1032), (32, 33, 2056, 1032),
           (128, 24, 9720, 1032), (128, 24, 17416, 520), (64, 24, 4856, 2056), (64, 24, 14344, 1032), (32, 24, 2056, 2056)]
GRADIENT = [(128, 1000, 9216, 520), (128, 1000, 9152, 520), (128, 1000, 9224, 520), (128, 2049, 5000, 264),
            (64, 600, 2048, 1032), (64, 600, 2056, 1032)]
PRODUCT = [(128, 2049, 5120, 656), (128, 2049, 5000, 1040), (128, 2049, 4936, 1040), (64, 300, 4104, 2064), (32, 33, 4104, 2064),
           (128, 24, 14344, 2064), (64, 24, 9656, 4112), (64, 24, 19464, 2064), (32, 24, 4104, 4112)]
HALVES, LEAST = dict(forward=1, gradient=2, product=2), dict(forward=32, gradient=64, product=32)


def width_of(op, T, cols, pairs):
    tk = ctypes.CDLL(lib_path("libforge_testkit.so"))
    tk.forge_testkit_pick_width.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    return tk.forge_testkit_pick_width(T, cols, HALVES[op], LEAST[op], pairs)


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()
    api.forge_set_wait_limit_ns(200_000_000)
    api.forge_debug_skip_loads(False)
    yield
    api.forge_set_wait_limit_ns(0)


def _grid(shape, low, seed):
    return inputs.integer_grid(shape, -4, 4, low, seed, device="cuda")


@pytest.mark.parametrize("width,T,F,K", FORWARD)
def test_forward(width, T, F, K):
    X, W = _grid((T, K), 0, 3), _grid((2 * F, K), -8, 4)
    want = X.double() @ W.double().t()
    y = act("silu", want[:, :F])[0] * want[:, F:]
    Y, gu, _, _ = forward(X, W, "silu", "bf16")
    assert torch.equal(gu, want.to(B16))
    assert ((Y.double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -17) + 2.0 ** -134).all()
    alone, _, _, _ = forward(X, W, "silu", "none")
    coded, _, codes, scale = forward(X, W, "silu", "e4m3")
    assert torch.equal(alone, Y) and torch.equal(coded, Y)
    c, s = torch.empty((2 * T, F), dtype=E4M3, device="cuda"), torch.empty((2 * T, blocks(F)), device="cuda")
    api.forge_quantize_e4m3(want.float().view(2 * T, F), c, s)
    assert torch.equal(scale.reshape(-1), s.view(-1))
    assert torch.equal(codes.view(torch.uint8).reshape(-1), c.view(torch.uint8).view(-1))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("width,T,F,N", GRADIENT)
def test_gradient(width, T, F, N, keep):
    dY, Wd = _grid((T, N), 0, 6), _grid((N, F), -8, 7)
    args, gu = kept(T, F, keep)
    da, g, u = dY.double() @ Wd.double(), gu[:, :F], gu[:, F:]
    for kind in ACTS:
        got, y = gradient(dY, Wd, kind, **args)
        a, slope = act(kind, g)
        for have, want, room in ((got[:, :F], da * u * slope, (da * u).abs()), (got[:, F:], da * a, (da * a).abs()),
                                 (y, a * u, (a * u).abs())):
            assert ((have.double() - want).abs() <= want.abs() * 2.0 ** -8 + room * 2.0 ** -17 + 2.0 ** -134).all()


@pytest.mark.parametrize("width,T,N,K", PRODUCT)
def test_product(width, T, N, K):
    a = _whole((T, K), 1), _powers((T, blocks(K)), 2), _whole((N, K), 3), _powers((blocks(N), blocks(K)), 4)
    assert torch.equal(_product(*a), _exact(*a)[0].float().to(B16))


def test_the_shapes_reach_every_width():
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    for op, table in (("forward", FORWARD), ("gradient", GRADIENT), ("product", PRODUCT)):
        for width, T, cols, _ in table:
            assert width_of(op, T, cols, pairs) == width, (op, T, cols)
