"""The product of E4M3 codes with a scale for each block of 128.

Small whole codes and scales that are powers of two make every float32 partial
sum exact, so Y is the correctly rounded bf16 of the exact sum.  On normal data
a sum of K terms carries one rounding (2^-23, were it a truncation) for each
instruction of 32 terms, each fold of a block and each of the two scales:
(K / 32 + K / 128 + 4) 2^-23 of the sum of magnitudes, then bf16's 2^-8."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_codes import B16, E4M3, F32, blocks, spread

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8, 16), (1, 4096, 256), (2, 128, 128), (5, 264, 144), (33, 72, 2064), (128, 512, 384), (129, 1000, 400),
          (256, 256, 128), (257, 2056, 1040), (300, 640, 4096), (2049, 520, 272), (1531, 5120, 656)]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()
    api.forge_set_wait_limit_ns(200_000_000)
    api.forge_debug_skip_loads(False)
    yield
    api.forge_set_wait_limit_ns(0)


def _product(xq, xs, wq, ws):
    """Y, with a guard row behind it that has to stay as it was."""
    T, N = xq.shape[0], wq.shape[0]
    Y = torch.full((T + 1, N), float("nan"), dtype=B16, device="cuda")
    Y[T] = 7
    api.forge_linear_e4m3(xq, xs, wq, ws, Y[:T])
    api.forge_get_device_status()
    assert (Y[T] == 7).all()
    return Y[:T]


def _exact(xq, xs, wq, ws):
    x = xq.double() * spread(xs.double(), xq.shape, 1)
    w = wq.double() * spread(ws.double(), wq.shape, 128)
    return x @ w.t(), x.abs() @ w.abs().t()


def _whole(shape, seed):
    return inputs.integer_grid(shape, -4, 4, 0, seed, dtype=F32, device="cuda").to(E4M3)


def _powers(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.exp2(torch.randint(-3, 4, shape, generator=g, device="cuda").float())


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_exact_sums(T, N, K):
    a = _whole((T, K), 1), _powers((T, blocks(K)), 2), _whole((N, K), 3), _powers((blocks(N), blocks(K)), 4)
    assert torch.equal(_product(*a), _exact(*a)[0].float().to(B16))


def _random(T, N, K, seed=1):
    x, w = inputs.normal((T, K), 1.0, seed, device="cuda"), inputs.normal((N, K), 0.02, seed + 1, device="cuda")
    xq, wq = torch.empty((T, K), dtype=E4M3, device="cuda"), torch.empty((N, K), dtype=E4M3, device="cuda")
    xs, ws = torch.empty((T, blocks(K)), device="cuda"), torch.empty((blocks(N), blocks(K)), device="cuda")
    api.forge_quantize_e4m3(x, xq, xs)
    api.forge_quantize_e4m3(w, wq, ws, block_rows=128)
    return xq, xs, wq, ws


@pytest.mark.parametrize("T,N,K", SHAPES + [(77, 4096, 14336), (4099, 1024, 512)])
def test_normal_data(T, N, K):
    a = _random(T, N, K)
    want, size = _exact(*a)
    off = (_product(*a).double() - want).abs()
    assert (off <= want.abs() * 2.0 ** -8 + size * ((K / 32 + K / 128 + 4) * 2.0 ** -23)).all()


@pytest.mark.parametrize("N,K", [(2432, 2064), (2440, 272), (4104, 1040)])
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16, 17, 32])
def test_exact_sums_of_few_rows(T, N, K):
    """On either side of the rows, and of the features (16 for each of 152 SMs), at which another form takes over."""
    a = _whole((T, K), 1), _powers((T, blocks(K)), 2), _whole((N, K), 3), _powers((blocks(N), blocks(K)), 4)
    assert torch.equal(_product(*a), _exact(*a)[0].float().to(B16))


def test_factors_out_of_float32s_range():
    """Scales whose product is not a normal float32, though the values are."""
    T, N, K = 8, 128, 512
    xq, wq = _whole((T, K), 1), _whole((N, K), 2)
    xq[:, 256:384] = torch.zeros((), device="cuda").to(E4M3)
    pairs = ((2.0 ** -126, 2.0 ** -12), (2.0 ** 20, 2.0 ** -20), (2.0 ** 100, 2.0 ** 100), (2.0 ** -90, 2.0 ** -45))
    xs = torch.tensor([[p[0] for p in pairs]] * T, device="cuda")
    ws = torch.tensor([[p[1] for p in pairs]], device="cuda")
    for keep in range(4):  # one block at a time, the others zero
        x = torch.zeros_like(xq.float())
        cut = slice(keep * 128, keep * 128 + 128)
        x[:, cut] = xq.float()[:, cut]
        x = x.to(E4M3)
        assert torch.equal(_product(x, xs, wq, ws), _exact(x, xs, wq, ws)[0].to(B16))


def test_values_that_are_not_finite():
    """A NaN scale or code shows in its row (or its columns) alone."""
    xq, xs, wq, ws = _random(130, 264, 400)
    xs[3, 1] = float("nan")
    xq.view(torch.uint8)[70, 17] = 0x7F
    ws[2, 0] = float("nan")
    bad = torch.isnan(_product(xq, xs, wq, ws))
    want = torch.zeros_like(bad)
    want[3], want[70], want[:, 256:] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T", [6, 13])
def test_values_that_are_not_finite_in_few_rows(T):
    """The same in the products of a few rows; codes of either sign, in each place of a word."""
    xq, xs, wq, ws = _random(T, 2568, 2064)
    for t, k in ((0, 3), (2, 130), (5, 2061)):
        xq.view(torch.uint8)[t, k] = 0x7F if t else 0xFF
    wq.view(torch.uint8)[2567, 17], wq.view(torch.uint8)[40, 2062] = 0xFF, 0x7F
    ws[3, 1] = float("nan")
    xs[T - 2, 16] = float("nan")
    bad = torch.isnan(_product(xq, xs, wq, ws))
    want = torch.zeros_like(bad)
    want[[0, 2, 5, T - 2]] = True
    want[:, [2567, 40]] = True
    want[:, 384:512] = True
    assert torch.equal(bad, want)


def test_nothing_to_sum_and_nothing_to_do():
    e = lambda *s, d=F32: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    Y = torch.full((3, 16), 5.0, dtype=B16, device="cuda")
    api.forge_linear_e4m3(e(3, 0, d=E4M3), e(3, 0), e(16, 0, d=E4M3), e(1, 0), Y)
    assert (Y == 0).all()
    api.forge_linear_e4m3(e(0, 16, d=E4M3), e(0, 1), e(16, 16, d=E4M3), e(1, 1), e(0, 16, d=B16))
    api.forge_linear_e4m3(e(3, 16, d=E4M3), e(3, 1), e(0, 16, d=E4M3), e(0, 1), e(3, 0, d=B16))
    api.forge_get_device_status()


def test_a_wait_that_runs_out_is_reported():
    a = _random(40, 264, 400)
    api.forge_set_wait_limit_ns(20_000_000)
    api.forge_debug_skip_loads(True)
    try:
        Y = torch.zeros((40, 264), dtype=B16, device="cuda")
        api.forge_linear_e4m3(*a, Y)
        with pytest.raises(api.ForgeError, match="TIMEOUT"):
            api.forge_get_device_status()
    finally:
        api.forge_debug_skip_loads(False)
        api.forge_set_wait_limit_ns(200_000_000)
    want, size = _exact(*a)
    assert ((_product(*a).double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -18).all()


def test_captured_two_streams():
    """Two captured calls in flight together, replayed on new values."""
    a, b = _random(100, 520, 656, 11), _random(9, 1032, 272, 21)
    ya, yb = torch.empty((100, 520), dtype=B16, device="cuda"), torch.empty((9, 1032), dtype=B16, device="cuda")
    graphs, streams = [], []
    for args, y in ((a, ya), (b, yb)):
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            api.forge_linear_e4m3(*args, y)
        graphs.append(graph)
        streams.append(stream)
    for seed in (31, 41):
        for to, new in zip(a + b, _random(100, 520, 656, seed) + _random(9, 1032, 272, seed + 1)):
            to.copy_(new)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, _product(*a)) and torch.equal(yb, _product(*b))
