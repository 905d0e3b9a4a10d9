"""E4M3 codes in blocks of 128, and back.

The scale is one float32 division and a maximum, the code one float32 reciprocal,
one product and one rounding, so both are torch's float32 bit for bit; against
64 bits a decoded value is off by half a step of its code (2^-4 of it, 2^-10 of
the scale below the smallest normal code) and three float32 roundings."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build

pytestmark = pytest.mark.gpu

B16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
LEAST = 2.0 ** -126
SHAPES = [(1, 8), (1, 128), (1, 4096), (3, 136), (129, 120), (300, 264), (128, 128), (257, 1032), (17, 5128), (2050, 640)]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def blocks(n):
    return (n + 127) // 128


def spread(scale, shape, rows):
    s = scale.repeat_interleave(128, 1)[:, :shape[1]]
    return s if rows == 1 else s.repeat_interleave(rows, 0)[:shape[0]]


def scales(x, rows):
    """max|x| / 448 of every block, in float32."""
    T, K = x.shape
    R = T if rows == 1 else blocks(T) * 128
    pad = torch.zeros((R, blocks(K) * 128), device=x.device)
    pad[:T, :K] = x.float().abs()
    most = pad.view(R // rows, rows, -1, 128).amax((1, 3))
    s = (most / torch.full_like(most, 448.0)).clamp(min=LEAST)
    return torch.where(most > 0, s, most) + (most - most)  # (an infinite maximum gives NaN)


def coded(T, K, rows, fill=0xFF):
    """Codes and scales with a guard row behind each, all NaN."""
    codes = torch.full((T + 1, K), fill, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.full(((T if rows == 1 else blocks(T)) + 1, blocks(K)), float("nan"), device="cuda")
    return codes, scale


def outliers(T, K, dtype, seed=3):
    x = inputs.normal((T, K), 1.0, seed, F32, "cuda") * torch.exp(2 * inputs.normal((K,), 1.0, seed + 1, F32, "cuda"))
    return x.to(dtype)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("T,K", SHAPES)
def test_codes_and_scales(T, K, dtype, rows):
    x = outliers(T, K, dtype)
    x[T // 2] = 0
    codes, scale = coded(T, K, rows)
    api.forge_quantize_e4m3(x, codes[:T], scale[:-1], block_rows=rows)
    want = scales(x, rows)
    assert torch.equal(scale[:-1], want) and torch.isnan(scale[-1]).all()
    inv = torch.where(want > 0, 1 / want, 0)
    q = (x.float() * spread(inv, x.shape, rows)).clamp(-448, 448).to(E4M3)
    assert torch.equal(codes[:T].view(torch.uint8), q.view(torch.uint8)) and (codes[T:].view(torch.uint8) == 0xFF).all()
    s = spread(want, x.shape, rows).double()
    off = (codes[:T].double() * s - x.double()).abs()
    assert (off <= x.double().abs() * (2.0 ** -4 + 2.0 ** -21) + s * 2.0 ** -10).all()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("T,K", SHAPES)
def test_values_of_codes(T, K, dtype, rows):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * K)
    codes = torch.randint(0, 256, (T, K), generator=g, device="cuda", dtype=torch.uint8).view(E4M3)  # NaN codes among them
    scale = inputs.normal((T if rows == 1 else blocks(T), blocks(K)), 1.0, 5, F32, "cuda")
    x = torch.full((T + 1, K), 7.0, dtype=dtype, device="cuda")
    api.forge_dequantize_e4m3(codes, scale, x[:T], block_rows=rows)
    want = (codes.float() * spread(scale, (T, K), rows)).to(dtype)
    assert torch.equal(torch.isnan(x[:T]), torch.isnan(want))
    assert torch.equal(x[:T].nan_to_num(), want.nan_to_num()) and (x[T] == 7).all()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [B16, F32])
def test_blocks_at_the_edges_of_the_floats(dtype, rows):
    """Blocks of the smallest and largest values, of zeros, and with values that are not finite."""
    T, K = 256, 9 * 128
    x = outliers(T, K, dtype)
    for b, size in enumerate((2.0 ** -133, 2.0 ** -126, 2.0 ** -120, 2.0 ** 100, 0.0)):
        x[:, b * 128:(b + 1) * 128] = (inputs.normal((T, 128), 0.5, b, F32, "cuda").clamp(-2, 2) * size).to(dtype)
    x[:, 5 * 128] = torch.finfo(dtype).max
    x[:, 6 * 128 + 1], x[:, 7 * 128 + 2] = float("inf"), float("nan")
    codes, scale = coded(T, K, rows)
    api.forge_quantize_e4m3(x, codes[:T], scale[:-1], block_rows=rows)
    scale = scale[:-1]
    assert torch.isnan(scale[:, 6:8]).all() and torch.isnan(codes[:T, 6 * 128:8 * 128].float()).all()
    assert (scale[:, 4] == 0).all() and (codes[:T, 4 * 128:5 * 128].float() == 0).all()
    assert (scale[:, :3] >= LEAST).all()
    ok = [c for b in (0, 1, 2, 3, 5, 8) for c in range(b * 128, b * 128 + 128)]
    s = spread(scale, x.shape, rows).double()[:, ok]
    off = (codes[:T].double()[:, ok] * s - x.double()[:, ok]).abs()
    assert (off <= x.double()[:, ok].abs() * (2.0 ** -4 + 2.0 ** -21) + s * 2.0 ** -10).all()
    back = torch.empty_like(x)
    api.forge_dequantize_e4m3(codes[:T], scale, back, block_rows=rows)
    assert torch.equal(torch.isnan(back), torch.isnan(spread(scale, x.shape, rows)))


def test_largest_index_in_use():
    """More than 2^32 bytes of values: offsets past 32 bits."""
    T, K = 65600, 32768
    x = torch.zeros((T, K), dtype=B16, device="cuda")
    x[-3:] = outliers(3, K, B16)
    codes, scale = coded(T, K, 1)
    api.forge_quantize_e4m3(x, codes[:T], scale[:-1])
    few, few_scale = coded(3, K, 1)
    api.forge_quantize_e4m3(x[-3:], few[:3], few_scale[:-1])
    assert torch.equal(codes[T - 3:T].view(torch.uint8), few[:3].view(torch.uint8)) and torch.equal(scale[-4:-1], few_scale[:-1])
    assert (scale[:T - 3] == 0).all()
    back = x.clone()
    api.forge_dequantize_e4m3(codes[:T], scale[:-1], back)
    assert torch.equal(back[-3:], (few[:3].float() * spread(few_scale[:-1], (3, K), 1)).to(B16)) and (back[:-3] == 0).all()


def test_captured_on_a_stream_of_its_own():
    x = outliers(33, 1032, B16)
    codes, scale = coded(33, 1032, 1)
    back = torch.empty_like(x)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        api.forge_quantize_e4m3(x, codes[:33], scale[:-1])
        api.forge_dequantize_e4m3(codes[:33], scale[:-1], back)
    for seed in (7, 8):
        x.copy_(outliers(33, 1032, B16, seed))
        graph.replay()
        torch.cuda.synchronize()
        a, s = coded(33, 1032, 1)
        api.forge_quantize_e4m3(x, a[:33], s[:-1])
        assert torch.equal(a.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s[:-1], scale[:-1])
        assert torch.equal(back, (a[:33].float() * spread(s[:-1], x.shape, 1)).to(B16))
