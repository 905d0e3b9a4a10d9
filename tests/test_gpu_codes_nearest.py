"""What "to the nearest" means for the E4M3 codes: the scale's reciprocal and its product with x are rounded once
each, so x / scale is formed to within 2^-23 of itself, and no code lies nearer to the quotient in 64 bits than the
one written by more than twice that."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api
from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_codes import B16, F32, coded, outliers, spread

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("T,K", [(1, 4096), (300, 264), (2050, 640)])
def test_no_code_is_nearer(T, K, dtype, rows):
    x = outliers(T, K, dtype, seed=9)
    codes, scale = coded(T, K, rows)
    api.forge_quantize_e4m3(x, codes[:T], scale[:-1], block_rows=rows)
    every = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[~every.isnan()].unique()
    q = x.double() / spread(scale[:-1].double(), x.shape, rows)
    at = torch.searchsorted(every, q.contiguous()).clamp(1, every.numel() - 1)
    best = torch.minimum((every[at] - q).abs(), (every[at - 1] - q).abs())
    assert ((codes[:T].double() - q).abs() <= best + q.abs() * (2.0 ** -22 + 2.0 ** -46)).all()
