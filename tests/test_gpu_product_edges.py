"""The product of E4M3 codes at its edges: a wait that runs out with results on their
way to memory (what was finished arrives whole, and nothing else is written), and
factors of two scales that float32 does not hold."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api
from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_codes import B16, blocks
from test_gpu_product_e4m3 import _exact, _powers, _product, _whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()
    api.forge_set_wait_limit_ns(200_000_000)
    api.forge_debug_skip_loads(False)
    yield
    api.forge_set_wait_limit_ns(0)


@pytest.mark.parametrize("N", [5120, 4936])
def test_results_under_way_when_a_wait_runs_out(N):
    """Every CTA pair finishes its first 256 x 256 tile, whose copies out of shared memory have then to end before
    the pair does, and waits in vain for the operands of its second."""
    T, K = 2049, 400
    a = _whole((T, K), 1), _powers((T, blocks(K)), 2), _whole((N, K), 3), _powers((blocks(N), blocks(K)), 4)
    want = _exact(*a)[0].float().to(B16)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    Y = torch.full((T + 1, N), 9.0, dtype=B16, device="cuda")
    Y[T] = 7
    api.forge_set_wait_limit_ns(20_000_000)
    assert api.lib().forge_debug_skip_loads(2) == 0
    try:
        api.forge_linear_e4m3(*a, Y[:T])
        with pytest.raises(api.ForgeError, match="TIMEOUT"):
            api.forge_get_device_status()
    finally:
        api.forge_debug_skip_loads(False)
        api.forge_set_wait_limit_ns(200_000_000)
    assert (Y[T] == 7).all()
    done = 0
    for t in range(0, T, 256):
        for n in range(0, N, 256):
            got, exact = Y[t:min(t + 256, T), n:n + 256], want[t:t + 256, n:n + 256]
            if torch.equal(got, exact):
                done += 1
            else:
                assert (got == 9).all(), (t, n)
    assert done == pairs  # of 9 x 20
    assert torch.equal(_product(*a), want)


@pytest.mark.parametrize("T,N", [(5, 264), (13, 2568), (24, 14344), (24, 9656), (24, 4104), (33, 4104), (300, 4104), (2049, 4936)])
def test_factors_out_of_float32s_range(T, N):
    """Scales whose product is no ordinary float32, though the values are, in every other row, so that a warp has
    both; at each width of the tiles.  One block of the reduction at a time, the others zero."""
    K = 528
    xq, wq = _whole((T, K), 1), _whole((N, K), 2)
    scales = ((2.0 ** -120, 2.0 ** -10), (2.0 ** 20, 2.0 ** -20), (2.0 ** 70, 2.0 ** 45), (2.0 ** -90, 2.0 ** -42), (2.0 ** -126, 2.0 ** 3))
    xs = torch.tensor([[s[0] for s in scales]] * T, device="cuda")
    xs[1::2] = 1.0
    ws = torch.tensor([[s[1] for s in scales]] * blocks(N), device="cuda")
    for b in range(len(scales)):
        x = torch.zeros_like(xq.float())
        x[:, b * 128:(b + 1) * 128] = xq.float()[:, b * 128:(b + 1) * 128]
        x = x.to(xq.dtype)
        want = _exact(x, xs, wq, ws)[0]
        assert want.abs().max() < 2.0 ** 127
        got = _product(x, xs, wq, ws)
        assert torch.equal(got, want.float().to(B16)), b
        assert torch.equal(got, _product(x, xs, wq, ws))
