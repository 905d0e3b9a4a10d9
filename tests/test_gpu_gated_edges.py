"""The gate where its sigmoid leaves float32's normal range, and values that are not finite.

Bounds: e = exp(-|z|) carries 2^-22 and |z| 2^-23 of itself, at most 2^-16 for |z| < 110, z of the tanh form four
float32 roundings of itself, at most 2^-15 of e; what follows adds a few 2^-24: 2^-14 of the value in all.  Below
2^-126 e is a multiple of 2^-149 and off by two of them, times |g| (and the slope's d).  Then bf16's 2^-8 of the
value, or half a step of its numbers below 2^-126, 2^-134."""

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api, inputs
from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_codes import B16, blocks
from test_gpu_gated import ACTS, act, decoded, forward, gradient

pytestmark = pytest.mark.gpu

# SiLU from 2^-113 (g = -83) to below bf16's smallest; the tanh form likewise from z = -80 on
FAR = {"silu": [-83.0 - i / 2 for i in range(48)], "gelu_tanh": [-9.625 - i / 16 for i in range(48)]}


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    api.lib()


def close(got, want, small):
    """small: what 2^-149 of e makes of the value."""
    assert ((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -134 + small * 2.0 ** -148).all(), \
        ((got.double() - want).abs() / want.abs()).max()


@pytest.mark.parametrize("u", [1.0, 2.0 ** 12])
@pytest.mark.parametrize("kind", ACTS)
def test_small_gates_forward(kind, u):
    """G and U are single products, so exact; few rows, and tiles with each kind of what is kept."""
    g = torch.tensor(FAR[kind], device="cuda").to(B16)
    F = g.numel()
    W = torch.zeros((2 * F, 8), dtype=B16, device="cuda")
    W[:F, 0], W[F:, 0] = g, u
    want = act(kind, g.double())[0] * u
    assert (want.abs() > 2.0 ** -126).sum() >= 8 and (want.abs() < 2.0 ** -126 * u).sum() >= 8
    for T, keep in ((5, "none"), (40, "none"), (40, "bf16"), (40, "e4m3")):
        X = torch.zeros((T, 8), dtype=B16, device="cuda")
        X[:, 0] = 1
        Y = forward(X, W, kind, keep)[0]
        close(Y, want.expand(T, F), g.double().abs() * u)


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ACTS)
def test_small_gates_gradient(kind, keep):
    g = torch.tensor(FAR[kind], device="cuda").to(B16)
    T, F = 40, g.numel()
    gu = torch.ones((T, 2 * F), dtype=B16, device="cuda")
    gu[:, :F] = g
    args, v = dict(gu=gu), gu.double()
    if keep == "e4m3":
        codes, scale = torch.empty((2 * T, F), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((2 * T, blocks(F)), device="cuda")
        api.forge_quantize_e4m3(gu.view(2 * T, F), codes, scale)
        args = dict(codes=codes.view(T, 2 * F), scale=scale.view(T, 2, -1))
        v = decoded(args["codes"], args["scale"])
    dY, Wd = torch.ones((T, 8), dtype=B16, device="cuda"), torch.full((8, F), 0.125, dtype=B16, device="cuda")
    dGU, Y = gradient(dY, Wd, kind, **args)  # dA = 1
    g, u = v[:, :F], v[:, F:]
    a, slope = act(kind, g)
    close(dGU[:, F:], a, g.abs())
    close(Y, a * u, (g * u).abs())
    close(dGU[:, :F], slope * u, (1 + 40 * g.abs()) * u.abs())


@pytest.mark.parametrize("keep", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("T", [5, 24, 40, 300])
def test_values_that_are_not_finite_stay_where_they_are(T, keep):
    """A NaN in a token spoils its row, a NaN in a weight its feature, and repeating the call gives the same bits."""
    F, K = 264, 136
    X, W = inputs.normal((T, K), 1.0, 1, device="cuda"), inputs.normal((2 * F, K), 0.1, 2, device="cuda")
    X[T - 1, 7], X[1, K - 1], W[33, 70], W[F + 200, 0] = (float("nan"),) * 4
    Y, gu, codes, scale = forward(X, W, "silu", keep)
    bad = torch.zeros((T, F), dtype=torch.bool, device="cuda")
    bad[T - 1] = bad[1] = True
    bad[:, 33] = bad[:, 200] = True
    assert torch.equal(torch.isnan(Y), bad)
    if keep == "bf16":
        both = torch.zeros((T, 2 * F), dtype=torch.bool, device="cuda")
        both[T - 1] = both[1] = True
        both[:, 33] = both[:, F + 200] = True
        assert torch.equal(torch.isnan(gu), both)
    if keep == "e4m3":
        rows = torch.isnan(scale)
        assert rows[T - 1].all() and rows[1].all() and rows[:, 0, 0].all() and rows[:, 1, 1].all()
        assert not rows[0, 0, 1:].any() and not rows[0, 1, 0] and not rows[0, 1, 2]
    for a, b in zip((Y, gu, codes, scale), forward(X, W, "silu", keep)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
