"""Refusals of the gated feed-forward products, the E4M3 codes and their product,
on the host: no argument below reaches a CUDA call, so the pointers are never
followed."""

import ctypes

import pytest
import torch

from optimizer_tcgen05_dw_gb300 import api
from optimizer_tcgen05_dw_gb300.build import build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build()
    return api.lib()


def _message(L):
    return L.forge_last_error_message().decode()


SHARED = [
    (dict(T=-1), 1, "negative"), (dict(F=-8), 1, "negative"), (dict(F=12), 1, "multiples of 8"),
    (dict(act=2), 1, "act 2"), (dict(act=-1), 1, "act -1"), (dict(T=1 << 31), 2, "31 bits"), (dict(F=1 << 30), 2, "31 bits"),
    (dict(gu=FAKE, gu_codes=FAKE, gu_scale=FAKE), 1, "one of them"), (dict(gu=None, gu_codes=FAKE), 1, "go together"),
    (dict(gu=None, gu_scale=FAKE), 1, "go together"), (dict(gu=FAKE + 8), 1, "gu must be 16-byte"),
    (dict(gu=None, gu_codes=FAKE + 8, gu_scale=FAKE), 1, "gu_codes must be"),
    (dict(gu=None, gu_codes=FAKE, gu_scale=FAKE + 2), 1, "gu_scale must be 4-byte"), (dict(Y=FAKE + 2), 1, "Y must be")]


@pytest.mark.parametrize("change,status,word", SHARED + [
    (dict(K=-8), 1, "negative"), (dict(K=4), 1, "multiples of 8"), (dict(K=1 << 31), 2, "31 bits"), (dict(X=0), 1, "X is NULL"),
    (dict(W=FAKE + 8), 1, "W must be"), (dict(Y=0), 1, "Y is NULL"), (dict(T=1 << 30, F=1 << 29), 2, "tiles")])
def test_gated_refusals(L, change, status, word):
    a = dict(T=16, F=64, K=128, act=0, X=FAKE, W=FAKE, Y=FAKE, gu=FAKE)
    a.update(change)
    rc = L.forge_gated_linear(ctypes.byref(api.ForgeGated(**a)), None)
    assert rc == status and word in _message(L), (rc, _message(L))


@pytest.mark.parametrize("change,status,word", SHARED + [
    (dict(N=-8), 1, "negative"), (dict(N=4), 1, "multiples of 8"), (dict(N=1 << 31), 2, "31 bits"), (dict(N=0), 2, "N > 0"),
    (dict(dY=0), 1, "dY is NULL"), (dict(Wd=FAKE + 8), 1, "Wd must be"), (dict(dGU=0), 1, "dGU is NULL"),
    (dict(dGU=FAKE + 4), 1, "dGU must be"), (dict(gu=None), 1, "gu or gu_codes is needed")])
def test_gated_gradient_refusals(L, change, status, word):
    a = dict(T=16, F=64, N=128, act=1, dY=FAKE, Wd=FAKE, gu=FAKE, dGU=FAKE)
    a.update(change)
    rc = L.forge_gated_dgrad(ctypes.byref(api.ForgeGatedGrad(**a)), None)
    assert rc == status and word in _message(L), (rc, _message(L))


@pytest.mark.parametrize("change,status,word", [
    (dict(rows=-1), 1, "negative"), (dict(cols=-8), 1, "negative"), (dict(cols=12), 1, "multiple of 8"), (dict(dt=2), 1, "x_dtype"),
    (dict(block=64), 1, "block_rows"), (dict(rows=1 << 31), 2, "31 bits"), (dict(cols=1 << 31), 2, "31 bits"),
    (dict(rows=1 << 30, cols=1 << 30), 2, "31 bits"), (dict(rows=1 << 21, cols=1 << 20, block=1), 2, "in 40"), (dict(x=None), 1, "x is NULL"), (dict(x=FAKE + 8), 1, "x must be"),
    (dict(codes=None), 1, "codes is NULL"), (dict(codes=FAKE + 8), 1, "codes must be"), (dict(scale=None), 1, "scale is NULL"),
    (dict(scale=FAKE + 1), 1, "scale must be 4-byte")])
def test_codes_refusals(L, change, status, word):
    a = dict(x=FAKE, dt=1, codes=FAKE, scale=FAKE, rows=16, cols=128, block=1)
    a.update(change)
    for rc in (L.forge_quantize_e4m3(a["x"], a["dt"], a["codes"], a["scale"], a["rows"], a["cols"], a["block"], None),
               L.forge_dequantize_e4m3(a["codes"], a["scale"], a["x"], a["dt"], a["rows"], a["cols"], a["block"], None)):
        assert rc == status and word in _message(L), (rc, _message(L))


@pytest.mark.parametrize("change,status,word", [
    (dict(T=-1), 1, "negative"), (dict(N=12), 1, "N must be a multiple of 8"), (dict(K=24), 1, "K of 16"),
    (dict(K=1 << 31), 2, "31 bits"), (dict(Xq=0), 1, "Xq is NULL"), (dict(Wq=FAKE + 8), 1, "Wq must be"),
    (dict(x_scale=0), 1, "x_scale is NULL"), (dict(w_scale=FAKE + 2), 1, "w_scale must be 4-byte"), (dict(Y=0), 1, "Y is NULL"),
    (dict(Y=FAKE + 8), 1, "Y must be"), (dict(T=1 << 30, N=1 << 30), 2, "tiles")])
def test_product_refusals(L, change, status, word):
    a = dict(T=16, N=64, K=128, Xq=FAKE, x_scale=FAKE, Wq=FAKE, w_scale=FAKE, Y=FAKE)
    a.update(change)
    rc = L.forge_linear_e4m3(ctypes.byref(api.ForgeLinearE4m3(**a)), None)
    assert rc == status and word in _message(L), (rc, _message(L))


def test_nothing_to_do_needs_no_device(L):
    assert L.forge_gated_linear(ctypes.byref(api.ForgeGated(T=0, F=8, K=8)), None) == 0
    assert L.forge_gated_linear(ctypes.byref(api.ForgeGated(T=8, F=0, K=8)), None) == 0
    assert L.forge_gated_dgrad(ctypes.byref(api.ForgeGatedGrad(T=0, F=8, N=8)), None) == 0
    assert L.forge_quantize_e4m3(None, 1, None, None, 0, 8, 1, None) == 0
    assert L.forge_dequantize_e4m3(None, None, None, 1, 8, 0, 128, None) == 0
    assert L.forge_linear_e4m3(ctypes.byref(api.ForgeLinearE4m3(T=0, N=8, K=16)), None) == 0


def test_null_structs(L):
    assert L.forge_gated_linear(None, None) == 1 and L.forge_gated_dgrad(None, None) == 1
    assert L.forge_linear_e4m3(None, None) == 1


def test_the_binding_refuses_what_the_library_could_not_see():
    b = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    e = lambda *n: torch.zeros(n).to(torch.float8_e4m3fn)  # noqa: E731
    f = torch.zeros
    with pytest.raises(ValueError, match="act"):
        api._act("relu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.forge_gated_linear(b(4, 8), b(16, 8), b(4, 8))
    with pytest.raises(ValueError, match=r"W: expected shape \(16, 8\)"):
        api.forge_gated_linear(_cuda(b(4, 8)), b(17, 8), b(4, 8))
    with pytest.raises(TypeError, match="W: expected"):
        api.forge_gated_linear(_cuda(b(4, 8)), f(16, 8), b(4, 8))
    with pytest.raises(ValueError, match=r"\[T, K\]"):
        api.forge_gated_linear(b(8), b(16, 8), b(4, 8))
    with pytest.raises(ValueError, match="one of them"):
        api._kept(4, 8, b(4, 16), e(4, 16), f(4, 2, 1))
    with pytest.raises(ValueError, match="gu_scale is required"):
        api._kept(4, 8, None, _cuda(e(4, 16)), None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.forge_gated_dgrad(b(4, 8), b(8, 16), b(4, 32), gu=b(4, 32))
    with pytest.raises(ValueError, match="block_rows"):
        api.forge_quantize_e4m3(f(4, 8), e(4, 8), f(4, 1), block_rows=64)
    with pytest.raises(TypeError, match="x: expected"):
        api.forge_quantize_e4m3(f(4, 8).half(), e(4, 8), f(4, 1))
    with pytest.raises(ValueError, match="contiguous"):
        api.forge_dequantize_e4m3(e(4, 8), f(4, 1), f(8, 4).t())
    with pytest.raises(TypeError, match="Xq: expected"):
        api.forge_linear_e4m3(torch.zeros((4, 16), dtype=torch.uint8), f(4, 1), e(8, 16), f(1, 1), b(4, 8))


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    t = torch.zeros(4)  # (on the host: device -1)
    with pytest.raises(ValueError, match="current device, cuda:1"):
        api._here(None, t)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    api._here(t, None)
    calls = []
    monkeypatch.setattr(api, "_here", lambda *a: calls.append(len(a)) or (_ for _ in ()).throw(ValueError("elsewhere")))
    b, e, f = (lambda *n, d=d: _cuda(torch.zeros(n).to(d)) for d in (torch.bfloat16, torch.float8_e4m3fn, torch.float32))
    for call in (lambda: api.forge_gated_linear(b(4, 8), b(16, 8), b(4, 8)), lambda: api.forge_gated_dgrad(b(4, 8), b(8, 16), b(4, 32), gu=b(4, 32)),
                 lambda: api.forge_quantize_e4m3(f(4, 8), e(4, 8), f(4, 1)), lambda: api.forge_dequantize_e4m3(e(4, 8), f(4, 1), b(4, 8)),
                 lambda: api.forge_linear_e4m3(e(4, 16), f(4, 1), e(8, 16), f(1, 1), b(4, 8))):
        with pytest.raises(ValueError, match="elsewhere"):
            call()
    assert calls == [6, 7, 3, 3, 5]


class _cuda(torch.Tensor):
    """A host tensor that says it is on the device, for the checks behind that one."""

    @staticmethod
    def __new__(cls, t):
        return t.as_subclass(cls)

    is_cuda = True
