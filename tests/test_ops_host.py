"""Refusals of the operators around the linear step, on the host: no argument
below reaches a CUDA call, so the pointers are never followed."""

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


def _multi(L, items, wd=0, gd=0, sd=0, kind="adamw", step=1, hp=None, count=None):
    table = (api.ForgeTensor * max(1, len(items)))(*items)
    hp = api.hparams() if hp is None else hp
    return L.forge_multi_opt_step(table, len(items) if count is None else count, wd, gd, sd, api.OPT_KINDS[kind],
                                  ctypes.byref(hp), step, 0, None)


@pytest.mark.parametrize("change,kw,status,word", [
    (dict(n=-1), {}, 1, "n = -1"), (dict(W=0), {}, 1, "W must be"), (dict(W=FAKE + 4), {}, 1, "W must be"),
    (dict(grad=FAKE + 2), {}, 1, "grad must be"), (dict(s1=0), {}, 1, "needs s1"), (dict(s2=0), {}, 1, "needs s2"),
    (dict(), dict(wd=7), 1, "w_dtype"), (dict(), dict(gd=2), 1, "g_dtype"), (dict(), dict(sd=9), 1, "s_dtype"),
    (dict(), dict(sd=1), 1, "s1_scale"), (dict(), dict(step=0), 1, "step"), (dict(), dict(count=-1), 1, "count"),
    (dict(n=1 << 50), {}, 2, "2^41")])
def test_multi_refusals(L, change, kw, status, word):
    item = dict(n=100, grad=FAKE, W=FAKE, s1=FAKE, s2=FAKE)
    item.update(change)
    rc = _multi(L, [api.ForgeTensor(**item)], **kw)
    assert rc == status and word in _message(L), (rc, _message(L))


def test_multi_nothing_to_do_needs_no_device(L):
    assert _multi(L, []) == 0
    assert _multi(L, [api.ForgeTensor(0, None, None, None, None, None, None)]) == 0


@pytest.mark.parametrize("change,status,word", [
    (dict(T=-1), 1, "negative T"), (dict(K=12), 1, "multiple of 8"), (dict(K=0), 1, "multiple of 8"),
    (dict(K=16392), 2, "16384"), (dict(T=1 << 31), 2, "2^31"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(x=0), 1, "x is NULL"), (dict(w=FAKE + 8), 1, "w must be"),
    (dict(residual=FAKE), 1, "needs h"), (dict(yq=FAKE), 1, "go together"), (dict(yq_scale=FAKE), 1, "go together"),
    (dict(T=24, yt=FAKE), 1, "T % 16"), (dict(yt=FAKE, yt_scale=0.0), 1, "yt_scale"),
    (dict(yt=FAKE, yt_scale=1e-45), 1, "yt_scale"), (dict(amax=FAKE), 1, "output of yt"),
    (dict(y=FAKE + 1), 1, "y must be")])
def test_norm_refusals(L, change, status, word):
    a = dict(T=16, K=64, x=FAKE, w=FAKE, eps=1e-6, yt_scale=1.0)
    a.update(change)
    rc = L.forge_rmsnorm_fwd(ctypes.byref(api.ForgeRmsnorm(**a)), None)
    assert rc == status and word in _message(L), (rc, _message(L))


@pytest.mark.parametrize("change,status,word", [
    (dict(K=20), 1, "multiple of 8"), (dict(dw=0), 1, "dw is NULL"), (dict(workspace=0), 1, "workspace is NULL"),
    (dict(rstd=0), 1, "rstd"), (dict(dh=FAKE + 2), 1, "dh must be"), (dict(K=1 << 20), 2, "16384")])
def test_norm_gradient_refusals(L, change, status, word):
    a = dict(T=16, K=64, dy=FAKE, h=FAKE, w=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE)
    a.update(change)
    rc = L.forge_rmsnorm_bwd(ctypes.byref(api.ForgeRmsnormGrad(**a)), None)
    assert rc == status and word in _message(L), (rc, _message(L))


def test_null_structs(L):
    assert L.forge_rmsnorm_fwd(None, None) == 1 and L.forge_rmsnorm_bwd(None, None) == 1
    hp = api.hparams()
    assert L.forge_multi_opt_step(None, 3, 0, 0, 0, 0, ctypes.byref(hp), 1, 0, None) == 1


def test_the_binding_refuses_what_the_library_could_not_see():
    f = lambda n, d=torch.float32: torch.zeros(n, dtype=d)  # noqa: E731
    with pytest.raises(TypeError, match="one dtype"):
        api.make_tensors([f(4), f(4, torch.bfloat16)], [f(4), f(4)])
    with pytest.raises(ValueError, match="expected 2 tensors"):
        api.make_tensors([f(4), f(4)], [f(4)])
    with pytest.raises(TypeError, match="kept alike"):
        api.make_tensors([f(4)], [f(4)], [f(4)], [f(4, torch.uint8)])
    with pytest.raises(TypeError, match="kept alike"):
        api.make_tensors([f(4)], [f(4)], [f(4)], [f(4, torch.bfloat16)])
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.make_tensors([f(4)], [f(4)])
    with pytest.raises(ValueError, match="contiguous"):
        api.make_tensors([f((4, 4)).t()], [f(16)])
    with pytest.raises(ValueError, match="block"):
        api.make_tensors([f(4)], [f(4)], [f(4, torch.int8)], [f(4, torch.uint8)], block=48)
    x = torch.zeros((2, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.forge_rmsnorm_fwd(x, x[0], 1e-6, y=x)
    with pytest.raises(TypeError, match="expected torch.bfloat16"):
        api.forge_rmsnorm_fwd(x.float(), x[0], 1e-6, y=x)
    with pytest.raises(ValueError, match=r"\[T, K\]"):
        api.forge_rmsnorm_fwd(x[0], x[0], 1e-6)
