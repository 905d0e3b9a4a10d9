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


def _grouped(**kw):
    a = dict(T=40, N=64, K=128, groups=4, offsets=FAKE, X=FAKE, dY=FAKE, Y=FAKE, dX=FAKE)
    a.update(kw)
    return ctypes.byref(api.ForgeGrouped(**a))


@pytest.mark.parametrize("change,status,word", [
    (dict(T=-1), 1, "negative"), (dict(groups=-1), 1, "negative"), (dict(N=12), 1, "multiples of 8"),
    (dict(K=100), 1, "multiples of 8"), (dict(groups=1025), 2, "1024 groups"), (dict(offsets=0), 1, "offsets"),
    (dict(offsets=FAKE + 2), 1, "offsets"), (dict(T=1 << 31), 2, "31 bits"), (dict(N=1 << 24, groups=200), 2, "31 bits")])
def test_grouped_refusals(L, change, status, word):
    st = api.ForgeState(FAKE, api.W_BF16_SR, api.STATE_FP32, FAKE, FAKE, None, None)
    hp = api.hparams()
    for call in (lambda g: L.forge_grouped_linear(g, FAKE, None), lambda g: L.forge_grouped_dgrad(g, FAKE, None),
                 lambda g: L.forge_grouped_bwd_step(g, ctypes.byref(st), 0, ctypes.byref(hp), 1, 0, None)):
        rc = call(_grouped(**change))
        assert rc == status and word in _message(L), (rc, _message(L))


@pytest.mark.parametrize("state,kind,step,change,status,word", [
    (dict(w_dtype=0), 0, 1, {}, 2, "bf16 weights"), (dict(s1=0), 0, 1, {}, 1, "needs s1"),
    (dict(s_dtype=1), 0, 1, {}, 1, "scale"), (dict(s_dtype=1), 0, 1, dict(K=72), 1, "K % 64"),
    (dict(), 9, 1, {}, 1, "opt_kind"), (dict(), 0, 0, {}, 1, "step"), (dict(), 0, 1, dict(X=0), 1, "X is NULL"),
    (dict(), 0, 1, dict(dY=FAKE + 8), 1, "dY must"), (dict(), 0, 1, dict(dX=FAKE + 8), 1, "dX must"),
    (dict(W=0), 0, 1, {}, 1, "W must")])
def test_grouped_step_refusals(L, state, kind, step, change, status, word):
    a = dict(W=FAKE, w_dtype=1, s_dtype=0, s1=FAKE, s2=FAKE, s1_scale=None, s2_scale=None)
    a.update(state)
    st, hp = api.ForgeState(**a), api.hparams()
    rc = L.forge_grouped_bwd_step(_grouped(**change), ctypes.byref(st), kind, ctypes.byref(hp), step, 0, None)
    assert rc == status and word in _message(L), (rc, _message(L))


def test_grouped_nothing_to_do_needs_no_device(L):
    assert L.forge_grouped_linear(_grouped(T=0), FAKE, None) == 0
    assert L.forge_grouped_linear(_grouped(N=0), FAKE, None) == 0
    assert L.forge_grouped_dgrad(_grouped(T=0), FAKE, None) == 0
    st, hp = api.ForgeState(FAKE, api.W_BF16_SR, api.STATE_FP32, FAKE, FAKE, None, None), api.hparams()
    assert L.forge_grouped_bwd_step(_grouped(groups=0, dX=None), ctypes.byref(st), 0, ctypes.byref(hp), 1, 0, None) == 0


def test_null_structs(L):
    assert L.forge_grouped_linear(None, None, None) == 1 and L.forge_grouped_dgrad(None, None, None) == 1
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
    b = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match=r"\[groups, N, K\]"):
        api.forge_grouped_linear(b(4, 8), b(8, 8), torch.zeros(2, dtype=torch.int32), b(4, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.forge_grouped_linear(b(4, 8), b(2, 8, 8), torch.zeros(3, dtype=torch.int32), b(4, 8))
    x = torch.zeros((2, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.forge_rmsnorm_fwd(x, x[0], 1e-6, y=x)
    with pytest.raises(TypeError, match="expected torch.bfloat16"):
        api.forge_rmsnorm_fwd(x.float(), x[0], 1e-6, y=x)
    with pytest.raises(ValueError, match=r"\[T, K\]"):
        api.forge_rmsnorm_fwd(x[0], x[0], 1e-6)
