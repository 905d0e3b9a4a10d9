"""Workloads of the operators around the fused linear step, each with a plain
form in elementary float32 torch operations.

Three families, as they meet in one training step of a block with experts:

* ``norm``    root-mean-square norm with the residual's addition, its output in
              bf16 or as E4M3 codes with scales, and its gradient;
* ``experts`` matrix products grouped by expert over ragged token groups: the
              forward product, the input gradient, and the backward step that
              updates every expert's weights in place;
* ``adamw``   an AdamW step over many tensors at once.

``own`` selects the framework's kernels; otherwise the plain form runs.  Layer
widths are those of the linears in ``optimizer_tcgen05_dw_gb300/inputs.py``
(hidden 4096 and 5120, key/value width 1024) or generic powers of two.
"""

import math

import numpy as np
import torch

own = False

HP = dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
STEP = 10
EPS = 1e-6
E4M3_MAX = 448.0
Y_SCALE = 2.0 ** -5  # per-tensor scale from earlier steps: largest |y| about 6, with head room


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token: the norm before a block, latency only
        dict(name="norm_decode", op="norm", dir="fwd", out="bf16", residual=True, T=1, K=4096),
        # the norm ahead of the E4M3 step: token-contiguous codes, one scale for the tensor
        dict(name="norm_fwd_e4m3_tensor", op="norm", dir="fwd", out="e4m3_tensor", residual=True, T=16384, K=4096),
        # an odd batch, codes with one scale a token, as a row-scaled product reads them
        dict(name="norm_fwd_e4m3_token", op="norm", dir="fwd", out="e4m3_token", residual=False, T=4099, K=5120),
        # its gradient in training, with the residual stream's
        dict(name="norm_bwd", op="norm", dir="bwd", out="bf16", residual=True, T=12289, K=5120),
        # a few decoded tokens, each sent to some of the experts: weights are read for a handful of rows
        dict(name="experts_decode", op="experts", dir="fwd", states="none", T=16, E=16, N=2048, K=4096, skew=0.7),
        # training: long groups, unevenly filled
        dict(name="experts_fwd", op="experts", dir="fwd", states="none", T=16384, E=16, N=4096, K=4096, skew=0.5),
        # many small experts, an odd number of tokens
        dict(name="experts_dgrad", op="experts", dir="dgrad", states="none", T=8191, E=64, N=1024, K=2048, skew=0.6),
        # the backward step of a small layer, moments in 32 bits
        dict(name="experts_step", op="experts", dir="step", states="fp32", T=4099, E=8, N=1024, K=4096, skew=0.5),
        # the backward step in training, moments in bf16
        dict(name="experts_step_bf16", op="experts", dir="step", states="bf16", T=16384, E=16, N=2048, K=4096, skew=0.5),
        # the norm weights of 40 layers and the last one: many short tensors, latency
        dict(name="adamw_norms", op="adamw", count=81, largest=5120, spread=0.0, w="fp32", g="fp32", states="fp32"),
        # embedding, biases and gates in bf16 with stochastic rounding, odd lengths
        dict(name="adamw_bf16", op="adamw", count=24, largest=131334145, spread=0.55, w="bf16", g="bf16", states="fp32"),
        # the same kind of set with moments in 8 bits
        dict(name="adamw_int8", op="adamw", count=40, largest=16777216, spread=0.25, w="bf16", g="fp32", states="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, unit, lo, hi):
    """A width that is a multiple of `unit`; 3072 is not drawn, as no configuration here has it."""
    n = unit * _log(rng, lo, hi)
    return n if n != 3072 else n + unit


def draw(rng):
    op = rng.choice(("norm", "norm", "experts", "experts", "adamw"))
    if op == "norm":
        back = rng.random() < 0.4
        out = "bf16" if back else rng.choice(("bf16", "e4m3_token", "e4m3_tensor"))
        T = _log(rng, 1, 16384)
        if out == "e4m3_tensor":
            T = max(16, T // 16 * 16)  # 16-byte rows of codes
        K = _width(rng, 8, 16, 640)
        return dict(op=op, dir="bwd" if back else "fwd", out=out, residual=rng.random() < 0.6, T=T, K=K)
    if op == "experts":
        way = rng.choice(("fwd", "dgrad", "step"))
        E = _log(rng, 1, 64)
        N = _width(rng, 8, 16, 512) if rng.random() < 0.5 else _width(rng, 64, 2, 64)
        K = _width(rng, 8, 16, 512) if rng.random() < 0.5 else _width(rng, 64, 2, 64)
        while E * N * K > 16 * 4096 * 4096:
            E = max(1, E // 2)
        return dict(op=op, dir=way, states=rng.choice(("fp32", "bf16")) if way == "step" else "none",
                    T=_log(rng, 1, 16384), E=E, N=N, K=K, skew=round(rng.uniform(0.0, 1.2), 2))
    case = dict(op=op, count=_log(rng, 1, 400), largest=_log(rng, 64, 16777216), spread=round(rng.uniform(0.0, 0.6), 2),
                w=rng.choice(("fp32", "bf16")), g=rng.choice(("fp32", "bf16")), states=rng.choice(("fp32", "bf16", "int8")))
    while sum(_sizes(case)) > 1.2e8:
        case["count"] //= 2
    return case


def _counts(T, E, skew):
    """Tokens of each expert, most first: shares 1 / (i + 1)^skew, whole numbers that add up to T."""
    share = [(i + 1.0) ** -skew for i in range(E)]
    edges, run = [0], 0.0
    for s in share:
        run += s
        edges.append(int(round(T * run / sum(share))))
    return [b - a for a, b in zip(edges, edges[1:])]


def _sizes(case):
    """Lengths of the tensors: equal (spread 0), or each a fixed share shorter than the one before, odd ones among them."""
    n, got = float(case["largest"]), []
    for i in range(case["count"]):
        got.append(max(1, int(n) - (i % 3 if case["spread"] else 0)))
        n = max(1.0, n * (1.0 - case["spread"]))
    return got


def work(case):
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        if case["dir"] == "bwd":  # dy, h (and the residual's gradient) in, dx out; the weight and its gradient
            return dict(bytes=T * K * (6 + 2 * case["residual"]) + 4 * T + 6 * K, flops=11 * T * K)
        per = 2 + 4 * case["residual"] + (2 if case["out"] == "bf16" else 1)  # x, residual and the sum, the output
        return dict(bytes=T * K * per + 4 * T * (2 if case["out"] == "e4m3_token" else 1) + 2 * K, flops=6 * T * K)
    if case["op"] == "experts":
        T, E, N, K = (case[k] for k in ("T", "E", "N", "K"))
        live = sum(c > 0 for c in _counts(T, E, case["skew"]))
        if case["dir"] != "step":
            return dict(bytes=2 * T * (N + K) + 2 * live * N * K, flops=2 * T * N * K)
        return dict(bytes=2 * T * (N + 2 * K) + E * N * K * (4 + (16 if case["states"] == "fp32" else 8)),
                    flops=4 * T * N * K + 16 * E * N * K)
    n = sum(_sizes(case))
    per = (8 if case["w"] == "fp32" else 4) + (4 if case["g"] == "fp32" else 2) + dict(fp32=16, bf16=8, int8=4.25)[case["states"]]
    if case["states"] == "int8":
        per += 2.125 + 8  # the moments read back as the values they stand for
    return dict(bytes=n * per, flops=16 * n)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 13)

    def normal(shape, std, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    return dict(norm=_prepare_norm, experts=_prepare_experts, adamw=_prepare_adamw)[case["op"]](case, seed, gen, normal)


def _prepare_norm(case, seed, gen, normal):
    T, K = case["T"], case["K"]
    st = dict(case=case, w=1.0 + normal((K,), 0.1, torch.float32))
    st["w"] = st["w"].to(torch.bfloat16)
    if case["dir"] == "bwd":
        st["h"] = normal((T, K), 1.5)
        st["dy"] = normal((T, K), 1e-3)
        st["dh"] = normal((T, K), 1e-3) if case["residual"] else None
        hf = st["h"].float()
        st["rstd"] = torch.rsqrt((hf * hf).mean(1) + EPS)
        st["dx"] = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
        st["dw"] = torch.empty(K, device="cuda")
    else:
        st["x"] = normal((T, K), 1.0)
        st["res"] = normal((T, K), 1.5) if case["residual"] else None
        st["h"] = torch.empty((T, K), dtype=torch.bfloat16, device="cuda") if case["residual"] else None
        st["rstd"] = torch.empty(T, device="cuda")
        if case["out"] == "bf16":
            st["y"] = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
        elif case["out"] == "e4m3_token":
            st["q"] = torch.empty((T, K), dtype=torch.float8_e4m3fn, device="cuda")
            st["scale"] = torch.empty(T, device="cuda")
        else:
            st["qt"] = torch.empty((K, T), dtype=torch.float8_e4m3fn, device="cuda")
            st["amax"] = torch.empty(1, device="cuda")
    if own and case["dir"] == "bwd":
        from optimizer_tcgen05_dw_gb300 import api
        st["work"] = torch.empty(api.forge_rmsnorm_bwd_workspace(T, K), device="cuda")
    return st


def _prepare_experts(case, seed, gen, normal):
    T, E, N, K = (case[k] for k in ("T", "E", "N", "K"))
    counts = np.random.RandomState(int(seed) % (2 ** 31)).permutation(_counts(T, E, case["skew"]))
    st = dict(case=case, counts=[int(c) for c in counts], most=max(1, int(counts.max())), seed=int(seed))
    st["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    st["W"] = normal((E, N, K), 0.02)
    if case["dir"] != "dgrad":
        st["X"] = normal((T, K), 1.0)
    if case["dir"] == "fwd":
        st["Y"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    else:
        st["dY"] = normal((T, N), 1e-3)
        st["dX"] = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    if case["dir"] == "step":
        # moments of the size that steady gradients leave: their spread is 1e-3 times the root of a group's length
        dt, size = torch.float32 if case["states"] == "fp32" else torch.bfloat16, 1e-3 * math.sqrt(max(1.0, T / E))
        st["m"] = normal((E, N, K), 0.25 * size, dt)
        st["v"] = normal((E, N, K), size, torch.float32).square().to(dt)
    return st


def _prepare_adamw(case, seed, gen, normal):
    """The tensors lie in flat buffers, each from a multiple of 64 elements on, as a program that keeps them together has them."""
    sizes = _sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + (n + 63) // 64 * 64)
    total = starts[-1]
    pad = torch.ones(total, dtype=torch.bool, device="cuda")
    for s, n in zip(starts, sizes):
        pad[s:s + n] = False

    def flat(std, dtype):
        t = normal((total,), std, dtype)
        t[pad] = 0
        return t

    wt, gt = (torch.float32 if case[k] == "fp32" else torch.bfloat16 for k in ("w", "g"))
    st = dict(case=case, seed=int(seed), starts=torch.tensor(starts, device="cuda"), w=flat(0.02, wt), g=flat(1e-3, gt))
    m, v = flat(1e-3, torch.float32), flat(1e-3, torch.float32).square_()
    if case["states"] == "int8":
        st["ma"], st["va"] = m.view(-1, 64).abs().amax(1), v.view(-1, 64).amax(1)
        st["m"] = _encode(m, st["ma"], True)
        st["v"] = _encode(v, st["va"], False)
        st["m32"], st["v32"] = m, v  # where the moments are read back to
    else:
        dt = torch.float32 if case["states"] == "fp32" else torch.bfloat16
        st["m"], st["v"] = m.to(dt), v.to(dt)
    if own:
        from optimizer_tcgen05_dw_gb300 import api
        cut = lambda t: [t[s:s + n] for s, n in zip(starts, sizes)]  # noqa: E731
        scales = lambda t: [t[s // 64:(s + n + 63) // 64] for s, n in zip(starts, sizes)]  # noqa: E731
        more = dict(s1_scale=scales(st["ma"]), s2_scale=scales(st["va"])) if case["states"] == "int8" else {}
        st["tensors"] = api.make_tensors(cut(st["w"]), cut(st["g"]), cut(st["m"]), cut(st["v"]), **more)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if own:
        return dict(norm=_own_norm, experts=_own_experts, adamw=_own_adamw)[case["op"]](st)
    return dict(norm=_plain_norm, experts=_plain_experts, adamw=_plain_adamw)[case["op"]](st)


def _own_norm(st):
    from optimizer_tcgen05_dw_gb300 import api
    case = st["case"]
    if case["dir"] == "bwd":
        api.forge_rmsnorm_bwd(st["dy"], st["h"], st["w"], st["rstd"], st["dx"], st["dw"], st["work"], dh=st["dh"])
        return dict(dx=st["dx"], dw=st["dw"])
    out = dict(h=st["h"], rstd=st["rstd"])
    if case["out"] == "bf16":
        api.forge_rmsnorm_fwd(st["x"], st["w"], EPS, residual=st["res"], h=st["h"], rstd=st["rstd"], y=st["y"])
        return dict(out, y=st["y"])
    if case["out"] == "e4m3_token":
        api.forge_rmsnorm_fwd(st["x"], st["w"], EPS, residual=st["res"], h=st["h"], rstd=st["rstd"],
                              yq=st["q"], yq_scale=st["scale"])
        return dict(out, q=st["q"], scale=st["scale"])
    api.forge_rmsnorm_fwd(st["x"], st["w"], EPS, residual=st["res"], h=st["h"], rstd=st["rstd"],
                          yt=st["qt"], yt_scale=Y_SCALE, amax=st["amax"])
    return dict(out, qt=st["qt"], amax=st["amax"])


def _own_experts(st):
    from optimizer_tcgen05_dw_gb300 import api
    case = st["case"]
    if case["dir"] == "fwd":
        api.forge_grouped_linear(st["X"], st["W"], st["offsets"], st["Y"])
        return dict(Y=st["Y"])
    if case["dir"] == "dgrad":
        api.forge_grouped_dgrad(st["dY"], st["W"], st["offsets"], st["dX"])
        return dict(dX=st["dX"])
    api.forge_grouped_bwd_step(st["X"], st["dY"], st["W"], st["offsets"], "adamw", HP, STEP, st["seed"], st["m"], st["v"],
                               dX=st["dX"])
    return dict(W=st["W"], m=st["m"], v=st["v"], dX=st["dX"])


def _own_adamw(st):
    from optimizer_tcgen05_dw_gb300 import api
    api.forge_multi_opt_step(st["tensors"], "adamw", HP, STEP, st["seed"])
    if st["case"]["states"] != "int8":
        return dict(w=st["w"], m=st["m"], v=st["v"])
    for code, scale, to, signed in ((st["m"], st["ma"], st["m32"], True), (st["v"], st["va"], st["v32"], False)):
        api.forge_dequantize_state(code.view(-1, 64), scale.view(-1, 1), to.view(-1, 64), signed)
    return dict(w=st["w"], m=st["m32"], v=st["v32"])


# ---------------------------------------------------------------- plain forms

def _plain_norm(st):
    case = st["case"]
    w = st["w"].float()
    if case["dir"] == "bwd":
        h, r = st["h"].float(), st["rstd"][:, None]
        dy = st["dy"].float()
        n, g = h * r, dy * w
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return dict(dx=dx.to(torch.bfloat16), dw=(dy * n).sum(0))
    h = st["x"].float()
    if st["res"] is not None:  # the stream keeps bf16, and the norm reads what it keeps
        h = (h + st["res"].float()).to(torch.bfloat16)
    out = dict(h=h if st["res"] is not None else None)
    h = h.float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * w
    out["rstd"] = rstd
    if case["out"] == "bf16":
        return dict(out, y=y.to(torch.bfloat16))
    if case["out"] == "e4m3_token":
        scale = y.abs().amax(1) / E4M3_MAX
        q = y / torch.where(scale > 0, scale, 1.0)[:, None]
        return dict(out, q=q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale=scale)
    q = (y / Y_SCALE).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(out, qt=q.t().contiguous(), amax=y.abs().amax().reshape(1))


def _plain_experts(st):
    """Every expert's tokens padded to the longest group, and one product over all experts."""
    case = st["case"]
    T, E = case["T"], case["E"]
    row = torch.arange(T, device="cuda")
    offsets = st["offsets"].long()
    expert = torch.bucketize(row, offsets[1:], right=True)
    place = expert * st["most"] + row - offsets[expert]

    def spread(t):
        to = torch.zeros((E * st["most"], t.shape[1]), device="cuda")
        to[place] = t.float()
        return to.view(E, st["most"], -1)

    def gather(t):
        return t.reshape(E * st["most"], -1)[place].to(torch.bfloat16)

    W = st["W"].float()
    if case["dir"] == "fwd":
        return dict(Y=gather(spread(st["X"]) @ W.transpose(1, 2)))
    dY = spread(st["dY"])
    dX = gather(dY @ W)
    if case["dir"] == "dgrad":
        return dict(dX=dX)
    g = dY.transpose(1, 2) @ spread(st["X"])
    w, m, v = _plain_rule(W, g, st["m"].float(), st["v"].float())
    group = torch.arange(w.numel() // 8, device="cuda")
    st["W"].copy_(_round_sr(w, group, st["seed"] + torch.zeros_like(group)))
    st["m"].copy_(m)
    st["v"].copy_(v)
    return dict(W=st["W"], m=st["m"], v=st["v"], dX=dX)


def _plain_adamw(st):
    case = st["case"]
    int8 = case["states"] == "int8"
    m, v = (_decode(st["m"], st["ma"], 127.0), _decode(st["v"], st["va"], 255.0)) if int8 else (st["m"].float(), st["v"].float())
    w, m, v = _plain_rule(st["w"].float(), st["g"].float(), m, v)
    if case["w"] == "bf16":
        group = torch.arange(w.numel() // 8, device="cuda")
        starts = st["starts"] // 8
        tensor = torch.bucketize(group, starts[1:], right=True)
        w = _round_sr(w, group - starts[tensor], st["seed"] + tensor)
    st["w"].copy_(w)
    if not int8:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return dict(w=st["w"], m=st["m"], v=st["v"])
    st["ma"].copy_(m.view(-1, 64).abs().amax(1))
    st["va"].copy_(v.view(-1, 64).amax(1))
    st["m"].copy_(_encode(m, st["ma"], True))
    st["v"].copy_(_encode(v, st["va"], False))
    return dict(w=st["w"], m=_decode(st["m"], st["ma"], 127.0), v=_decode(st["v"], st["va"], 255.0))


def _f32(x):
    return float(np.float32(x))


def _scalars():
    """AdamW's scalars of this step, formed in 64 bits and rounded once."""
    lr, b1, b2, eps, wd = (_f32(HP[k]) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    c1, c2 = 1.0 - b1 ** STEP, 1.0 - b2 ** STEP
    return [_f32(x) for x in (b1, 1.0 - b1, b2, 1.0 - b2, 1.0 / math.sqrt(c2), eps, 1.0 - lr * wd, lr / c1)]


def _plain_rule(w, g, m, v):
    b1, ob1, b2, ob2, inv_c2, eps, decay, size = _scalars()
    m = m * b1 + g * ob1
    v = v * b2 + (g * g) * ob2
    return w * decay - (m / (torch.sqrt(v) * inv_c2 + eps)) * size, m, v


def _round_sr(w, group, key):
    """float32 to bf16 by adding 16 random bits below the kept ones: Philox4x32-10 words of (group of 8 elements, step), keyed by the seed."""
    low = 0xFFFFFFFF
    c = [group & low, group >> 32, torch.full_like(group, STEP), torch.zeros_like(group)]
    k0, k1 = key & low, (key >> 32) & low
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & low) ^ c[1] ^ k0, p1 & low, ((p0 >> 32) & low) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).view(w.shape).to(torch.int32)
    pattern = w.view(torch.int32)
    up = (pattern + bits) & -65536
    return torch.where(torch.isfinite(w), up, pattern).view(torch.float32).to(torch.bfloat16)


def _encode(x, absmax, signed):
    """8-bit codes of blocks of 64: x over the block's step, to the nearest (ties to even)."""
    top = 127.0 if signed else 255.0
    step = absmax / torch.full_like(absmax, top)
    q = torch.round(x.view(-1, 64) / torch.where(step > 0, step, 1.0)[:, None])
    return q.clamp(-top if signed else 0.0, top).view(-1).to(torch.int8 if signed else torch.uint8)


def _decode(code, absmax, top):
    return (code.view(-1, 64).float() * (absmax / torch.full_like(absmax, top))[:, None]).view(-1)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st, case)
    if case["op"] == "experts":
        return _exact_experts(st, case)
    f = lambda t: t.double()  # noqa: E731
    int8 = case["states"] == "int8"
    m = f(st["m"]).view(-1, 64) * f(st["ma"])[:, None] / 127 if int8 else f(st["m"])
    v = f(st["v"]).view(-1, 64) * f(st["va"])[:, None] / 255 if int8 else f(st["v"])
    w, m, v = _exact_rule(f(st["w"]), f(st["g"]), m.reshape(-1), v.reshape(-1))
    return dict(w=w, m=None if int8 else m, v=None if int8 else v)


def _exact_rule(w, g, m, v):
    m = HP["beta1"] * m + (1 - HP["beta1"]) * g
    v = HP["beta2"] * v + (1 - HP["beta2"]) * g ** 2
    mh, vh = m / (1 - HP["beta1"] ** STEP), v / (1 - HP["beta2"] ** STEP)
    return w - HP["lr"] * HP["weight_decay"] * w - HP["lr"] * mh / (vh.sqrt() + HP["eps"]), m, v


def _exact_norm(st, case):
    w = st["w"].double()
    if case["dir"] == "bwd":
        h, dy, r = st["h"].double(), st["dy"].double(), st["rstd"].double()
        dot = torch.einsum("tk,k,tk->t", dy, w, h)
        dx = r[:, None] * dy * w - h * (r ** 3 * dot / case["K"])[:, None]
        if st["dh"] is not None:
            dx += st["dh"].double()
        return dict(dx=dx, dw=torch.einsum("tk,tk,t->k", dy, h, r))
    h = st["x"].double()
    if st["res"] is not None:
        h = (h + st["res"].double()).to(torch.bfloat16).double()
    r = (h.square().sum(1) / case["K"] + EPS) ** -0.5
    y = torch.einsum("tk,t,k->tk", h, r, w)
    out = dict(h=h if st["res"] is not None else None, rstd=r)
    if case["out"] == "bf16":
        return dict(out, y=y)
    if case["out"] == "e4m3_token":
        scale = y.abs().amax(1) / 448
        return dict(out, q=y / scale[:, None], scale=scale)
    return dict(out, qt=(y / Y_SCALE).t(), amax=y.abs().max().reshape(1))


def _exact_experts(st, case):
    T, E, N, K = (case[k] for k in ("T", "E", "N", "K"))
    if T * N * K > 3e11:
        return None
    out = {}
    to = 0
    rows = []
    for e in range(E):
        rows.append(slice(to, to + st["counts"][e]))
        to += st["counts"][e]
    if case["dir"] == "fwd":
        return dict(Y=torch.cat([st["X"][r].double() @ st["W"][e].double().t() for e, r in enumerate(rows)]))
    out["dX"] = torch.cat([st["dY"][r].double() @ st["W"][e].double() for e, r in enumerate(rows)])
    if case["dir"] == "dgrad":
        return out
    new = [_exact_rule(st["W"][e].double(), st["dY"][r].double().t() @ st["X"][r].double(), st["m"][e].double(),
                       st["v"][e].double()) for e, r in enumerate(rows)]
    for i, name in enumerate(("W", "m", "v")):
        out[name] = torch.stack([n[i] for n in new])
    return out
