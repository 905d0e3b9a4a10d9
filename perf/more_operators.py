"""Workloads of a gated feed-forward block trained with activations in 8 bits,
each with a plain form in elementary float32 torch operations.

Three families, as they meet in one training step of such a block:

* ``gated``    both projections of a token, the activation of the gate and the
               product with the other, and their gradient through the down
               projection, with what the gradient needs kept in bf16 or 8 bits;
* ``codes``    activations (a scale for each 128 elements of a row) and weights
               (a scale for each 128 x 128) to E4M3 codes, and back;
* ``product``  the matrix product of two such tensors.

``own`` selects the framework's kernels; otherwise the plain form runs.  Widths
are those of the linears in ``optimizer_tcgen05_dw_gb300/inputs.py`` (hidden
4096 and 5120, feed-forward 14336 and 17408) or generic.
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
LEAST = 2.0 ** -126  # the smallest scale of a block that is not zero
B16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token through the projections: both weights are read for one row
        dict(name="gated_decode", op="gated", dir="fwd", act="silu", keep="none", T=1, K=4096, F=14336),
        # a small batch of decoded tokens
        dict(name="gated_decode_batch", op="gated", dir="fwd", act="silu", keep="none", T=24, K=5120, F=17408),
        # training, the projections kept in bf16 for the gradient
        dict(name="gated_fwd", op="gated", dir="fwd", act="silu", keep="bf16", T=16384, K=4096, F=14336),
        # training on an odd number of tokens, the projections kept in 8 bits
        dict(name="gated_fwd_kept8", op="gated", dir="fwd", act="gelu_tanh", keep="e4m3", T=4099, K=5120, F=17408),
        # its gradient, from the projections in bf16
        dict(name="gated_bwd", op="gated", dir="bwd", act="silu", keep="bf16", T=16384, K=4096, F=14336),
        # and from 8 bits
        dict(name="gated_bwd_kept8", op="gated", dir="bwd", act="gelu_tanh", keep="e4m3", T=4099, K=5120, F=17408),
        # the activations of one decoded token, ahead of a product in 8 bits: latency only
        dict(name="codes_decode", op="codes", dir="to", rows=1, x="bf16", T=1, K=4096),
        # the widest activation of a layer into its checkpoint
        dict(name="codes_write", op="codes", dir="to", rows=1, x="bf16", T=16384, K=14336),
        # and out of it, in the backward pass: an odd number of tokens
        dict(name="codes_read", op="codes", dir="from", rows=1, x="bf16", T=12289, K=5120),
        # a few tokens in serving: the weights' codes are read once
        dict(name="product_decode", op="product", T=5, N=4096, K=14336),
        # an odd batch
        dict(name="product_odd", op="product", T=1531, N=5120, K=17408),
        # training
        dict(name="product_fwd", op="product", T=16384, N=14336, K=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = 16384 * 4096 * 14336  # T K F of the largest listed case


def draw(rng):
    op = rng.choice(("gated", "gated", "codes", "product"))
    if op == "codes":
        rows = rng.choice((1, 1, 128))
        case = dict(op=op, dir=rng.choice(("to", "from")), rows=rows, x=rng.choice(("bf16", "bf16", "fp32")),
                    T=_log(rng, 1, 16384), K=8 * _log(rng, 8, 2176))
        while case["T"] * case["K"] > 16384 * 14336 // 2:
            case["T"] = max(1, case["T"] // 2)
        return case
    T = _log(rng, 1, 16384)
    if op == "product":
        case = dict(op=op, T=T, N=8 * _log(rng, 8, 2176), K=16 * _log(rng, 8, 1088))
        while case["T"] * case["N"] * case["K"] > MOST:
            case["T"] //= 2
        return case
    back = rng.random() < 0.5
    case = dict(op=op, dir="bwd" if back else "fwd", act=rng.choice(("silu", "gelu_tanh")),
                keep=rng.choice(("bf16", "e4m3") if back else ("none", "bf16", "e4m3")),
                T=T, K=8 * _log(rng, 16, 640), F=8 * _log(rng, 16, 2176))
    while case["T"] * case["K"] * case["F"] > MOST:
        case["T"] //= 2
    return case


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    if case["op"] == "codes":
        T, K = case["T"], case["K"]
        scales = _blocks(K) * (T if case["rows"] == 1 else _blocks(T))
        return dict(bytes=T * K * (1 + (4 if case["x"] == "fp32" else 2)) + 4 * scales, flops=2 * T * K)
    if case["op"] == "product":
        T, N, K = case["T"], case["N"], case["K"]
        return dict(bytes=T * K + N * K + 4 * _blocks(K) * (T + _blocks(N)) + 2 * T * N, flops=2 * T * N * K)
    T, K, F = case["T"], case["K"], case["F"]
    kept = dict(none=0, bf16=4 * T * F, e4m3=2 * T * F + 8 * T * _blocks(F))[case["keep"]]
    if case["dir"] == "fwd":  # x and both weights in, the block's hidden activation and what is kept out
        return dict(bytes=2 * T * K + 4 * F * K + 2 * T * F + kept, flops=4 * T * K * F + 8 * T * F)
    # the gradient and the down projection's weight in, with what was kept; both projections' gradients
    # and the hidden activation (for the down projection's own gradient) out
    return dict(bytes=2 * T * K + 2 * F * K + kept + 6 * T * F, flops=2 * T * K * F + 16 * T * F)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 6271 + 29)

    def normal(shape, std, dtype=B16):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    return dict(gated=_prepare_gated, codes=_prepare_codes, product=_prepare_product)[case["op"]](case, normal)


def _activations(T, K, normal, dtype=B16):
    """Tokens whose columns differ in size, as activations' do, the last few of a batch padding."""
    x = normal((T, K), 1.0, torch.float32) * torch.exp(normal((K,), 0.5, torch.float32))
    if T >= 64:
        x[T - T // 64:] = 0
    return x.to(dtype)


def _prepare_gated(case, normal):
    T, K, F = case["T"], case["K"], case["F"]
    st = dict(case=case)
    empty = lambda *s, dtype=B16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    if case["dir"] == "fwd":
        st["X"], st["W"] = normal((T, K), 1.0), normal((2 * F, K), 0.02)
        st["Y"] = empty(T, F)
        if case["keep"] == "bf16":
            st["gu"] = empty(T, 2 * F)
        elif case["keep"] == "e4m3":
            st["codes"], st["scale"] = empty(T, 2 * F, dtype=E4M3), empty(T, 2, _blocks(F), dtype=torch.float32)
        return st
    st["dY"], st["Wd"] = normal((T, K), 1e-3), normal((K, F), 0.02)
    st["dGU"], st["Y"] = empty(T, 2 * F), empty(T, F)
    gu = normal((T, 2 * F), 1.3)
    if case["keep"] == "bf16":
        st["gu"] = gu
    else:
        codes, scale = _encode(gu.view(2 * T, F), 1)
        st["codes"], st["scale"] = codes.view(T, 2 * F), scale.view(T, 2, _blocks(F))
    return st


def _prepare_codes(case, normal):
    T, K = case["T"], case["K"]
    xt = torch.float32 if case["x"] == "fp32" else B16
    x = _activations(T, K, normal, xt) if case["rows"] == 1 else normal((T, K), 0.02, xt)
    st = dict(case=case)
    if case["dir"] == "to":
        rows = T if case["rows"] == 1 else _blocks(T)
        return dict(st, x=x, codes=torch.empty((T, K), dtype=E4M3, device="cuda"),
                    scale=torch.empty((rows, _blocks(K)), device="cuda"))
    st["codes"], st["scale"] = _encode(x, case["rows"])
    return dict(st, x=torch.empty((T, K), dtype=xt, device="cuda"))


def _prepare_product(case, normal):
    T, N, K = case["T"], case["N"], case["K"]
    st = dict(case=case, Y=torch.empty((T, N), dtype=B16, device="cuda"))
    st["xq"], st["xs"] = _encode(_activations(T, K, normal), 1)
    st["wq"], st["ws"] = _encode(normal((N, K), 0.02), BLOCK)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        return dict(gated=_own_gated, codes=_own_codes, product=_own_product)[st["case"]["op"]](st)
    return dict(gated=_plain_gated, codes=_plain_codes, product=_plain_product)[st["case"]["op"]](st)


def _own_gated(st):
    from optimizer_tcgen05_dw_gb300 import api
    case = st["case"]
    kept = dict(gu=st.get("gu"), gu_codes=st.get("codes"), gu_scale=st.get("scale"))
    if case["dir"] == "fwd":
        api.forge_gated_linear(st["X"], st["W"], st["Y"], act=case["act"], **kept)
        return dict(Y=st["Y"], **kept)
    api.forge_gated_dgrad(st["dY"], st["Wd"], st["dGU"], act=case["act"], Y=st["Y"], **kept)
    return dict(dGU=st["dGU"], Y=st["Y"])


def _own_codes(st):
    from optimizer_tcgen05_dw_gb300 import api
    case = st["case"]
    if case["dir"] == "to":
        api.forge_quantize_e4m3(st["x"], st["codes"], st["scale"], block_rows=case["rows"])
        return dict(codes=st["codes"], scale=st["scale"])
    api.forge_dequantize_e4m3(st["codes"], st["scale"], st["x"], block_rows=case["rows"])
    return dict(x=st["x"])


def _own_product(st):
    from optimizer_tcgen05_dw_gb300 import api
    api.forge_linear_e4m3(st["xq"], st["xs"], st["wq"], st["ws"], st["Y"])
    return dict(Y=st["Y"])


# ---------------------------------------------------------------- plain forms

def _spread(scale, shape, rows):
    """A scale for each element, from one for each block of `rows` x 128."""
    T, K = shape
    s = scale.repeat_interleave(BLOCK, 1)[:, :K]
    return s if rows == 1 else s.repeat_interleave(rows, 0)[:T]


def _encode(x, rows):
    """E4M3 codes of blocks of `rows` x 128 and their scales: the largest magnitude of a block becomes 448."""
    T, K = x.shape
    x = x.float()
    R = T if rows == 1 else _blocks(T) * rows
    pad = torch.zeros((R, _blocks(K) * BLOCK), device=x.device)
    pad[:T, :K] = x.abs()
    most = pad.view(R // rows, rows, -1, BLOCK).amax((1, 3))
    scale = torch.where(most > 0, (most / E4M3_MAX).clamp(min=LEAST), most)
    q = x / _spread(torch.where(scale > 0, scale, 1.0), x.shape, rows)
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def _decode(codes, scale, rows):
    return codes.float() * _spread(scale, codes.shape, rows)


def _act(kind, g):
    """The activation of the gate and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c, k = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(c * (g + k * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * k * g * g)


def _plain_gated(st):
    case = st["case"]
    T, F = case["T"], case["F"]
    if case["dir"] == "fwd":
        gu = st["X"].float() @ st["W"].float().t()
        out = dict(Y=(_act(case["act"], gu[:, :F])[0] * gu[:, F:]).to(B16))
        if case["keep"] == "e4m3":
            codes, scale = _encode(gu.view(2 * T, F), 1)
            return dict(out, gu=None, gu_codes=codes.view(T, 2 * F), gu_scale=scale.view(T, 2, -1))
        return dict(out, gu=gu.to(B16) if case["keep"] == "bf16" else None, gu_codes=None, gu_scale=None)
    da = st["dY"].float() @ st["Wd"].float()
    if case["keep"] == "bf16":
        gu = st["gu"].float()
    else:
        gu = _decode(st["codes"].view(2 * T, F), st["scale"].view(2 * T, -1), 1).view(T, 2 * F)
    g, u = gu[:, :F], gu[:, F:]
    a, slope = _act(case["act"], g)
    return dict(dGU=torch.cat([da * u * slope, da * a], 1).to(B16), Y=(a * u).to(B16))


def _plain_codes(st):
    case = st["case"]
    if case["dir"] == "to":
        codes, scale = _encode(st["x"], case["rows"])
        return dict(codes=codes, scale=scale)
    return dict(x=_decode(st["codes"], st["scale"], case["rows"]).to(st["x"].dtype))


def _plain_product(st):
    x = _decode(st["xq"], st["xs"], 1)
    return dict(Y=(x @ _decode(st["wq"], st["ws"], BLOCK).t()).to(B16))


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return dict(gated=_exact_gated, codes=_exact_codes, product=_exact_product)[case["op"]](st, case)


def _values(codes, scale, rows):
    """What codes stand for: every column block times its scales."""
    v = codes.double()
    for b in range(_blocks(codes.shape[1])):
        s = scale[:, b].double()
        if rows > 1:
            s = s[torch.arange(codes.shape[0], device=s.device) // rows]
        v[:, b * BLOCK:(b + 1) * BLOCK] *= s[:, None]
    return v


def _exact_codes(st, case):
    if case["dir"] == "from":
        return dict(x=_values(st["codes"], st["scale"], case["rows"]))
    x, rows = st["x"].double(), case["rows"]
    cuts = [x[:, b * BLOCK:(b + 1) * BLOCK].abs().amax(1) for b in range(_blocks(case["K"]))]
    most = torch.stack(cuts, 1)
    if rows > 1:
        most = torch.stack([c.amax(0) for c in most.split(rows)])
    scale = most / 448
    whole = scale[torch.arange(case["T"], device=x.device) // rows]
    codes = torch.empty_like(x)
    for b in range(_blocks(case["K"])):
        cut = slice(b * BLOCK, (b + 1) * BLOCK)
        codes[:, cut] = x[:, cut] / whole[:, b:b + 1].clamp(min=1e-300)
    return dict(codes=codes, scale=scale)


def _exact_product(st, case):
    wt = _values(st["wq"], st["ws"], BLOCK).t()
    x = _values(st["xq"], st["xs"], 1)
    return dict(Y=torch.cat([c @ wt for c in x.split(2048)]))


def _slope(kind, g):
    if kind == "silu":
        return torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return torch.sigmoid(2 * inner) + g * 2 * torch.sigmoid(2 * inner) * torch.sigmoid(-2 * inner) \
        * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)


def _gate(kind, g):
    """g sigmoid(g), or g (1 + tanh z) / 2 = g sigmoid(2 z)."""
    if kind == "silu":
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def _exact_gated(st, case):
    T, F = case["T"], case["F"]
    if case["dir"] == "fwd":
        w = st["W"].double().t()
        gu = torch.cat([c.double() @ w for c in st["X"].split(2048)])
        out = dict(Y=_gate(case["act"], gu[:, :F]) * gu[:, F:], gu=None, gu_codes=None, gu_scale=None)
        if case["keep"] == "bf16":
            out["gu"] = gu
        if case["keep"] == "e4m3":
            got = _exact_codes(dict(x=gu.view(2 * T, F)), dict(dir="to", rows=1, T=2 * T, K=F))
            out["gu_codes"], out["gu_scale"] = got["codes"].view(T, 2 * F), got["scale"].view(T, 2, -1)
        return out
    w = st["Wd"].double()
    da = torch.cat([c.double() @ w for c in st["dY"].split(2048)])
    if case["keep"] == "bf16":
        gu = st["gu"].double()
    else:
        gu = _values(st["codes"].view(2 * T, F), st["scale"].view(2 * T, -1), 1).view(T, 2 * F)
    g, u = gu[:, :F], gu[:, F:]
    a = _gate(case["act"], g)
    return dict(dGU=torch.cat([da * u * _slope(case["act"], g), da * a], 1), Y=a * u)
