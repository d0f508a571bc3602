"""The 8-bit layer's operators as they are timed and compared: the W8A8 product, the whole W8A8 linear layer,
the channels-last group norm, and the norm that hands 8-bit codes to the layer.

Each case runs either in plain form (elementary torch operations in 32 bits) or through the package's kernels
(`own`).  Shapes: the transformer widths of bit_diffusion_model_amd/workloads.py (hidden 3072, 9216 = 3 x 3072,
12288 = 4 x 3072, 4096 image + 512 text tokens) and generic U-Net / autoencoder widths (channels 128 to 1280 in
32 groups, images of 8 x 8 to 512 x 512 positions).

Definitions (every product and quotient below is one rounding to 32 bits; what decides a code is a definition,
not an approximation, so both forms and the 64-bit one take the same decisions on the same inputs):
  quantize   v = x inv_s;  a = max(max_k |v|, 2^-96);  r = 127 / a;  s_x = a / 127;  q = round_half_even(v r)
  product    y = (sum_k qX qW) s_x[m] s_w[n] + bias[n], the sum over whole numbers, y rounded once
  norm       y = act((x - mean) / sqrt(var + eps) gamma + beta), mean and var of a group over all positions
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_FLOOR = 2.0 ** -96


def _r128(k):
    return (k + 127) // 128 * 128


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one conditioning vector through a projection: the product alone, nothing but latency and the weights' read
        {"name": "product, 1 token", "op": "product", "M": 1, "K": 3072, "N": 9216, "y": "bf16", "bias": True},
        # odd sizes in every direction: a ragged batch of tokens, widths that are no multiple of any tile
        {"name": "product, ragged", "op": "product", "M": 333, "K": 1000, "N": 1111, "y": "f32", "bias": True},
        # the second MLP layer over all tokens of an image: the largest product
        {"name": "product, MLP fc2", "op": "product", "M": 4608, "K": 12288, "N": 3072, "y": "bf16", "bias": False},
        # a batch of 4 conditioning vectors: the serving form of the layer
        {"name": "layer, 4 tokens", "op": "layer", "M": 4, "K": 3072, "N": 9216, "x": "bf16", "y": "bf16",
         "smooth": True, "bias": True, "pad": 0},
        # the text tokens' projection, read out of a wider buffer (row stride longer than the row)
        {"name": "layer, 512 text tokens", "op": "layer", "M": 512, "K": 3072, "N": 3072, "x": "bf16", "y": "bf16",
         "smooth": True, "bias": True, "pad": 3072},
        # the QKV projection of all tokens
        {"name": "layer, QKV", "op": "layer", "M": 4608, "K": 3072, "N": 9216, "x": "bf16", "y": "bf16",
         "smooth": True, "bias": True, "pad": 0},
        # the first MLP layer with its GELU, from 32-bit activations
        {"name": "layer, MLP fc1 f32 GELU", "op": "layer", "M": 4608, "K": 3072, "N": 12288, "x": "f32", "y": "gelu",
         "smooth": True, "bias": True, "pad": 0},
        # the deepest U-Net level: 8 x 8 positions, two images
        {"name": "norm, 8x8x1280", "op": "norm", "B": 2, "S": 64, "G": 32, "C": 1280, "x": "bf16", "y": "bf16",
         "act": "silu", "pad": 0},
        # the first U-Net level: 64 x 64 positions, 10 channels to a group
        {"name": "norm, 64x64x320", "op": "norm", "B": 2, "S": 4096, "G": 32, "C": 320, "x": "bf16", "y": "bf16",
         "act": "silu", "pad": 0},
        # an autoencoder's decoder in 32 bits: 512 x 512 positions, past the card's caches
        {"name": "norm, 512x512x256 f32", "op": "norm", "B": 1, "S": 262144, "G": 32, "C": 256, "x": "f32", "y": "f32",
         "act": "silu", "pad": 0},
        # the norm before a spatial transformer and its projection, 32 x 32 positions
        {"name": "norm and layer, 32x32x640", "op": "norm_layer", "B": 2, "S": 1024, "G": 32, "C": 640, "N": 640,
         "x": "bf16", "act": "none", "smooth": True, "pad": 0},
        # the same at 64 x 64 positions of four images, with an activation
        {"name": "norm and layer, 64x64x320", "op": "norm_layer", "B": 4, "S": 4096, "G": 32, "C": 320, "N": 1280,
         "x": "bf16", "act": "silu", "smooth": True, "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "layer", "norm", "norm_layer"])
    if op in ("product", "layer"):
        # the largest listed product is 4608 x 12288 x 3072
        while True:
            c = {"op": op, "M": _log(rng, 1, 9216), "K": _log(rng, 64, 12288), "N": _log(rng, 32, 12288)}
            if c["M"] * c["K"] * c["N"] <= 4608 * 12288 * 3072:
                break
        if rng.random() < 0.5:
            c["K"] = _r128(c["K"])
        c["y"] = rng.choice(["bf16", "f32", "gelu"])
        c["bias"] = rng.random() < 0.5
        if op == "layer":
            c["x"] = rng.choice(["bf16", "bf16", "f32"])
            c["smooth"] = rng.random() < 0.7
            c["pad"] = rng.choice([0, 0, 8, 100, 1])
        return c
    G = rng.choice([8, 16, 32, 32, 32])
    while True:
        c = {"op": op, "B": rng.choice([1, 1, 2, 3, 4]), "S": _log(rng, 1, 262144), "G": G, "C": G * _log(rng, 1, 80)}
        c["N"] = _log(rng, 32, 2560)
        n = c["B"] * c["S"]
        if op == "norm":
            del c["N"]
            if n * c["C"] <= 262144 * 256:
                break
        elif n * c["C"] <= 262144 * 64 and n * c["N"] <= 4608 * 12288:
            break
    c["x"] = rng.choice(["bf16", "bf16", "f32"])
    c["act"] = rng.choice(["none", "silu", "gelu"])
    c["pad"] = rng.choice([0, 0, 8, 3])
    if op == "norm":
        c["y"] = rng.choice([c["x"], "bf16"])
    else:
        c["smooth"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, K, N):
    """8-bit weight codes [N][K padded to 128, zeros there] of normal weights with one scale to an output channel."""
    w = _randn(g, N, K) / math.sqrt(K)
    sw = w.abs().amax(1) / 127.0
    q = torch.zeros(N, _r128(K), dtype=torch.int8, device="cuda")
    q[:, :K] = torch.round(w / sw[:, None]).clamp_(-127, 127).to(torch.int8)
    return q, sw


def _padded(t, pad):
    """t as the leading columns of rows that are `pad` values longer."""
    if not pad:
        return t
    b = torch.empty(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device=t.device)
    b[..., :t.shape[-1]] = t
    return b[..., :t.shape[-1]]


def _smoothing(g, K, outliers):
    """1 / s of the smoothing step: outlier channels (30 times the others) are divided down, the rest lie near 1."""
    s = torch.exp(0.2 * _randn(g, K))
    s[outliers] *= math.sqrt(30.0)
    return 1.0 / s


def _inputs(case, seed):
    g, op = _gen(seed), case["op"]
    d = dict(case)
    if op == "product":
        K = case["K"]
        d["qX"] = torch.zeros(case["M"], _r128(K), dtype=torch.int8, device="cuda")
        x = _randn(g, case["M"], K)
        a = x.abs().amax(1, keepdim=True)
        d["qX"][:, :K] = torch.round(x * (127.0 / a)).to(torch.int8)
        d["sX"] = (a / 127.0).reshape(-1).contiguous()
    elif op == "layer":
        K = case["K"]
        x = _randn(g, case["M"], K)
        out = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]
        x[:, out] *= 30.0
        d["X"] = _padded(x.to(_DT[case["x"]]), case["pad"])
        d["inv_s"] = _smoothing(g, K, out) if case["smooth"] else None
    else:
        C = case["C"]
        x = _randn(g, case["B"], case["S"], C)
        x *= torch.exp(0.5 * _randn(g, C))
        x += _randn(g, C)
        d["X"] = _padded(x.to(_DT[case["x"]]), case["pad"])
        d["gamma"], d["beta"], d["eps"] = 1.0 + 0.2 * _randn(g, C), 0.2 * _randn(g, C), 1e-5
        if op == "norm_layer":
            K = C
            out = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]
            d["inv_s"] = _smoothing(g, K, out) if case["smooth"] else None
    if op != "norm":
        d["qW"], d["sW"] = _weights(g, K, case["N"])
        d["bias"] = 0.1 * _randn(g, case["N"]) if case.get("bias", True) else None
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    if own:  # the layer and the norm as a program holds them: descriptions of the tensors above, nothing computed
        from bit_diffusion_model_amd import svdq

        if d["op"] != "norm":
            d["layer"] = svdq.Int8Linear(d["qW"], d["sW"], d.get("K", d.get("C")), inv_s=d.get("inv_s"), bias=d["bias"])
        if d["op"] in ("norm", "norm_layer"):
            act = {"none": svdq.GN_NONE, "silu": svdq.GN_SILU, "gelu": svdq.GN_GELU}[d["act"]]
            d["gn"] = svdq.GroupNorm(d["G"], d["C"], d["gamma"], d["beta"], d["eps"], act)
        d["ydtype"] = {"f32": svdq.F32, "bf16": svdq.BF16, "gelu": svdq.BF16_GELU}[d.get("y", "bf16")]
    return d


# ------------------------------------------------------------------------------------------- the plain forms

def _gelu(v):
    return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))


def _act(v, act):
    return v / (1.0 + torch.exp(-v)) if act == "silu" else _gelu(v) if act == "gelu" else v


def _plain_quantize(v, inv_s):
    if inv_s is not None:
        v = v * inv_s
    a = v.abs().amax(-1, keepdim=True).clamp_min(_FLOOR)
    c127 = torch.full_like(a, 127.0)  # a tensor, so that both quotients are true divisions
    return torch.round(v * (c127 / a)), a / c127


def _plain_product(q, sx, d):
    K = q.shape[-1]
    y = torch.matmul(q, d["qW"][:, :K].to(torch.float32).t()) * sx * d["sW"]
    if d["bias"] is not None:
        y = y + d["bias"]
    y_as = d.get("y", "bf16")
    return _gelu(y).to(torch.bfloat16) if y_as == "gelu" else y.to(_DT[y_as])


def _plain_norm(d):
    B, S, G, C = d["B"], d["S"], d["G"], d["C"]
    x = d["X"].to(torch.float32).reshape(B, S, G, C // G)
    x = x - x.mean((1, 3), keepdim=True)
    x = x * torch.rsqrt((x * x).mean((1, 3), keepdim=True) + d["eps"])
    return _act(x.reshape(B, S, C) * d["gamma"] + d["beta"], d["act"])


def _plain(d):
    if d["op"] == "product":
        return _plain_product(d["qX"][:, :d["K"]].to(torch.float32), d["sX"][:, None], d)
    if d["op"] == "layer":
        return _plain_product(*_plain_quantize(d["X"].to(torch.float32), d["inv_s"]), d)
    y = _plain_norm(d)
    if d["op"] == "norm":
        return y.to(_DT[d["y"]])
    return _plain_product(*_plain_quantize(y.reshape(-1, d["C"]), d["inv_s"]), d)


def run(state):
    if not own:
        return _plain(state)
    op, yd = state["op"], state["ydtype"]
    if op == "product":
        return state["layer"].gemm(state["qX"], state["sX"], yd)
    if op == "layer":
        return state["layer"].forward(state["X"], yd)
    if op == "norm":
        return state["gn"].forward(state["X"], yd)
    return state["gn"].forward_linear(state["X"], state["layer"], yd)


# -------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2, "gelu": 2}
    if op in ("product", "layer"):
        M, K, N = case["M"], case["K"], case["N"]
        n = N * K + 4 * N + (4 * N if case["bias"] else 0) + M * N * size[case["y"]]
        n += M * K + 4 * M if op == "product" else M * K * size[case["x"]] + (4 * K if case["smooth"] else 0)
        return {"bytes": n, "flops": 2 * M * N * K + (4 * M * K if op == "layer" else 0)}
    n = case["B"] * case["S"] * case["C"]
    b = n * size[case["x"]] + 8 * case["C"]
    f = n * (5 if case["act"] == "none" else 9)
    if op == "norm":
        return {"bytes": b + n * size[case["y"]], "flops": f}
    M, K, N = case["B"] * case["S"], case["C"], case["N"]
    return {"bytes": b + N * K + 8 * N + M * N * 2 + (4 * K if case["smooth"] else 0), "flops": f + 4 * n + 2 * M * N * K}


# -------------------------------------------------------------------------------------------------- 64 bits

def _gelu64(v):
    return v * torch.special.erfc(-v / math.sqrt(2.0)) / 2.0


def _quantize64(v, inv_s, rounded):
    """The definition: where the values come in 32 bits (`rounded`), each product and quotient that decides a code
    is rounded to 32 bits, as the definition says; otherwise the values themselves are in 64 bits."""
    f = (lambda t: t.to(torch.float32).to(torch.float64)) if rounded else (lambda t: t)
    if inv_s is not None:
        v = f(v * inv_s.double())
    a = torch.maximum(v.abs().amax(-1, keepdim=True), torch.tensor(_FLOOR, dtype=torch.float64, device=v.device))
    return torch.round(f(v * f(127.0 / a))), f(a / 127.0)


def exact(case, seed):
    d = _inputs(case, seed)
    op = d["op"]
    if op == "product":
        q, s = d["qX"][:, :d["K"]].double(), d["sX"].double()[:, None]
    elif op == "layer":
        q, s = _quantize64(d["X"].double(), d["inv_s"], True)
    else:
        B, S, G, C = d["B"], d["S"], d["G"], d["C"]
        x = d["X"].double().reshape(B, S, G, C // G)
        var, mean = torch.var_mean(x, dim=(1, 3), unbiased=False, keepdim=True)
        y = ((x - mean) / torch.sqrt(var + d["eps"])).reshape(B, S, C) * d["gamma"].double() + d["beta"].double()
        y = y * torch.sigmoid(y) if d["act"] == "silu" else _gelu64(y) if d["act"] == "gelu" else y
        if op == "norm":
            return y
        q, s = _quantize64(y.reshape(B * S, C), d["inv_s"], False)
    w = d["qW"][:, :q.shape[1]].double() * d["sW"].double()[:, None]
    y = torch.matmul(q * s, w.t())
    if d["bias"] is not None:
        y = y + d["bias"].double()
    return _gelu64(y) if d.get("y") == "gelu" else y
