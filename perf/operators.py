"""Cases of the operators around the attention: rotary positions with several axes, the norms
before and after a block with its gate and residual scale, and the 8-bit product with a scale
per block of 128 with the quantiser that makes its operands.

``run`` computes each in elementary torch operations, or, with ``own`` set, by this
repository's entry points.  ``exact`` restates the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
TINY = 2.0 ** -100  # smallest block maximum the quantiser divides by
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 8 streams, shared key heads, mixed text / image positions
        {"name": "rope_token", "op": "rope", "B": 8, "L": 1, "H": 16, "Hk": 4, "d": 128, "r": 128, "axes": 3,
         "dtype": "bf16", "packed": False, "adjacent": False, "per_axis": False, "inverse": False},
        # q and k of the long layer, read from the packed projection output, positions of a video
        {"name": "rope_video", "op": "rope", "B": 4, "L": 16384, "H": 12, "Hk": 12, "d": 64, "r": 64, "axes": 3,
         "dtype": "bf16", "packed": True, "adjacent": False, "per_axis": False, "inverse": False},
        # a single token a stream, all of a block's norms and its residual
        {"name": "norm_token", "op": "norm", "back": False, "B": 8, "L": 1, "C": 768, "dtype": "bf16",
         "param": "bf16", "y": True, "post": "rms", "pre": "rms", "gate": "channel", "bias": False},
        # the long layer's hidden states between two blocks, a gate for each sequence
        {"name": "norm_long", "op": "norm", "back": False, "B": 4, "L": 16384, "C": 768, "dtype": "bf16",
         "param": "bf16", "y": True, "post": "rms", "pre": "rms", "gate": "batch", "bias": False},
        # the same in training, with fp32 parameters
        {"name": "norm_long_back", "op": "norm", "back": True, "B": 4, "L": 16384, "C": 768, "dtype": "bf16",
         "param": "fp32", "y": True, "post": "rms", "pre": "rms", "gate": "batch", "bias": False},
        # layer norms with biases on an fp32 stream of odd sizes
        {"name": "norm_ragged_back", "op": "norm", "back": True, "B": 3, "L": 1371, "C": 1030, "dtype": "fp32",
         "param": "fp32", "y": True, "post": "layer", "pre": "layer", "gate": "channel", "bias": True},
        # a layer's input for a training step: rows for the product, columns for the weight's gradient
        {"name": "quant_activations", "op": "quant", "R": 65536, "C": 768, "dtype": "bf16", "fmt": "e4m3",
         "square": False, "rows": True, "cols": True},
        # an fp32 master weight, for the product and for the input's gradient
        {"name": "quant_weight", "op": "quant", "R": 4096, "C": 4096, "dtype": "fp32", "fmt": "e4m3",
         "square": True, "rows": True, "cols": True},
        # serving a few tokens: the weight is read once
        {"name": "product_tokens", "op": "product", "M": 4, "N": 8192, "K": 8192, "fa": "e4m3", "fb": "e4m3",
         "square": True, "bias": False, "out": "bf16"},
        # a ragged batch
        {"name": "product_ragged", "op": "product", "M": 777, "N": 2050, "K": 1104, "fa": "e4m3", "fb": "e4m3",
         "square": True, "bias": True, "out": "bf16"},
        # the long layer's q, k, v projection
        {"name": "product_qkv", "op": "product", "M": 65536, "N": 2304, "K": 768, "fa": "e4m3", "fb": "e4m3",
         "square": True, "bias": True, "out": "bf16"},
        # its weight's gradient: both operands scaled along the tokens, gradients in e5m2
        {"name": "product_weight_grad", "op": "product", "M": 2304, "N": 768, "K": 65536, "fa": "e5m2",
         "fb": "e4m3", "square": False, "bias": False, "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm", "quant", "product"])
    if op == "rope":
        d = rng.choice([64, 64, 128, 128, 80, 96])
        Hk = rng.choice([1, 2, 4, 8, 12])
        packed = rng.random() < 0.4
        H = Hk * (1 if packed else rng.choice([1, 2, 4]))
        tokens = 50_000_000 // ((H + Hk) * d)
        B = min(_log(rng, 1, 8), tokens)
        return {"op": op, "B": B, "L": _log(rng, 1, max(1, min(16384, tokens // B))), "H": H, "Hk": Hk, "d": d,
                "r": rng.choice([d, d, d, d // 2]), "axes": rng.choice([1, 2, 3, 3]),
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "packed": packed,
                "adjacent": rng.random() < 0.3, "per_axis": rng.random() < 0.4, "inverse": rng.random() < 0.4}
    if op == "norm":
        C = _log(rng, 48, 8192)
        if rng.random() < 0.7:
            C = max(64, C // 64 * 64)
        B = _log(rng, 1, 8)
        y = rng.random() < 0.85
        post = rng.choice(["rms", "layer", "none"]) if y else "none"
        return {"op": op, "back": rng.random() < 0.5, "B": B, "L": _log(rng, 1, max(1, min(16384, 25_000_000 // (C * B)))),
                "C": C, "dtype": (dt := rng.choice(["bf16", "bf16", "fp16", "fp32"])), "param": rng.choice([dt, "fp32"]),
                "y": y, "post": post, "pre": rng.choice(["rms", "layer", "none"]) if y else rng.choice(["rms", "layer"]),
                "gate": rng.choice(["none", "channel", "batch"]) if y else "none", "bias": rng.random() < 0.5}
    if op == "quant":
        R = _log(rng, 1, 65536)
        rows = rng.random() < 0.8
        return {"op": op, "R": R, "C": _log(rng, 16, max(16, min(8192, 50_000_000 // R))),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "square": rng.random() < 0.4, "rows": rows, "cols": True if not rows else rng.random() < 0.5}
    M = _log(rng, 1, 16384)
    N = _log(rng, 16, 8192)
    K = _log(rng, 16, max(16, min(8192, 100_000_000_000 // (M * N))))
    if rng.random() < 0.6:
        N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
    return {"op": op, "M": M, "N": N, "K": K, "fa": rng.choice(["e4m3", "e4m3", "e5m2"]), "fb": "e4m3",
            "square": rng.random() < 0.7, "bias": rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "fp32"])}


# ---------------------------------------------------------------- inputs
def _sections(c):
    """Pairs of each axis: an equal share, the remainder to the first."""
    n, a = c["r"] // 2, c["axes"]
    s = [n // a] * a
    s[0] += n - sum(s)
    return s


def _rope_tables(c):
    """Axis and frequency of each pair."""
    axis, freq = [], []
    n = c["r"] // 2
    for a, s in enumerate(_sections(c)):
        for i in range(s):
            j = len(axis)
            axis.append(a)
            freq.append(10000.0 ** (-i / s) if c["per_axis"] else 10000.0 ** (-j / n))
    return axis, freq


def _positions(c, g):
    """A text prefix, then frames of a video on a grid, as [axes, B, L]."""
    B, L, A = c["B"], c["L"], c["axes"]
    t = torch.arange(L, device="cuda").expand(B, L) + torch.randint(0, 100_000, (B, 1), generator=g, device="cuda")
    pre = torch.randint(0, 64, (B, 1), generator=g, device="cuda")
    i = (torch.arange(L, device="cuda").expand(B, L) - pre).clamp(min=0)
    frame, at = i // 576, i % 576
    p = torch.stack([t - i + frame, t - i + at // 24, t - i + at % 24])
    return (p if A == 3 else p[1:] if A == 2 else t[None]).contiguous()


def _pad16(codes):
    """The same codes in rows that start at multiples of 16 bytes."""
    R, C = codes.shape
    if C % 16 == 0:
        return codes.contiguous()
    p = torch.zeros((R, -(-C // 16) * 16), dtype=torch.uint8, device=codes.device).view(codes.dtype)
    p[:, :C] = codes
    return p[:, :C]


def _activations(R, C, g):
    """Normal values with some louder columns, as hidden states have."""
    loud = 1 + 20 * (torch.rand(C, generator=g, device="cuda") < 0.01)
    return torch.randn(R, C, generator=g, device="cuda") * loud


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, scale=1.0, shift=0.0, dtype=None):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype or DTYPES[c["dtype"]])

    if c["op"] == "rope":
        B, L, H, Hk, d = c["B"], c["L"], c["H"], c["Hk"], c["d"]
        if c["packed"]:
            x = rand(B, L, 3, H, d)
            c["q"], c["k"] = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
        else:
            c["q"], c["k"] = rand(B, H, L, d), rand(B, Hk, L, d)
        c["positions"] = _positions(c, g)
        axis, freq = _rope_tables(c)
        c["axis"] = torch.tensor(axis, device="cuda")
        c["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        if own:
            from block_sparse_attention_bigbird_b200 import bsa
            c["rope"] = bsa.bsa_rope_build(_sections(c), 10000.0, per_axis=c["per_axis"], adjacent=c["adjacent"])
    elif c["op"] == "norm":
        B, L, C = c["B"], c["L"], c["C"]
        P = DTYPES[c["param"]]
        c["x"] = rand(B, L, C, scale=2.0, shift=0.1)
        c["yt"] = rand(B, L, C, scale=0.7, shift=-0.05) if c["y"] else None
        for n in ("post", "pre"):
            c[n + "_weight"] = rand(C, scale=0.2, shift=1.0, dtype=P) if c[n] != "none" else None
            c[n + "_bias"] = rand(C, scale=0.2, dtype=P) if c[n] == "layer" and c["bias"] else None
        c["gatet"] = (None if c["gate"] == "none" else
                      rand(*((C,) if c["gate"] == "channel" else (B, C)), scale=0.3, shift=0.5, dtype=P))
        c["branch"], c["stream"] = (0.5, 0.875) if c["y"] else (1.0, 1.0)
        if c["back"]:
            # c["x"] stands for the stream after the block; its statistics come from the forward
            s = torch.zeros(B * L, 4, device="cuda")
            for k, n, t in ((0, "post", c["yt"]), (2, "pre", c["x"])):
                if c[n] != "none":
                    t = t.double().reshape(B * L, C)
                    m = t.mean(1) if c[n] == "layer" else torch.zeros(B * L, dtype=torch.float64, device="cuda")
                    s[:, k] = m
                    s[:, k + 1] = ((t - m[:, None]).square().mean(1) + EPS).rsqrt()
            c["stats"] = s
            c["dstream"] = rand(B, L, C)
            c["dnormed"] = rand(B, L, C) if c["pre"] != "none" else None
    elif c["op"] == "quant":
        c["x"] = (_activations(c["R"], c["C"], g) if not c["square"]
                  else torch.randn(c["R"], c["C"], generator=g, device="cuda") / math.sqrt(c["C"])).to(DTYPES[c["dtype"]])
    else:
        M, N, K = c["M"], c["N"], c["K"]
        a, c["a_scale"] = _quantise(_activations(M, K, g), c["fa"], 1, 128)
        b, c["b_scale"] = _quantise(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K), c["fb"],
                                    128 if c["square"] else 1, 128)
        c["a"], c["b"] = _pad16(a), _pad16(b)
        c["bt"] = rand(N, dtype=torch.bfloat16) if c["bias"] else None
    return c


# ---------------------------------------------------------------- plain forms
def _blocks(x, br, bc):
    """x [R, C] padded with zeros and seen as blocks [R / br, br, C / bc, bc]."""
    R, C = x.shape
    nr, nc = -(-R // br), -(-C // bc)
    if (nr * br, nc * bc) != (R, C):
        x = torch.nn.functional.pad(x, (0, nc * bc - C, 0, nr * br - R))
    return x.view(nr, br, nc, bc)


def _quantise(x, fmt, br, bc):
    R, C = x.shape
    x = _blocks(x.float(), br, bc)
    top = x.abs().amax((1, 3), keepdim=True).clamp(min=TINY)
    codes = (x * (TOP[fmt] / top)).clamp(-TOP[fmt], TOP[fmt])
    codes = codes.view(x.shape[0] * br, -1)[:R, :C].to(DTYPES[fmt])
    return codes, (top / TOP[fmt])[:, 0, :, 0].contiguous()


def _rope(c):
    a = c["positions"].double()[c["axis"]].permute(1, 2, 0) * c["freq"]  # [B, L, r / 2]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin
    out = []
    for x in (c["q"], c["k"]):
        x, t = x.float(), x.dtype
        n = c["r"] // 2
        if c["adjacent"]:
            u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
            w = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
        else:
            u, v = x[..., :n], x[..., n:2 * n]
            w = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
        out.append(torch.cat((w, x[..., 2 * n:]), -1).to(t))
    return out


def _unit(x, kind):
    """x normalised over its last axis, without weight and bias."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()


def _affine(n, w, b):
    n = n if w is None else n * w.float()
    return n if b is None else n + b.float()


def _over_tokens(gate):
    return None if gate is None else gate.float() if gate.dim() == 1 else gate.float()[:, None]


def _norm(c):
    x, t = c["x"].float(), c["x"].dtype
    if c["y"]:
        y = c["yt"].float()
        if c["post"] != "none":
            y = _affine(_unit(y, c["post"]), c["post_weight"], c["post_bias"])
        g = _over_tokens(c["gatet"])
        x = c["stream"] * x + c["branch"] * (y if g is None else g * y)
    out = {"stream": x.to(t)} if c["y"] else {}
    if c["pre"] != "none":
        out["normed"] = _affine(_unit(x, c["pre"]), c["pre_weight"], c["pre_bias"]).to(t)
    return out


def _unit_back(n, rstd, dn, kind):
    """The gradient of x where n = (x - mean) * rstd has gradient dn."""
    dn = dn - n * (dn * n).mean(-1, keepdim=True) - (dn.mean(-1, keepdim=True) if kind == "layer" else 0.0)
    return dn * rstd


def _norm_back(c):
    x, t, C = c["x"].float(), c["x"].dtype, c["C"]
    s = c["stats"].view(*x.shape[:2], 4)
    D, out = c["dstream"].float(), {}
    if c["pre"] != "none":
        dh = c["dnormed"].float()
        n = (x - s[..., 2:3]) * s[..., 3:4]
        out["pre_weight"] = (dh * n).sum((0, 1)).to(c["pre_weight"].dtype)
        if c["pre_bias"] is not None:
            out["pre_bias"] = dh.sum((0, 1)).to(c["pre_bias"].dtype)
        D = D + _unit_back(n, s[..., 3:4], dh * c["pre_weight"].float(), c["pre"])
    out["x"] = (c["stream"] * D).to(t)
    if not c["y"]:
        return out
    y, g = c["yt"].float(), _over_tokens(c["gatet"])
    n = (y - s[..., 0:1]) * s[..., 1:2] if c["post"] != "none" else y
    dz = c["branch"] * D
    if g is not None:
        z = _affine(n, c["post_weight"], c["post_bias"])
        out["gate"] = (dz * z).sum(1 if c["gate"] == "batch" else (0, 1)).to(c["gatet"].dtype)
        dz = dz * g
    if c["post"] != "none":
        out["post_weight"] = (dz * n).sum((0, 1)).to(c["post_weight"].dtype)
        if c["post_bias"] is not None:
            out["post_bias"] = dz.sum((0, 1)).to(c["post_bias"].dtype)
        dz = _unit_back(n, s[..., 1:2], dz * c["post_weight"].float(), c["post"])
    out["y"] = dz.to(t)
    return out


def _quant(c):
    out = {}
    br = 128 if c["square"] else 1
    if c["rows"]:
        out["codes"], out["scale"] = _quantise(c["x"], c["fmt"], br, 128)
    if c["cols"]:
        out["codes_t"], out["scale_t"] = _quantise(c["x"].t(), c["fmt"], br, 128)
    return out


def _spread(scale, rows, cols):
    """A scale for each element from one for each block."""
    br = 128 if scale.shape[0] != rows else 1
    return scale.repeat_interleave(br, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _product(c):
    a = c["a"].float() * _spread(c["a_scale"], c["M"], c["K"])
    b = c["b"].float() * _spread(c["b_scale"], c["N"], c["K"])
    d = a @ b.t()
    if c["bt"] is not None:
        d = d + c["bt"].float()
    return d.to(DTYPES[c["out"]])


# ---------------------------------------------------------------- one pass
def run(state):
    c = state
    if not own:
        if c["op"] == "rope":
            return _rope(c)
        if c["op"] == "norm":
            return _norm_back(c) if c["back"] else _norm(c)
        return _quant(c) if c["op"] == "quant" else _product(c)
    from block_sparse_attention_bigbird_b200 import bsa
    if c["op"] == "rope":
        return list(bsa.bsa_rope_apply(c["q"], c["k"], c["positions"], c["rope"], inverse=c["inverse"]))
    if c["op"] == "norm":
        args = {"post": None if c["post"] == "none" else c["post"], "post_weight": c["post_weight"],
                "post_bias": c["post_bias"], "gate": c["gatet"], "pre": None if c["pre"] == "none" else c["pre"],
                "pre_weight": c["pre_weight"], "pre_bias": c["pre_bias"], "branch_scale": c["branch"],
                "stream_scale": c["stream"]}
        if not c["back"]:
            stream, normed, _ = bsa.bsa_block_norm(c["x"], c["yt"], eps=EPS, **args)
            out = {"stream": stream if c["y"] else None, "normed": normed}
        else:
            out = bsa.bsa_block_norm_backward(c["dstream"], c["dnormed"], c["x"], c["yt"], c["stats"], **args)
        return {k: v for k, v in out.items() if v is not None}
    if c["op"] == "quant":
        got = bsa.bsa_fp8_quantize(c["x"], square=c["square"], rows=c["rows"], cols=c["cols"], dtype=DTYPES[c["fmt"]])
        names = (["codes", "scale"] if c["rows"] else []) + (["codes_t", "scale_t"] if c["cols"] else [])
        return dict(zip(names, got))
    return bsa.bsa_fp8_matmul(c["a"], c["a_scale"], c["b"], c["b_scale"], bias=c["bt"], out_dtype=DTYPES[c["out"]])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "rope":
        n = c["B"] * c["L"] * (c["H"] + c["Hk"]) * c["d"]
        return {"bytes": 2 * n * size[c["dtype"]] + 8 * c["axes"] * c["B"] * c["L"], "flops": 3 * n}
    if c["op"] == "norm":
        n = c["B"] * c["L"] * c["C"] * size[c["dtype"]]
        pre, y = c["pre"] != "none", c["y"]
        # forward: x, y in, the stream and its norm out; backward: the stream, y and two gradients in, two out
        arrays = (1 + 1 + pre + 2 * y + pre) if c["back"] else (1 + 2 * y + pre)
        return {"bytes": n * arrays, "flops": (20 if c["back"] else 10) * n // size[c["dtype"]]}
    if c["op"] == "quant":
        n = c["R"] * c["C"]
        return {"bytes": n * (size[c["dtype"]] + c["rows"] + c["cols"]), "flops": 3 * n}
    M, N, K = c["M"], c["N"], c["K"]
    scales = 4 * (M + (N / 128 if c["square"] else N)) * K / 128
    return {"bytes": M * K + N * K + scales + M * N * size[c["out"]], "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits
def _grid(v, fmt):
    """The nearest values of the 8-bit format, ties to even."""
    low, digits = (-6, 3) if fmt == "e4m3" else (-14, 2)
    e = torch.frexp(v)[1].sub(1).clamp(min=low)
    step = torch.ldexp(torch.ones_like(v), e - digits)
    return (torch.round(v / step) * step).clamp(-TOP[fmt], TOP[fmt])


def _exact_quant(x, fmt, square):
    R, C = x.shape
    i = torch.arange(R, device=x.device) // (128 if square else 1)
    j = torch.arange(C, device=x.device) // 128
    top = x.new_zeros(int(i[-1]) + 1, C).index_reduce_(0, i, x.abs(), "amax")
    top = x.new_zeros(int(i[-1]) + 1, int(j[-1]) + 1).index_reduce_(1, j, top, "amax").clamp(min=TINY)
    return _grid(x / (top / TOP[fmt])[i][:, j], fmt), top / TOP[fmt]


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "rope":
        turn = c["positions"].double()[c["axis"]].permute(1, 2, 0)[:, None] * c["freq"]
        turn = torch.polar(torch.ones_like(turn), -turn if c["inverse"] else turn)
        out, n = [], c["r"] // 2
        for x in (c["q"], c["k"]):
            x = x.double()
            u, v = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if c["adjacent"] else (x[..., :n], x[..., n:2 * n])
            z = torch.complex(u.contiguous(), v.contiguous()) * turn
            z = torch.view_as_real(z)
            z = z.flatten(-2) if c["adjacent"] else z.transpose(-1, -2).flatten(-2)
            out.append(torch.cat((z, x[..., 2 * n:]), -1))
        return out
    if c["op"] == "norm":
        leaf = {k: c[k].double().requires_grad_(c["back"]) for k in
                ("x", "yt", "post_weight", "post_bias", "gatet", "pre_weight", "pre_bias") if c[k] is not None}

        def unit(kind, t, name):
            t = t - t.mean(-1, keepdim=True) if kind == "layer" else t
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)
            return t * leaf[name + "_weight"] + leaf.get(name + "_bias", 0.0)

        branch = None
        if c["y"]:
            branch = unit(c["post"], leaf["yt"], "post") if c["post"] != "none" else leaf["yt"]
            if "gatet" in leaf:
                branch = branch * (leaf["gatet"] if c["gate"] == "channel" else leaf["gatet"].unsqueeze(1))
        if not c["back"]:
            s = leaf["x"] if branch is None else c["stream"] * leaf["x"] + c["branch"] * branch
            out = {"stream": s} if c["y"] else {}
            if c["pre"] != "none":
                out["normed"] = unit(c["pre"], s, "pre")
            return out
        # the stream after the block is given: its total gradient first, then through the branch
        loss = (c["dstream"].double() * leaf["x"]).sum()
        if c["pre"] != "none":
            loss = loss + (c["dnormed"].double() * unit(c["pre"], leaf["x"], "pre")).sum()
        names = [k for k in leaf if k == "x" or k.startswith("pre")]
        got = dict(zip(names, torch.autograd.grad(loss, [leaf[k] for k in names])))
        D = got["x"]
        out = {k: v for k, v in got.items() if k != "x"} | {"x": c["stream"] * D}
        if branch is not None:
            names = [k for k in leaf if k in ("yt", "gatet", "post_weight", "post_bias")]
            more = torch.autograd.grad((c["branch"] * D * branch).sum(), [leaf[k] for k in names])
            out |= {{"yt": "y", "gatet": "gate"}.get(k, k): v for k, v in zip(names, more)}
        return out
    if c["op"] == "quant":
        out = {}
        if c["rows"]:
            out["codes"], out["scale"] = _exact_quant(c["x"].double(), c["fmt"], c["square"])
        if c["cols"]:
            out["codes_t"], out["scale_t"] = _exact_quant(c["x"].double().t().contiguous(), c["fmt"], c["square"])
        return out
    M, N, K = c["M"], c["N"], c["K"]
    total = torch.zeros(M, N, dtype=torch.float64, device="cuda") if c["bt"] is None else c["bt"].double().expand(M, N).clone()
    step = 128 * max(1, -(-K // 128) // 16)
    for k in range(0, K, step):
        blocks = torch.arange(k, min(K, k + step), device="cuda") // 128
        a = c["a"][:, k:k + step].double() * c["a_scale"].double()[:, blocks]
        sb = c["b_scale"].double()[:, blocks]
        if sb.shape[0] != N:
            sb = sb[torch.arange(N, device="cuda") // 128]
        total += a @ (c["b"][:, k:k + step].double() * sb).t()
    return total
