"""The operators around the block-scaled FP8 GEMM in a transformer sublayer: what a pass through each costs.

One sublayer is: normalise the residual stream into FP8 codes, multiply, apply the activation and
quantise again, multiply and add to the residual stream; and the gradients of those steps.

  norm           h = x + residual (rounded to the stream's type), y = h * rsqrt(mean(h^2) + eps) * weight,
                 y as FP8 codes with one scale per g x g block
  norm_backward  the gradient of x (and of the residual: the same tensor) and of the weight, from the gradient of y
  gemm           out = act(block-scaled A B + bias) + residual
  act            FP8 codes and scales of act(z)
  act_backward   FP8 codes and scales of dout * act'(z), and the bias's gradient, its column sums

`run` computes each in elementary torch operations where `own` is false, and calls the framework where it is true.
"""
import math

import torch

own = False

EPS = 1e-6
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step, hidden size 7168 (the small-M GEMM workload's K)
        {"name": "norm_decode", "op": "norm", "rows": 1, "cols": 7168, "dtype": "bf16", "gran": 128, "fmt": "e4m3", "residual": True, "train": False},
        # a prefill or training batch: 8192 tokens, hidden size 4096 (the FFN workload's M and K)
        {"name": "norm_batch", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "gran": 128, "fmt": "e4m3", "residual": True, "train": True},
        # an FP32 stream, rows and columns that end inside a scale block, no residual (the first layer's norm)
        {"name": "norm_ragged_f32", "op": "norm", "rows": 1000, "cols": 2064, "dtype": "f32", "gran": 64, "fmt": "e5m2", "residual": False, "train": True},
        # the training batch's backward pass, with the gradient that comes down the skip path
        {"name": "norm_backward_batch", "op": "norm_backward", "rows": 8192, "cols": 4096, "dtype": "bf16", "skip": True},
        # a ragged micro-batch in FP32
        {"name": "norm_backward_ragged_f32", "op": "norm_backward", "rows": 333, "cols": 1552, "dtype": "f32", "skip": False},
        # one token through a 7168 x 7168 projection into the residual stream
        {"name": "gemm_decode", "op": "gemm", "m": 1, "n": 7168, "k": 7168, "layout": "nt", "gran": 128, "a_fmt": "e4m3", "b_fmt": "e4m3", "bias": False, "act": "none", "out": "bf16"},
        # the FFN's second product over the training batch: 14336 -> 4096, bias and residual
        {"name": "gemm_ffn_down", "op": "gemm", "m": 8192, "n": 4096, "k": 14336, "layout": "nt", "gran": 128, "a_fmt": "e4m3", "b_fmt": "e4m3", "bias": True, "act": "none", "out": "bf16"},
        # sizes that end inside tiles and scale blocks, weight stored [K, N], activation before the residual
        {"name": "gemm_ragged_gelu", "op": "gemm", "m": 1000, "n": 1552, "k": 2064, "layout": "nn", "gran": 64, "a_fmt": "e4m3", "b_fmt": "e4m3", "bias": True, "act": "gelu", "out": "bf16"},
        # the FFN's hidden activation over the training batch
        {"name": "act_batch_gelu", "op": "act", "rows": 8192, "cols": 14336, "dtype": "bf16", "gran": 128, "fmt": "e4m3", "act": "gelu"},
        # the same for a few tokens of a decode step
        {"name": "act_decode_gelu", "op": "act", "rows": 8, "cols": 14336, "dtype": "bf16", "gran": 128, "fmt": "e4m3", "act": "gelu"},
        # its backward pass: gradients in E5M2, the first product's bias gradient beside them
        {"name": "act_backward_batch_gelu", "op": "act_backward", "rows": 8192, "cols": 14336, "dtype": "bf16", "gran": 128, "fmt": "e5m2", "act": "gelu"},
        # a ragged FP32 micro-batch with ReLU
        {"name": "act_backward_ragged_f32", "op": "act_backward", "rows": 777, "cols": 2064, "dtype": "f32", "gran": 256, "fmt": "e4m3", "act": "relu"},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(-(-lo // step), int(v) // step) * step


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "gemm", "act", "act_backward"])
    gran = rng.choice([64, 128, 256])
    fmt = rng.choice(["e4m3", "e5m2"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemm":
        n = _spread(rng, 16, 4096, 16)
        k = _spread(rng, 16, 14336, 16)
        m = _spread(rng, 1, 8192)
        layout = rng.choice(["nt", "nn", "tn", "tt"])
        if layout[0] == "t":  # A stored [K, M]: rows of M bytes, a multiple of 16
            m = -(-m // 16) * 16
        return {"op": op, "m": m, "n": n, "k": k, "layout": layout, "gran": gran, "a_fmt": fmt, "b_fmt": "e4m3",
                "bias": rng.random() < 0.5, "act": rng.choice(["none", "relu", "gelu"]), "out": rng.choice(["bf16", "bf16", "f32"])}
    rows = _spread(rng, 1, 8192)
    if op in ("norm", "norm_backward"):
        cols = _spread(rng, 16, 16384, 16)
        if op == "norm":
            return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "gran": gran, "fmt": fmt,
                    "residual": rng.random() < 0.7, "train": rng.random() < 0.5}
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "skip": rng.random() < 0.7}
    cols = _spread(rng, 16, 14336, 16)
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "gran": gran, "fmt": fmt, "act": rng.choice(["none", "relu", "gelu"] if op == "act_backward" else ["relu", "gelu"])}


# ------------------------------------------------------------------ inputs


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _stream(gen, rows, cols):
    """A residual stream: every token has its own size, and a few columns are far larger than the others."""
    size = torch.exp2(_normal(gen, rows, 1))
    heavy = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    return _normal(gen, rows, cols) * size * heavy


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "gemm":
        m, n, k, g = case["m"], case["n"], case["k"], case["gran"]
        qa, s["sa"] = _quantize(_normal(gen, m, k), g, case["a_fmt"])
        qb, s["sb"] = _quantize(_normal(gen, n, k) * 0.02, g, case["b_fmt"])
        s["a"] = qa.t().contiguous() if case["layout"][0] == "t" else qa
        s["b"] = qb if case["layout"][1] == "t" else qb.t().contiguous()
        s["bias"] = _normal(gen, n) * 0.1 if case["bias"] else None
        s["residual"] = _stream(gen, m, n).to(FLOAT[case["out"]])
        return s
    rows, cols, dtype = case["rows"], case["cols"], FLOAT[case["dtype"]]
    if case["op"] == "norm":
        s["x"] = _stream(gen, rows, cols).to(dtype)
        s["residual"] = _stream(gen, rows, cols).to(dtype) if case["residual"] else None
        s["weight"] = (1 + 0.3 * _normal(gen, cols)).to(dtype)
    elif case["op"] == "norm_backward":
        s["h"] = _stream(gen, rows, cols).to(dtype)
        s["weight"] = (1 + 0.3 * _normal(gen, cols)).to(dtype)
        s["rstd"] = (1 / (s["h"].double().square().mean(1) + EPS).sqrt()).float()
        s["dy"] = (_normal(gen, rows, cols) * 0.01).to(dtype)
        s["skip"] = (_normal(gen, rows, cols) * 0.01).to(dtype) if case["skip"] else None
    else:
        s["z"] = (_normal(gen, rows, cols) * 1.5).to(dtype) if case["act"] != "none" else None
        if case["op"] == "act_backward":
            s["dout"] = (_normal(gen, rows, cols) * 0.01 * torch.exp2(_normal(gen, rows, 1))).to(dtype)
    return s


# ------------------------------------------------------------------ plain forms, in 32 bits


def _quantize(y, g, fmt):
    """FP8 codes of y / s and the scales s = amax / FMAX of its g x g blocks (1 where that is 0)."""
    rows, cols = y.shape
    rb, cb = -(-rows // g), -(-cols // g)
    t = torch.nn.functional.pad(y, (0, cb * g - cols, 0, rb * g - rows)).view(rb, g, cb, g)
    s = t.abs().amax(dim=(1, 3)) / FMAX[fmt]
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (t / s[:, None, :, None]).clamp(-FMAX[fmt], FMAX[fmt]).view(rb * g, cb * g)[:rows, :cols]
    return q.to(FP8[fmt]).contiguous(), s


def _dequantize(q, s, g):
    rows, cols = q.shape
    return q.float() * s.repeat_interleave(g, 0)[:rows].repeat_interleave(g, 1)[:, :cols]


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        # the stream is rounded to its type first: the normalised values are those that the next layer reads
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        v = h.float()
        rstd = torch.rsqrt((v * v).mean(1) + EPS)
        q, scales = _quantize(v * rstd[:, None] * s["weight"].float(), c["gran"], c["fmt"])
        return {"codes": q, "scales": scales, "stream": None if s["residual"] is None else h, "rstd": rstd if c["train"] else None}
    if c["op"] == "norm_backward":
        n = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        dn = dy * s["weight"].float()
        dx = (dn - n * (dn * n).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["skip"] is not None:
            dx = dx + s["skip"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * n).sum(0)}
    if c["op"] == "gemm":
        a = s["a"].t() if c["layout"][0] == "t" else s["a"]
        b = s["b"] if c["layout"][1] == "t" else s["b"].t()
        v = _dequantize(a, s["sa"], c["gran"]) @ _dequantize(b, s["sb"], c["gran"]).t()
        if s["bias"] is not None:
            v = v + s["bias"]
        return {"out": (_act(v, c["act"]) + s["residual"].float()).to(FLOAT[c["out"]])}
    if c["op"] == "act":
        q, scales = _quantize(_act(s["z"].float(), c["act"]), c["gran"], c["fmt"])
        return {"codes": q, "scales": scales}
    dz = s["dout"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), c["act"])
    q, scales = _quantize(dz, c["gran"], c["fmt"])
    return {"codes": q, "scales": scales, "dbias": dz.sum(0)}


# ------------------------------------------------------------------ the framework's calls


def _framework(s):
    import fp8_block_scaled_bsgemm_b200 as bsg
    c = s["case"]
    if c["op"] == "norm":
        r = bsg.rms_norm_quantize(s["x"], s["weight"], residual=s["residual"], eps=EPS, gran=c["gran"], fmt=c["fmt"], return_rstd=c["train"])
        return {"codes": r[0].view(FP8[c["fmt"]]), "scales": r[1], "stream": None if s["residual"] is None else r[2], "rstd": r[3] if c["train"] else None}
    if c["op"] == "norm_backward":
        dx, dweight = bsg.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dresidual=s["skip"])
        return {"dx": dx, "dweight": dweight}
    if c["op"] == "gemm":
        return {"out": bsg.gemm(s["a"], s["b"], s["sa"], s["sb"], layout=c["layout"], gran=c["gran"], bias=s["bias"],
                                activation=c["act"], out_dtype=FLOAT[c["out"]], residual=s["residual"])}
    if c["op"] == "act":
        q, scales = bsg.activation_quantize(s["z"], c["act"], gran=c["gran"], fmt=c["fmt"])
        return {"codes": q.view(FP8[c["fmt"]]), "scales": scales}
    q, scales, dbias = bsg.activation_backward_quantize(s["dout"], s["z"], c["act"], gran=c["gran"], fmt=c["fmt"])
    return {"codes": q.view(FP8[c["fmt"]]), "scales": scales, "dbias": dbias}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ------------------------------------------------------------------ cost


def work(case):
    if case["op"] == "gemm":
        m, n, k, g = case["m"], case["n"], case["k"], case["gran"]
        es = FLOAT[case["out"]].itemsize
        kb = -(-k // g)
        scales = 4 * kb * (-(-m // g) + -(-n // g))
        return {"bytes": m * k + n * k + scales + 2 * m * n * es + (4 * n if case["bias"] else 0), "flops": 2.0 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    es = FLOAT[case["dtype"]].itemsize
    n = rows * cols
    if case["op"] == "norm_backward":
        return {"bytes": n * es * (4 if case["skip"] else 3) + cols * (es + 4) + 4 * rows, "flops": 9.0 * n}
    scales = 4 * -(-rows // case["gran"]) * -(-cols // case["gran"])
    if case["op"] == "norm":
        return {"bytes": n * (es * (3 if case["residual"] else 1) + 1) + cols * es + scales + (4 * rows if case["train"] else 0), "flops": 7.0 * n}
    if case["op"] == "act":
        return {"bytes": n * (es + 1) + scales, "flops": 8.0 * n}
    return {"bytes": n * (es * (1 if case["act"] == "none" else 2) + 1) + scales + 4 * cols, "flops": 12.0 * n}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _exact_blocks(y, g, fmt):
    """What the codes are the nearest FP8 values of, and the scales: every block's largest magnitude over FMAX.

    The values stand before their rounding to 8 bits, so that an error says how far a code is from its value and not
    how many values lie next to a border. E5M2's rounding alone (2^-3, 0.05 in the mean) is too coarse to tell
    anything that way, so its codes have no value here; their scales have.
    """
    rows, cols = y.shape
    r = torch.arange(rows, device=y.device) // g
    c = torch.arange(cols, device=y.device) // g
    by_rows = torch.zeros(int(r[-1]) + 1, cols, device=y.device, dtype=torch.float64)
    by_rows = by_rows.scatter_reduce(0, r[:, None].expand(rows, cols), y.abs(), "amax")
    s = torch.zeros(by_rows.shape[0], int(c[-1]) + 1, device=y.device, dtype=torch.float64)
    s = s.scatter_reduce(1, c[None, :].expand(by_rows.shape[0], cols), by_rows, "amax") / FMAX[fmt]
    s[s == 0] = 1.0
    return y / s[r][:, c] if fmt == "e4m3" else None, s


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    if case["op"] == "gemm":
        g = case["gran"]
        a = s["a"].T.contiguous() if case["layout"][0] == "t" else s["a"]
        b = s["b"] if case["layout"][1] == "t" else s["b"].T.contiguous()
        i, j, k = (torch.arange(v, device="cuda") // g for v in (case["m"], case["n"], case["k"]))
        a.mul_(s["sa"][i][:, k])
        b.mul_(s["sb"][j][:, k])
        v = torch.einsum("mk,nk->mn", a, b)
        if s["bias"] is not None:
            v += s["bias"][None, :]
        if case["act"] == "relu":
            v = torch.maximum(v, torch.zeros_like(v))
        elif case["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        return {"out": v + s["residual"]}
    if case["op"] == "norm":
        h = s["x"]
        if s["residual"] is not None:
            h = (h + s["residual"]).to(FLOAT[case["dtype"]]).double()
        rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"] + EPS)
        codes, scales = _exact_blocks(h / rms[:, None] * s["weight"], case["gran"], case["fmt"])
        return {"codes": codes, "scales": scales, "stream": None if s["residual"] is None else h, "rstd": 1 / rms if case["train"] else None}
    if case["op"] == "norm_backward":
        # y = w h r with r = (mean(h^2) + eps)^(-1/2), so dr/dh_j = -r^3 h_j / cols
        r = s["rstd"][:, None]
        inner = torch.einsum("mc,mc,c->m", s["dy"], s["h"], s["weight"])[:, None]
        dx = r * s["dy"] * s["weight"] - r ** 3 * s["h"] * inner / case["cols"]
        if s["skip"] is not None:
            dx = dx + s["skip"]
        return {"dx": dx, "dweight": torch.einsum("mc,mc,m->c", s["dy"], s["h"], s["rstd"])}
    if case["op"] == "act":
        z = s["z"]
        y = torch.maximum(z, torch.zeros_like(z)) if case["act"] == "relu" else z * torch.special.ndtr(z)
        codes, scales = _exact_blocks(y, case["gran"], case["fmt"])
        return {"codes": codes, "scales": scales}
    dz = s["dout"]
    if case["act"] == "relu":
        dz = torch.where(s["z"] > 0, dz, torch.zeros_like(dz))
    elif case["act"] == "gelu":
        z = s["z"]
        dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    codes, scales = _exact_blocks(dz, case["gran"], case["fmt"])
    return {"codes": codes, "scales": scales, "dbias": dz.sum(dim=0)}
