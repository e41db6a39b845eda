"""The 8-bit block-scaled linear layers and the block-boundary norm: cases, plain forms and work.

Three operators, as one rank of a tensor-parallel transformer block chains them:

* ``quantize``  rows of a bf16 or fp32 matrix to 8-bit e4m3 codes with one power-of-two scale for
                each block of 128 consecutive features of a row;
* ``linear``    the colwise product (bias, GELU or SwiGLU) and the rowwise partial of two
                quantized operands;
* ``norm``      the boundary between two blocks: the partials' sum with its bias, the norm after
                the block, gate and residual, then the norm before the next block with its
                modulation, as bf16, fp32 or quantized rows.

``own = False`` computes them from elementary torch operations in 32 bits; ``own = True`` makes the
library's calls.  ``exact`` evaluates the definitions in 64 bits.
"""
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the conditioning rows of an adaLN projection, quantized before it: latency counts
        dict(name="quantize_4_rows", op="quantize", M=4, K=6144, dtype="bf16"),
        # one block's activations at 4608 tokens
        dict(name="quantize_tokens", op="quantize", M=4608, K=6144, dtype="bf16"),
        # fp32 rows of an odd width, as a summed partial of a narrow side layer has them
        dict(name="quantize_f32_ragged", op="quantize", M=1003, K=2309, dtype="f32"),
        # adaLN modulation of one sample at tp 4: the weight stream is all there is
        dict(name="linear_1_row", op="linear", style="colwise", M=1, N=9216, K=6144, act="none", bias=True, out="f32"),
        # a short text stream through the first FFN layer at tp 4
        dict(name="linear_77_rows", op="linear", style="colwise", M=77, N=4608, K=6144, act="gelu_tanh", bias=True, out="bf16"),
        # a few hundred tokens through the attention output at tp 8, ragged rows
        dict(name="linear_333_rows", op="linear", style="rowwise", M=333, N=6144, K=768, act="none", bias=False, out="f32"),
        # the FFN's first layer at tp 2, all tokens
        dict(name="linear_ffn_gelu", op="linear", style="colwise", M=4608, N=9216, K=6144, act="gelu_tanh", bias=True, out="bf16"),
        # the FFN's second layer at tp 4, all tokens: an fp32 partial
        dict(name="linear_ffn_rowwise", op="linear", style="rowwise", M=4608, N=6144, K=4608, act="none", bias=False, out="f32"),
        # the gated FFN's first layer at tp 4, all tokens
        dict(name="linear_ffn_swiglu", op="linear", style="colwise", M=4608, N=4608, K=6144, act="swiglu", bias=True, out="bf16"),
        # the first norm of a block for a few rows
        dict(name="norm_7_rows", op="norm", M=7, D=6144, x="bf16", parts=0, part="f32", bias=False, post="none", gate=False,
             pre="layer", affine=False, mod=True, z="bf16", groups=1, index=False, res=1.0),
        # a whole boundary at tp 4, all tokens, for quantized products: two samples
        dict(name="norm_boundary_fp8", op="norm", M=4608, D=6144, x="bf16", parts=4, part="f32", bias=True, post="none", gate=True,
             pre="layer", affine=False, mod=True, z="fp8", groups=2, index=False, res=1.0),
        # norms before and after the block, samples of unequal length in one batch, some rows padding
        dict(name="norm_sandwich", op="norm", M=2111, D=1536, x="f32", parts=1, part="bf16", bias=False, post="rms", gate=True,
             pre="rms", affine=True, mod=True, z="bf16", groups=5, index=True, res=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "norm"])
    if op == "quantize":
        M, K = _log(rng, 1, 4608), _log(rng, 1, 18432)
        while M * K > 4608 * 6144:
            M, K = max(1, M // 2), K
        return dict(op=op, M=M, K=K, dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        style = rng.choice(["colwise", "rowwise"])
        M, N, K = _log(rng, 1, 4608), 16 * _log(rng, 4, 576), 128 * _log(rng, 1, 72)
        act = rng.choice(["none", "gelu_tanh", "swiglu"]) if style == "colwise" else "none"
        while M * N * K * (2 if act == "swiglu" else 1) > 4608 * 9216 * 6144:
            M = M // 2
        return dict(op=op, style=style, M=M, N=N, K=K, act=act, bias=style == "colwise" and rng.random() < 0.6,
                    out="f32" if style == "rowwise" else rng.choice(["bf16", "f32"]))
    M, D = _log(rng, 1, 4608), _log(rng, 64, 6144)
    if rng.random() < 0.7:
        D = max(64, D // 8 * 8)
    parts = rng.choice([0, 1, 1, 2, 4])
    pre = rng.choice(["layer", "rms", "none"]) if parts else rng.choice(["layer", "rms"])
    gate, mod = bool(parts) and rng.random() < 0.7, pre != "none" and rng.random() < 0.7
    return dict(op=op, M=M, D=D, x=rng.choice(["bf16", "f32"]), parts=parts, part=rng.choice(["bf16", "f32"]) if parts == 1 else "f32",
                bias=bool(parts) and rng.random() < 0.5, post=rng.choice(["none", "rms", "layer"]) if parts else "none",
                gate=gate, pre=pre, affine=rng.random() < 0.4, mod=mod,
                z=rng.choice(["bf16", "f32", "fp8"]) if pre != "none" else "bf16", groups=min(M, rng.choice([1, 1, 2, 5])),
                index=(gate or mod) and rng.random() < 0.3, res=rng.choice([1.0, 1.0, 0.75]) if parts else 1.0)


# ------------------------------------------------------------------------------------ inputs

def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _plain_scale_exponent(amax):
    """Least e >= -126 with amax / 2^e <= 448; 0 for an all-zero block (fp32 in, integers out)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > E4M3_MAX / 512).to(torch.int32)
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(min=-126))


def _plain_quantize(x):
    """fp32 [M, K] -> e4m3 codes [M, K padded to 128], e8m0 scales [M, K padded / 128]."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    p = torch.zeros(M, kb * BLOCK, dtype=torch.float32, device=x.device)
    p[:, :K] = x
    p = p.view(M, kb, BLOCK)
    e = _plain_scale_exponent(p.abs().amax(2))
    codes = torch.ldexp(p, -e.unsqueeze(2)).to(torch.float8_e4m3fn).view(M, kb * BLOCK)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "quantize":
        # activations: some features are much larger than others
        spread = torch.exp(_normal(g, 1, c["K"]))
        return dict(case=c, x=(_normal(g, c["M"], c["K"]) * spread).to(_DT[c["dtype"]]))
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] == "swiglu" else N
        s = dict(case=c)
        s["x"], s["xs"] = _plain_quantize(_normal(g, M, K) * torch.exp(0.5 * _normal(g, 1, K)))
        s["w"], s["ws"] = _plain_quantize(_normal(g, rows, K, scale=K ** -0.5))
        # scale rows are read by dwords: a row's bytes are padded to a multiple of four
        for k in ("xs", "ws"):
            kb = s[k].shape[1]
            t = torch.zeros(s[k].shape[0], -(-kb // 4) * 4, dtype=torch.uint8, device="cuda")
            t[:, :kb] = s[k].view(torch.uint8)
            s[k] = t.view(torch.float8_e8m0fnu)[:, :kb]
        s["b"] = _normal(g, rows, dtype=torch.bfloat16) if c["bias"] else None
        return s
    M, D, G = c["M"], c["D"], c["groups"]
    s = dict(case=c, x=_normal(g, M, D, scale=2.0, dtype=_DT[c["x"]]))
    s["parts"] = [_normal(g, M, D, dtype=_DT[c["part"]]) for _ in range(c["parts"])]
    s["b"] = _normal(g, D, dtype=torch.bfloat16) if c["bias"] else None
    for k in ("post_w", "pre_w"):
        s[k] = _normal(g, D, scale=0.1, dtype=torch.float32).add_(1).to(torch.bfloat16) if c["affine"] else None
    for k in ("post_b", "pre_b"):
        s[k] = _normal(g, D, scale=0.1, dtype=torch.bfloat16) if c["affine"] else None
    mod = _normal(g, G, 3 * D, scale=0.5, dtype=torch.bfloat16)  # one adaLN projection's output: gate, scale, shift
    s["gate"] = mod[:, :D] if c["gate"] else None
    s["scale"], s["shift"] = (mod[:, D:2 * D], mod[:, 2 * D:]) if c["mod"] else (None, None)
    s["index"] = None
    if c["index"]:  # samples of unequal length one after another, the last few rows padding (-1)
        cut = torch.sort(torch.randint(0, M, (G - 1,), generator=g, device="cuda")).values
        s["index"] = torch.bucketize(torch.arange(M, device="cuda"), cut, right=True).to(torch.int32)
        s["index"][M - M // 50:] = -1
    return s


# ------------------------------------------------------------------------------------ plain forms

def _gelu(v):
    return v / (1 + torch.exp(-2 * 0.7978845608028654 * (v + 0.044715 * v * v * v)))


def _plain_linear(s, dt):
    c = s["case"]

    def widen(codes, scales):
        n, k = codes.shape
        return (codes.to(dt).view(n, k // BLOCK, BLOCK) * scales.to(dt).unsqueeze(2)).view(n, k)

    y = widen(s["x"], s["xs"]) @ widen(s["w"], s["ws"]).t()
    if s["b"] is not None:
        y = y + s["b"].to(dt)
    if c["act"] == "gelu_tanh":
        y = _gelu(y)
    elif c["act"] == "swiglu":
        a, u = y[:, :c["N"]], y[:, c["N"]:]
        y = a / (1 + torch.exp(-a)) * u
    return y


EPS = 1e-6


def _plain_norm(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    if kind != "none":
        v = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
        v = v if weight is None else v * weight.to(v.dtype)
        v = v if bias is None else v + bias.to(v.dtype)
    return v


def _plain_groups(s, t, dt):
    """Row r's modulation: its group's row of t, zeros where its index names no group."""
    c = s["case"]
    if s["index"] is None:
        at = torch.arange(c["M"], device="cuda") // -(-c["M"] // c["groups"])
        return t.to(dt)[at]
    at = s["index"].long()
    return torch.where((at >= 0).unsqueeze(1), t.to(dt)[at.clamp(min=0)], torch.zeros((), dtype=dt, device="cuda"))


def _plain_block_norm(s, dt):
    c = s["case"]
    h = s["x"].to(dt)
    if s["parts"]:
        y = s["parts"][0].to(dt)
        for p in s["parts"][1:]:
            y = y + p.to(dt)
        y = y if s["b"] is None else y + s["b"].to(dt)
        y = _plain_norm(y, c["post"], s["post_w"], s["post_b"])
        if s["gate"] is not None:
            y = y * _plain_groups(s, s["gate"], dt)
        h = c["res"] * h + y
    if c["pre"] == "none":
        return h, None
    z = _plain_norm(h, c["pre"], s["pre_w"], s["pre_b"])
    if s["scale"] is not None:
        z = z * (1 + _plain_groups(s, s["scale"], dt)) + _plain_groups(s, s["shift"], dt)
    return h, z


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "quantize":
        codes, scales = _plain_quantize(s["x"].float())
        return {"codes": codes, "scales": scales}
    if c["op"] == "linear":
        return {"y": _plain_linear(s, torch.float32).to(_DT[c["out"]])}
    h, z = _plain_block_norm(s, torch.float32)
    out = {"h": h.to(_DT[c["x"]])} if s["parts"] else {}
    if z is not None and c["z"] == "fp8":
        out["codes"], out["scales"] = _plain_quantize(z)
    elif z is not None:
        out["z"] = z.to(_DT[c["z"]])
    return out


# ------------------------------------------------------------------------------------ the library's calls

def _run_own(s, c):
    import tensor_sharded_linear_amd as tsl
    if c["op"] == "quantize":
        codes, scales = tsl.tp_quantize_fp8(s["x"])
        return {"codes": codes, "scales": scales}
    if c["op"] == "linear":
        if c["style"] == "rowwise":
            return {"y": tsl.tp_linear_rowwise_fp8(s["x"], s["xs"], s["w"], s["ws"])}
        return {"y": tsl.tp_linear_colwise_fp8(s["x"], s["xs"], s["w"], s["ws"], s["b"], act=c["act"], out_dtype=_DT[c["out"]])}
    post_affine, pre_affine = c["affine"] and c["post"] != "none", c["affine"] and c["pre"] != "none"
    h, z = tsl.tp_block_norm(
        s["x"], s["parts"] or None, bias=s["b"], post_norm=c["post"], post_weight=s["post_w"] if post_affine else None,
        post_bias=s["post_b"] if post_affine else None, gate=s["gate"], residual_scale=c["res"], pre_norm=c["pre"],
        pre_weight=s["pre_w"] if pre_affine else None, pre_bias=s["pre_b"] if pre_affine else None, scale=s["scale"],
        shift=s["shift"], eps=EPS, group_index=s["index"],
        group_rows=None if s["index"] is not None else -(-c["M"] // c["groups"]), z_dtype=_DT[c["z"]])
    out = {"h": h} if s["parts"] else {}
    if c["pre"] != "none" and c["z"] == "fp8":
        out["codes"], out["scales"] = z
    elif c["pre"] != "none":
        out["z"] = z
    return out


# ------------------------------------------------------------------------------------ work and exact values

_SIZE = {"bf16": 2, "f32": 4, "fp8": 1 + 1 / BLOCK}


def work(case):
    c = case
    if c["op"] == "quantize":
        kp = -(-c["K"] // BLOCK) * BLOCK
        return {"bytes": c["M"] * (c["K"] * _SIZE[c["dtype"]] + kp * _SIZE["fp8"]), "flops": 2 * c["M"] * c["K"]}
    if c["op"] == "linear":
        rows = c["N"] * (2 if c["act"] == "swiglu" else 1)
        return {"bytes": (c["M"] + rows) * c["K"] * _SIZE["fp8"] + c["M"] * c["N"] * _SIZE[c["out"]] + (2 * rows if c["bias"] else 0),
                "flops": 2 * c["M"] * rows * c["K"]}
    n = c["M"] * c["D"]
    b = n * _SIZE[c["x"]] + n * c["parts"] * _SIZE[c["part"]] + (n * _SIZE[c["x"]] if c["parts"] else 0)
    b += n * _SIZE[c["z"]] if c["pre"] != "none" else 0
    b += 2 * c["D"] * (c["groups"] * ((1 if c["gate"] else 0) + (2 if c["mod"] else 0)) + (1 if c["bias"] else 0)
                       + (2 if c["affine"] and c["post"] != "none" else 0) + (2 if c["affine"] and c["pre"] != "none" else 0))
    return {"bytes": b + (4 * c["M"] if c["index"] else 0), "flops": n * (c["parts"] + 12)}


def _exact_quantize(v):
    """The codes before their rounding to 8 bits (v over its block's scale), and the scales, in 64 bits."""
    M, K = v.shape
    kb = (K + BLOCK - 1) // BLOCK
    p = torch.nn.functional.pad(v, (0, kb * BLOCK - K)).reshape(M, kb, BLOCK)
    amax = p.abs().max(dim=2).values
    e = torch.ceil(torch.log2(amax / E4M3_MAX))
    # log2 of a value next to a power of two may round onto it: put e right by comparing
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > 0, e.clamp(min=-126), torch.zeros_like(e))
    scale = torch.exp2(e)
    return (p / scale.unsqueeze(2)).reshape(M, kb * BLOCK), scale


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64
    if c["op"] == "quantize":
        codes, scales = _exact_quantize(s["x"].to(f64))
        return {"codes": codes, "scales": scales}
    if c["op"] == "linear":
        x = s["x"].to(f64) * s["xs"].to(f64).repeat_interleave(BLOCK, dim=1)
        w = s["w"].to(f64) * s["ws"].to(f64).repeat_interleave(BLOCK, dim=1)
        y = torch.mm(x, w.t().contiguous())
        if s["b"] is not None:
            y += s["b"].to(f64)
        if c["act"] == "gelu_tanh":
            y = 0.5 * y * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
        elif c["act"] == "swiglu":
            y = y[:, :c["N"]] * torch.sigmoid(y[:, :c["N"]]) * y[:, c["N"]:]
        return {"y": y}

    def normed(v, kind, w, b):
        if kind == "none":
            return v
        centre = v.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros(1, 1, dtype=f64, device=v.device)
        v = (v - centre) * torch.rsqrt(((v - centre) ** 2).mean(dim=1, keepdim=True) + EPS)
        return v if w is None else v * w.to(f64) + b.to(f64)

    M, D, G = c["M"], c["D"], c["groups"]
    group = s["index"].long() if s["index"] is not None else torch.arange(M, device="cuda") // ((M + G - 1) // G)

    def of_group(t):  # a table with one more row, of zeros, for rows of no group
        return torch.cat([t.to(f64), torch.zeros(1, D, dtype=f64, device="cuda")]).index_select(0, torch.where(group < 0, G, group))

    out, h = {}, s["x"].to(f64)
    if s["parts"]:
        y = torch.stack([p.to(f64) for p in s["parts"]]).sum(0)
        if s["b"] is not None:
            y += s["b"].to(f64)
        y = normed(y, c["post"], s["post_w"], s["post_b"])
        out["h"] = h = c["res"] * h + (y if s["gate"] is None else of_group(s["gate"]) * y)
    if c["pre"] != "none":
        z = normed(h, c["pre"], s["pre_w"], s["pre_b"])
        if s["scale"] is not None:
            z = z + z * of_group(s["scale"]) + of_group(s["shift"])
        if c["z"] == "fp8":
            out["codes"], out["scales"] = _exact_quantize(z)
        else:
            out["z"] = z
    return out
