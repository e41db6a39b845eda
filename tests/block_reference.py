"""64-bit references of the quantized rows, their products and the block boundary, and the error
bounds their tests use.  u = 2^-24 is the rounding of one fp32 operation."""
import torch

U = 2.0 ** -24
F64 = torch.float64
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}  # relative


def e4m3_round(v):
    """Nearest e4m3 value (ties to even) of 64-bit values within +-448."""
    a = v.abs()
    ex = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6)
    step = torch.exp2(ex - 3)
    return torch.round(v / step) * step   # torch.round is half to even; v / step is exact


def scale_exponent(amax):
    """Least e >= -126 with amax <= 448 2^e, by comparison; 0 where amax is 0."""
    e = torch.full_like(amax, -126)
    for k in range(-126, 129):
        e = torch.where(amax > 448 * 2.0 ** k, torch.full_like(e, k + 1), e)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def quantize(x):
    """(code values, scale values) in 64 bits, CPU; NaN blocks where x is not finite."""
    m, k = x.shape
    kb = -(-k // 128)
    p = torch.zeros(m, kb * 128, dtype=F64)
    p[:, :k] = x.to(F64).cpu()
    p = p.view(m, kb, 128)
    bad = ~torch.isfinite(p).all(2)
    s = torch.exp2(scale_exponent(torch.where(bad, torch.zeros((), dtype=F64), p.abs().amax(2))))
    q = e4m3_round(torch.where(bad.unsqueeze(2), torch.zeros((), dtype=F64), p) / s.unsqueeze(2))
    nan = torch.full((), float("nan"), dtype=F64)
    return torch.where(bad.unsqueeze(2), nan, q).view(m, kb * 128), torch.where(bad, nan, s)


def values(codes, scales):
    """What quantized rows stand for, 64 bits on the CPU (exact)."""
    c, s = codes.cpu().float().to(F64), scales.cpu().contiguous().view(torch.uint8)
    s64 = torch.where(s == 255, torch.full((), float("nan"), dtype=F64), torch.exp2(s.to(F64) - 127))
    return c * s64.repeat_interleave(128, 1)


def dropped(x, w):
    """What the 8-bit matrix cores may drop of x w^T: among the products of 8 consecutive features each of
    the 7 others loses less than 2^-13 of the largest."""
    xg, wg = x.abs().float().view(x.shape[0], -1, 8), w.abs().float().view(w.shape[0], -1, 8)
    out = torch.zeros(x.shape[0], w.shape[0], dtype=F64)
    for g in range(xg.shape[1]):
        top = torch.zeros(x.shape[0], w.shape[0])
        for k in range(8):
            top = torch.maximum(top, torch.outer(xg[:, g, k], wg[:, g, k]))
        out += top
    return 7 * 2.0 ** -13 * out


def linear(x, w, bias, act, eight=False):
    """(result, bound on the error before the output's rounding) of act(x w^T + bias), x and w in 64 bits.

    The matrix cores' sum of K products may round or cut at each of its K additions, each by at
    most 2 u of the sum of magnitudes S, and on the 8-bit cores (`eight`) drop what dropped()
    says; the bias adds one rounding.  The activations: |gelu'| < 1.13 and |silu'| < 1.1; their exp2 and
    reciprocal are good to a few u, and exp2 of an argument v (a + b v^2) of relative error 4 u
    moves the result by at most 4 u |arg| times it, under 1e-5 (1 + |y|) in all."""
    k = x.shape[1]
    y, s = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        b = bias.to(F64).cpu()
        y, s = y + b, s + b.abs()
    e = (k + 2) * 2 * U * s + (dropped(x, w) if eight else 0)
    if act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
        return y, 1.2 * e + 1e-5 * (1 + y.abs())
    if act == "swiglu":
        n = y.shape[1] // 2
        g, v = y[:, :n], y[:, n:]
        sg = g * torch.sigmoid(g)
        eg, ev = e[:, :n], e[:, n:]
        return sg * v, 1.1 * eg * (v.abs() + ev) + sg.abs() * ev + 1e-5 * (1 + (sg * v).abs())
    return y, e


def check(got, ref, err, what=""):
    """got within err plus its type's half step of the 64-bit ref; non-finite places alike."""
    g = got.detach().cpu().to(F64)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    # below the least normal number the step is absolute (2^-126 eps, flushed or not)
    bound = err + HALF_STEP[got.dtype] * (ref.abs() + err) + 2.0 ** -126
    off = torch.where(nan, torch.zeros_like(ref), (g - ref).abs() - bound)
    assert not (off > 0).any(), f"{what}: {int((off > 0).sum())} beyond the bound, worst by {float(off.max()):.3g}"


def norm(v, ev, kind, weight, bias, eps):
    """(normed v, bound): v in 64 bits known to ev.  A lane adds at most 32 features, then 64 lanes
    and 16 waves: under 64 roundings in each sum, so a mean is off by 64 u of the mean magnitude,
    and the factor 1 / sqrt(var + eps) by under 64 u relatively, plus what ev brings."""
    if kind == "none":
        return v, ev
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    n = c * r
    shift = 64 * U * v.abs().mean(1, keepdim=True) + ev.mean(1, keepdim=True) + U * v.abs()
    shift = shift if kind == "layer" else torch.zeros_like(shift)
    ec = ev + shift
    rel = 72 * U + (ec * ec).mean(1, keepdim=True).sqrt() * r   # of r: Cauchy-Schwarz on sum c ec
    e = ec * r + n.abs() * rel + ec * r * rel
    if weight is not None:
        w = weight.to(F64).cpu()
        n, e = n * w, e * w.abs() + U * (n * w).abs()
    if bias is not None:
        n = n + bias.to(F64).cpu()
        e = e + U * n.abs()
    return n, e


def block_norm(x, parts, bias, post, gate, residual, pre, scale, shift, eps, group):
    """((h, bound), (z, bound) or None).  post and pre: (kind, weight, bias); gate, scale, shift: tables
    or None; group: int64 [M], -1 for rows of no group."""
    x = x.cpu().to(F64)
    zero = torch.zeros_like(x)

    def rows(t):
        t = t.cpu().to(F64).reshape(-1, x.shape[1])
        inside = ((group >= 0) & (group < t.shape[0])).unsqueeze(1)
        return torch.where(inside, t[group.clamp(0, t.shape[0] - 1)], zero), inside

    h, eh = x, zero
    if parts:
        terms = [p.cpu().to(F64) for p in parts] + ([bias.cpu().to(F64).expand_as(x)] if bias is not None else [])
        y = sum(terms)
        ey = len(terms) * U * sum(t.abs() for t in terms)
        y, ey = norm(y, ey, *post, eps)
        if gate is not None:
            g, inside = rows(gate)
            y, ey = torch.where(inside, y * g, zero), torch.where(inside, ey * g.abs() + U * (y * g).abs(), zero)
        h = residual * x + y
        eh = ey + 2 * U * ((residual * x).abs() + h.abs())
    if pre[0] == "none":
        return (h, eh), None
    z, ez = norm(h, eh, *pre, eps)
    if scale is not None:
        s, _ = rows(scale)
        ez = ez * (1 + s).abs() + 3 * U * (z * (1 + s)).abs()
        z = z * (1 + s)
    if shift is not None:
        t, _ = rows(shift)
        z = z + t
        ez = ez + U * z.abs()
    return (h, eh), (z, ez)


def check_quantized(codes, scales, z, ez, what=""):
    """Quantized rows of a z known to ez: each block's scale is the rule's for some amax within the
    bound, and each code within half a step of z over that scale."""
    m, d = z.shape
    kb = codes.shape[1] // 128
    pad = lambda t: torch.nn.functional.pad(t, (0, kb * 128 - d)).view(m, kb, 128)  # noqa: E731
    zp, ep = pad(z), pad(ez)
    s = scales.cpu().contiguous().view(torch.uint8).to(F64) - 127
    lo = scale_exponent((zp.abs() - ep).clamp(min=0).amax(2))
    hi = scale_exponent((zp.abs() + ep).amax(2))
    zero = zp.abs().amax(2) == 0
    assert torch.all(torch.where(zero, s == 0, (s >= lo) & (s <= hi))), f"{what}: scales"
    c = codes.cpu().float().to(F64).view(m, kb, 128)
    v, e = zp / torch.exp2(s).unsqueeze(2), ep / torch.exp2(s).unsqueeze(2)
    a = v.abs() + e
    half = torch.exp2(torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6) - 4)
    assert torch.all((c - v).abs() <= half + e), f"{what}: codes, worst {float(((c - v).abs() - half - e).max()):.3g}"
