"""tp_linear_colwise_fp8 and tp_linear_rowwise_fp8 against the definition in 64 bits on the same
codes and scales, and exactly on operands whose sums fp32 holds."""
import pytest
import torch

import block_reference as ref
import tensor_sharded_linear_amd as tsl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _pair(values_u8_codes, scale_bytes):
    """Device (codes, scales) with scale rows padded to whole dwords, the padding filled with NaN bytes."""
    m, kb = scale_bytes.shape
    s = torch.full((m, -(-kb // 4) * 4), 255, dtype=torch.uint8)
    s[:, :kb] = scale_bytes
    return values_u8_codes.cuda(), s.cuda().view(torch.float8_e8m0fnu)[:, :kb]


def _integers(g, rows, k):
    c = torch.randint(-4, 5, (rows, k), generator=g).float().to(torch.float8_e4m3fn)
    return _pair(c, torch.randint(127, 129, (rows, k // 128), generator=g, dtype=torch.uint8))


def _normal(g, rows, k, scale=1.0):
    return tsl.tp_quantize_fp8((torch.randn(rows, k, generator=g) * scale * torch.exp(torch.randn(1, k, generator=g) / 2)).cuda())


ROWS = [1, 2, 3, 5, 8, 15, 16, 17, 31, 33, 48, 63, 64, 65, 80, 97, 112, 127, 128, 129, 192, 193, 224, 255, 256, 257, 400]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", [(16, 128), (48, 640), (144, 1152), (272, 384), (528, 256)])
def test_exact_on_small_integers(m, n, k):
    """Codes -4..4 and scales 1 or 2: every partial sum is an integer below 2^24, so any order of
    fp32 additions gives the exact sum.  Every row, column and scale has its own value, so a
    misplaced one shows."""
    g = torch.Generator().manual_seed(m * 7919 + n * 31 + k)
    x, w = _integers(g, m, k), _integers(g, n, k)
    y = tsl.tp_linear_rowwise_fp8(*x, *w)
    want = ref.values(*x) @ ref.values(*w).t()
    assert torch.equal(y.cpu().double(), want)
    y = tsl.tp_linear_colwise_fp8(*x, *w)                   # bf16: the exact sum, rounded once
    assert torch.equal(y.cpu(), want.float().to(BF))


@pytest.mark.parametrize("m", [1, 4, 16, 23, 64, 77, 128, 130, 333])
@pytest.mark.parametrize("act,bias,out", [("none", False, BF), ("none", True, F32), ("gelu_tanh", True, BF),
                                          ("gelu_tanh", False, F32), ("swiglu", True, BF), ("swiglu", False, F32)])
def test_epilogues_within_the_derived_bound(m, act, bias, out):
    n, k = 208, 896
    g = torch.Generator().manual_seed(m)
    rows = 2 * n if act == "swiglu" else n
    x, w = _normal(g, m, k), _normal(g, rows, k, k ** -0.5)
    b = torch.randn(rows, generator=g).to(BF).cuda() if bias else None
    y = tsl.tp_linear_colwise_fp8(*x, *w, b, act=act, out_dtype=out)
    assert y.dtype == out
    ref.check(y, *ref.linear(ref.values(*x), ref.values(*w), b, act, out == BF and m > 96), what=f"{m} {act}")


@pytest.mark.parametrize("m,n,k", [(700, 1040, 2304), (1500, 2320, 768), (4608, 272, 128), (90, 4624, 512),
                                   (1, 9232, 6144), (2, 16, 18432), (97, 9216, 256), (500, 256, 4608),
                                   (1500, 64, 896), (75001, 16, 384), (18999, 64, 256)])
def test_many_tiles(m, n, k):
    g = torch.Generator().manual_seed(m + n + k)
    x, w = _integers(g, m, k), _integers(g, n, k)
    y = tsl.tp_linear_rowwise_fp8(*x, *w)
    want = ref.values(*x).cuda() @ ref.values(*w).cuda().t().contiguous()
    assert torch.equal(y.double(), want)
    assert torch.equal(tsl.tp_linear_colwise_fp8(*x, *w), want.float().to(BF))


@pytest.mark.parametrize("m", [3, 60, 300, 13000])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_strided_operands_and_outputs(m, act):
    """Operands are columns [512, 1280) of wider rows (scale columns [4, 10)), the output lies inside a
    wider buffer whose other elements stay as they were."""
    n = 96
    g = torch.Generator().manual_seed(m)
    rows = 2 * n if act == "swiglu" else n
    xc, xs = _integers(g, m, 2048)
    wc, ws = _integers(g, rows, 2048)
    x, w = (xc[:, 512:1280], xs[:, 4:10]), (wc[:, 512:1280], ws[:, 4:10])
    for out, pad in ((BF, 16), (F32, 8)):
        buf = torch.full((m + 2, n + 2 * pad), 7.0, dtype=out, device="cuda")
        y = tsl.tp_linear_colwise_fp8(*x, *w, act=act, out=buf[1:m + 1, pad:pad + n])
        ref.check(y, *ref.linear(ref.values(*x), ref.values(*w), None, act))
        buf[1:m + 1, pad:pad + n] = 7.0
        assert (buf == 7).all()


@pytest.mark.parametrize("m,n,out,rows,cols", [(2290, 6128, BF, 256, 256), (4600, 2288, BF, 224, 192), (1000, 4592, BF, 192, 192),
                                                (2290, 6128, F32, 256, 256), (4600, 9200, F32, 224, 256),
                                                (1000, 4592, F32, 192, 192)])
def test_strided_operands_of_the_large_tiles(m, n, out, rows, cols):
    assert tsl.tp_linear_fp8_tile_shape(m, n, 640, "none", out) == (rows, cols)
    g = torch.Generator().manual_seed(rows)
    xc, xs = _integers(g, m, 1536)
    wc, ws = _integers(g, n, 1536)
    x, w = (xc[:, 512:1152], xs[:, 4:9]), (wc[:, 512:1152], ws[:, 4:9])
    buf = torch.full((m + 2, n + 32), 7.0, dtype=out, device="cuda")
    y = tsl.tp_linear_colwise_fp8(*x, *w, out=buf[1:m + 1, 16:16 + n])
    want = ref.values(*x).cuda() @ ref.values(*w).cuda().t().contiguous()
    assert torch.equal(y, want.to(out))
    buf[1:m + 1, 16:16 + n] = 7.0
    assert (buf == 7).all()


@pytest.mark.parametrize("m", [1, 20, 100, 260, 8400])
def test_nan_blocks_reach_their_row_and_column_only(m):
    """A NaN scale in one activation row and one weight row makes that output row and column NaN."""
    g = torch.Generator().manual_seed(m)
    n, k = 144, 512
    xv, wv = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g)
    xv[m // 2, 300] = float("inf")
    wv[77, 5] = float("nan")
    x, w = tsl.tp_quantize_fp8(xv.cuda()), tsl.tp_quantize_fp8(wv.cuda())
    y = tsl.tp_linear_colwise_fp8(*x, *w, out_dtype=F32).cpu()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[m // 2] = True
    want[:, 77] = True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("m", [1, 20, 100, 260, 25000])
@pytest.mark.parametrize("out", [BF, F32])
def test_nan_scales_of_finite_codes(m, out):
    """A scale byte of 255 is NaN whatever the codes: one block of a row of each operand."""
    g = torch.Generator().manual_seed(m)
    n, k = 48, 640
    xc, wc = (torch.randn(r, k, generator=g).to(torch.float8_e4m3fn) for r in (m, n))
    xs, ws = (torch.full((r, k // 128), 127, dtype=torch.uint8) for r in (m, n))
    xs[m - 1, 3] = 255
    ws[11, 4] = 255
    y = tsl.tp_linear_colwise_fp8(*_pair(xc, xs), *_pair(wc, ws), out_dtype=out).cpu()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[m - 1] = True
    want[:, 11] = True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("m", [1, 40, 300, 19000])
def test_scales_over_their_whole_range(m):
    """Scales 2^-60 .. 2^60 whose products stay within fp32: the scale of each block counts."""
    g = torch.Generator().manual_seed(5)
    n, k = 64, 512
    xc = torch.randint(1, 5, (m, k), generator=g).float().to(torch.float8_e4m3fn)
    wc = torch.randint(1, 5, (n, k), generator=g).float().to(torch.float8_e4m3fn)
    e = torch.tensor([-60, 60, -20, 33])
    x = _pair(xc, (127 + e).to(torch.uint8).expand(m, 4).contiguous())
    w = _pair(wc, (127 - e + torch.randint(-2, 3, (n, 4), generator=g)).to(torch.uint8))
    y = tsl.tp_linear_rowwise_fp8(*x, *w)
    ref.check(y, *ref.linear(ref.values(*x), ref.values(*w), None, "none"))


@pytest.mark.parametrize("m", [1, 40, 300, 19000])
@pytest.mark.parametrize("out", [BF, F32])
def test_scales_near_the_ends_of_their_range(m, out):
    """Values of 2^-120 and 2^121 are normal numbers of the widened operands: no block is lost."""
    g = torch.Generator().manual_seed(7)
    n, k = 64, 512
    xc = torch.randint(1, 5, (m, k), generator=g).float().to(torch.float8_e4m3fn)
    wc = torch.randint(1, 5, (n, k), generator=g).float().to(torch.float8_e4m3fn)
    e = torch.tensor([-120, 119, -100, 100])
    x = _pair(xc, (127 + e).to(torch.uint8).expand(m, 4).contiguous())
    w = _pair(wc, (127 - e + torch.randint(-2, 3, (n, 4), generator=g)).to(torch.uint8))
    y = tsl.tp_linear_colwise_fp8(*x, *w, out_dtype=out)
    ref.check(y, *ref.linear(ref.values(*x), ref.values(*w), None, "none", out == BF and m > 96))


@pytest.mark.parametrize("m", [1, 20, 100, 260, 25000])
@pytest.mark.parametrize("out", [BF, F32])
def test_nan_codes_under_finite_scales(m, out):
    """The codes 0x7f and 0xff are NaN whatever the scale: one feature of a row of each operand."""
    g = torch.Generator().manual_seed(m)
    n, k = 48, 640
    xc, wc = (torch.randn(r, k, generator=g).to(torch.float8_e4m3fn) for r in (m, n))
    xs, ws = (torch.full((r, k // 128), 127, dtype=torch.uint8) for r in (m, n))
    xc.view(torch.uint8)[m - 1, 333] = 0x7f
    wc.view(torch.uint8)[11, 639] = 0xff
    y = tsl.tp_linear_colwise_fp8(*_pair(xc, xs), *_pair(wc, ws), out_dtype=out).cpu()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[m - 1] = True
    want[:, 11] = True
    assert torch.equal(torch.isnan(y), want)


# One ragged problem for every tile that exists: (m, n, act, output, tile rows, tile columns).  The last
# row and column tiles are partial, and K is three scale blocks: the scale dword's last byte is padding.
TILES = [(2290, 6128, "none", BF, 256, 256), (4600, 9200, "gelu_tanh", BF, 224, 256), (4600, 2288, "none", BF, 224, 192),
         (1000, 4592, "gelu_tanh", BF, 192, 192), (300, 9200, "none", BF, 128, 128), (333, 6128, "none", BF, 96, 128), (129, 9200, "none", BF, 64, 128),
         (4600, 4592, "swiglu", BF, 224, 128), (4090, 2032, "swiglu", BF, 256, 128), (4600, 2288, "swiglu", BF, 192, 128),
         (300, 4592, "swiglu", BF, 128, 64), (333, 3056, "swiglu", BF, 96, 64), (129, 4592, "swiglu", BF, 64, 64), (2290, 6128, "none", F32, 256, 256),
         (4600, 9200, "gelu_tanh", F32, 224, 256), (1000, 4592, "none", F32, 192, 192), (300, 9200, "gelu_tanh", F32, 128, 128), (333, 6128, "none", F32, 96, 128),
         (129, 9200, "none", F32, 64, 128), (4600, 4592, "swiglu", F32, 224, 128), (4090, 2032, "swiglu", F32, 256, 128),
         (300, 4592, "swiglu", F32, 128, 64), (333, 3056, "swiglu", F32, 96, 64), (129, 4592, "swiglu", F32, 64, 64)]


@pytest.mark.parametrize("m,n,act,out,rows,cols", TILES)
@pytest.mark.parametrize("k", [384, 1152])
def test_every_tile_with_ragged_edges(m, n, act, out, rows, cols, k):
    """Integer operands, so that sums are exact; the activation's bound is that of ref.linear."""
    assert tsl.tp_linear_fp8_tile_shape(m, n, k, act, out) == (rows, cols)
    g = torch.Generator().manual_seed(m + n)
    x, w = _integers(g, m, k), _integers(g, 2 * n if act == "swiglu" else n, k)
    b = torch.randint(-8, 9, (w[0].shape[0],), generator=g).to(BF).cuda()
    y = tsl.tp_linear_colwise_fp8(*x, *w, b, act=act, out_dtype=out).double()
    s = ref.values(*x).cuda() @ ref.values(*w).cuda().t().contiguous() + b.double()
    if act == "none":
        assert torch.equal(y, s.to(out).double())
        return
    if act == "gelu_tanh":
        want = 0.5 * s * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (s + 0.044715 * s ** 3)))
    else:
        want = s[:, :n] * torch.sigmoid(s[:, :n]) * s[:, n:]
    bound = 1e-5 * (1 + want.abs()) * 1.01 + ref.HALF_STEP[out] * want.abs()
    assert bool(((y - want).abs() <= bound).all())


# A problem for every instance of the split-K kernel: (m, n, act, its row blocks, its blocks of weight rows).
SPLITS = [(5, 48, "none", 1, 1), (21, 2576, "none", 2, 1), (35, 2736, "none", 3, 1), (1, 4368, "none", 1, 2), (23, 4368, "none", 2, 2),
          (41, 4368, "none", 3, 2), (51, 6272, "none", 4, 2), (70, 6272, "none", 5, 2), (85, 6272, "none", 6, 2),
          (9, 8464, "none", 1, 3), (31, 8464, "none", 2, 3), (47, 8464, "none", 3, 3), (63, 8464, "none", 4, 3), (79, 8464, "none", 5, 3),
          (95, 8464, "none", 6, 3), (2, 144, "swiglu", 1, 2), (27, 2064, "swiglu", 2, 2), (39, 2064, "swiglu", 3, 2),
          (57, 2576, "swiglu", 4, 2), (67, 2736, "swiglu", 5, 2), (267, 1360, "swiglu", 6, 2), (3, 4368, "swiglu", 1, 4),
          (25, 4368, "swiglu", 2, 4), (37, 4368, "swiglu", 3, 4), (61, 4368, "swiglu", 4, 4), (78, 4368, "swiglu", 5, 4)]


@pytest.mark.parametrize("m,n,act,mb,nb", SPLITS)
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("k", [384, 4736])
def test_every_split_with_ragged_edges(m, n, act, mb, nb, out, k):
    """Integer operands, so that sums are exact; the activation's bound is that of ref.linear."""
    if m > 96:
        k = 4736  # a tile's at the shorter K
    rows, cols = tsl.tp_linear_fp8_tile_shape(m, n, k, act, out)
    assert rows == 16 * mb and -(-cols // 16) * (2 if act == "swiglu" else 1) == nb, (rows, cols)
    g = torch.Generator().manual_seed(m + n)
    x, w = _integers(g, m, k), _integers(g, 2 * n if act == "swiglu" else n, k)
    b = torch.randint(-8, 9, (w[0].shape[0],), generator=g).to(BF).cuda()
    y = tsl.tp_linear_colwise_fp8(*x, *w, b, act=act, out_dtype=out).double()
    s = ref.values(*x).cuda() @ ref.values(*w).cuda().t().contiguous() + b.double()
    if act == "none":
        assert torch.equal(y, s.to(out).double())
        return
    want = s[:, :n] * torch.sigmoid(s[:, :n]) * s[:, n:]
    bound = 1e-5 * (1 + want.abs()) * 1.01 + ref.HALF_STEP[out] * want.abs()
    assert bool(((y - want).abs() <= bound).all())


@pytest.mark.parametrize("m,n", [(90, 128), (500, 128), (129, 9200), (1000, 4592), (2290, 6128)])
@pytest.mark.parametrize("out", [BF, F32])
def test_output_rows_beyond_32_bit_offsets(m, n, out):
    """Output rows far apart: the last ones lie more than 2^32 bytes behind the first."""
    g = torch.Generator().manual_seed(m)
    x, w = _integers(g, m, 256), _integers(g, n, 256)
    ld = ((1 << 32) // (m - 40) + 63) // 16 * 16
    y = torch.empty(m * ld, dtype=out, device="cuda").as_strided((m, n), (ld, 1))
    tsl.tp_linear_colwise_fp8(*x, *w, out=y)
    assert torch.equal(y.contiguous(), tsl.tp_linear_colwise_fp8(*x, *w, out_dtype=out))


def test_no_rows_is_a_no_op():
    w = _integers(torch.Generator().manual_seed(0), 32, 256)
    x = tsl.tp_quantize_fp8(torch.empty(0, 256, dtype=BF, device="cuda"))
    assert tsl.tp_linear_colwise_fp8(*x, *w).shape == (0, 32)
    assert tsl.tp_linear_rowwise_fp8(*x, *w).shape == (0, 32)


def test_rowwise_shards_sum_to_the_whole_product():
    """Quantized rows cut at multiples of 512 features: the partials of the cuts add up to the whole."""
    g = torch.Generator().manual_seed(9)
    x, w = _integers(g, 200, 2048), _integers(g, 160, 2048)
    whole = tsl.tp_linear_rowwise_fp8(*x, *w)
    parts = [tsl.tp_linear_rowwise_fp8(*(t[:, 512 * r // d:512 * (r + 1) // d] for t, d in
                                         ((x[0], 1), (x[1], 128), (w[0], 1), (w[1], 128)))) for r in range(4)]
    assert torch.equal(tsl.tp_partial_combine(parts, "sum"), whole)


def test_repeated_calls_give_the_same_bits():
    g = torch.Generator().manual_seed(11)
    for m in (1, 30, 120, 500):
        x, w = _normal(g, m, 1536), _normal(g, 400, 1536)
        first = tsl.tp_linear_rowwise_fp8(*x, *w)
        for _ in range(3):
            assert torch.equal(tsl.tp_linear_rowwise_fp8(*x, *w), first)
