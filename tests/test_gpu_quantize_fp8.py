"""tp_quantize_fp8 against its definition in 64 bits: codes and scales are equal, bit for bit (the
scaling is by powers of two, so the conversion's rounding is the only one)."""
import pytest
import torch

import tensor_sharded_linear_amd as tsl
from block_reference import quantize

pytestmark = pytest.mark.gpu


def _same(x, codes, scales):
    q, s = quantize(x)
    c = codes.cpu().float().double()
    assert torch.equal(torch.isnan(c), torch.isnan(q))
    assert torch.equal(torch.nan_to_num(c), torch.nan_to_num(q))
    b = scales.cpu().contiguous().view(torch.uint8)
    want = torch.where(torch.isnan(s), torch.full_like(s, 255.0), torch.log2(s) + 127).to(torch.uint8)
    assert torch.equal(b, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 7), (5, 129), (17, 127), (64, 256), (33, 1000), (2, 6144),
                                 (257, 640), (7, 18432)])
def test_codes_and_scales_equal_the_definition(m, k, dtype):
    g = torch.Generator().manual_seed(m * 1000 + k)
    x = (torch.randn(m, k, generator=g) * torch.exp2(torch.randint(-20, 20, (m, 1), generator=g).float())).to(dtype).cuda()
    codes, scales = tsl.tp_quantize_fp8(x)
    assert codes.shape == (m, -(-k // 128) * 128) and scales.shape == (m, -(-k // 128))
    assert codes.dtype == torch.float8_e4m3fn and scales.dtype == torch.float8_e8m0fnu
    _same(x, codes, scales)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_at_the_borders(dtype):
    """Maxima at 448 2^k and next to it, ties, subnormal codes, the smallest and largest numbers, zero
    blocks, signed zeros."""
    fi = torch.finfo(dtype)
    rows = []
    for top in (448.0, 448.0 * (1 + fi.eps), 448.0 * (1 - fi.eps), 449.0, 256.0, 512.0, 1.75, 1.75 * (1 + fi.eps), fi.max,
                fi.tiny, fi.tiny * fi.eps * 4, 0.0, 2.0 ** -120, 448.0 * 2.0 ** -126):
        r = torch.linspace(-1, 1, 128, dtype=torch.float64) * top
        r[5] = -0.0
        rows.append(r)
    ties = torch.tensor([448.0] + [(8 + i + 0.5) * 2.0 ** (e - 3) for e in range(-7, 8) for i in range(8)] +
                        [2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -10 * (1 + fi.eps), 2.0 ** -11, 0, 0, 0], dtype=torch.float64)
    assert ties.numel() == 128
    rows += [ties, -ties]
    x = torch.stack(rows).to(dtype).cuda()
    _same(x, *tsl.tp_quantize_fp8(x))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_blocks_are_nan_and_their_neighbours_are_not(bad):
    x = torch.randn(4, 512, generator=torch.Generator().manual_seed(3))
    x[1, 130] = bad
    x[3, 511] = bad
    for dtype in (torch.bfloat16, torch.float32):
        d = x.to(dtype).cuda()
        codes, scales = tsl.tp_quantize_fp8(d)
        _same(d, codes, scales)
        f = codes.cpu().float()
        assert torch.isnan(f[1, 128:256]).all() and torch.isnan(f[3, 384:]).all() and int(torch.isnan(f).sum()) == 256


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_strided_rows_and_outputs_in_place_of_a_larger_buffer(dtype, offset):
    """Columns [offset, offset + 200) of wider rows; outputs inside wider buffers whose other bytes stay."""
    g = torch.Generator().manual_seed(offset)
    x = torch.randn(37, 261, generator=g).to(dtype).cuda()[:, offset:offset + 200]
    codes = torch.full((40, 288), 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((40, 8), 9, dtype=torch.uint8, device="cuda")
    co, so = codes.view(torch.float8_e4m3fn)[:37, 16:272], scales.view(torch.float8_e8m0fnu)[:37, 4:6]
    tsl.tp_quantize_fp8(x, codes=co, scales=so)
    _same(x, co, so)
    assert (codes[37:] == 3).all() and (codes[:, :16] == 3).all() and (codes[:, 272:] == 3).all()
    assert (scales[37:] == 9).all() and (scales[:, :4] == 9).all() and (scales[:, 6:] == 9).all()


def test_no_rows_is_a_no_op():
    codes, scales = tsl.tp_quantize_fp8(torch.empty(0, 300, dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 384) and scales.shape == (0, 3)


def test_more_elements_than_32_bits_address():
    """Rows beyond 2^32 bytes of input: the last row is the definition's."""
    m, k = 70001, 32768
    x = torch.empty(m, k, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    codes, scales = tsl.tp_quantize_fp8(x)
    _same(x[-2:], codes[-2:], scales[-2:])
    _same(x[:1], codes[:1], scales[:1])
