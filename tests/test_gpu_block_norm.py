"""tp_block_norm against its definition in 64 bits, within bounds that follow the fp32 arithmetic."""
import pytest
import torch

import block_reference as ref
import tensor_sharded_linear_amd as tsl

pytestmark = pytest.mark.gpu
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


def _run(m, d, *, x=BF, parts=0, part=F32, bias=False, post="none", gate=False, pre="layer", affine=False, mod=False,
         z=BF, groups=1, index=None, residual=1.0, table=BF, seed=0, group_rows=None, edit=None, in_place=False, eps=EPS):
    g = torch.Generator().manual_seed(seed + 31 * m + d)
    n = lambda *s, k=1.0, dt=F32: (torch.randn(*s, generator=g) * k).to(dt)  # noqa: E731
    t = dict(x=n(m, d, k=2.0, dt=x), parts=[n(m, d, dt=part) for _ in range(parts)], bias=n(d, dt=BF) if bias else None)
    t["post"] = (n(d, k=0.1, dt=BF) + 1, n(d, dt=BF)) if affine and post != "none" else (None, None)
    t["pre"] = (n(d, k=0.1, dt=BF) + 1, n(d, dt=BF)) if affine and pre != "none" else (None, None)
    for k in ("gate", "scale", "shift"):
        t[k] = n(groups, d, k=0.5, dt=table) if (gate if k == "gate" else mod) else None
    if edit:
        edit(t)
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    xd = dev(t["x"])
    if index is not None:
        how = dict(group_index=torch.tensor(index, dtype=torch.int32).cuda())
        group = torch.tensor(index, dtype=torch.int64)
        group = torch.where((group < 0) | (group >= groups), torch.full_like(group, -1), group)
    else:
        per = group_rows or max(1, -(-m // groups))
        how = dict(group_rows=per)
        group = torch.arange(m) // per
    h, got = tsl.tp_block_norm(
        xd, [dev(p) for p in t["parts"]] or None, bias=dev(t["bias"]), post_norm=post, post_weight=dev(t["post"][0]),
        post_bias=dev(t["post"][1]), gate=dev(t["gate"]), residual_scale=residual, pre_norm=pre,
        pre_weight=dev(t["pre"][0]), pre_bias=dev(t["pre"][1]), scale=dev(t["scale"]), shift=dev(t["shift"]), eps=eps,
        z_dtype=z, h_out=xd if in_place else None, **how)
    (wh, eh), wz = ref.block_norm(t["x"], t["parts"], t["bias"], (post, *t["post"]), t["gate"], residual,
                                  (pre, *t["pre"]), t["scale"], t["shift"], eps, group)
    if parts:
        assert h.dtype == x
        ref.check(h, wh, eh, "h")
    else:
        assert h is xd
    if pre == "none":
        assert got is None
    elif z == FP8:
        ref.check_quantized(*got, *wz, "z")
    else:
        assert got.dtype == z
        ref.check(got, *wz, "z")
    return h, got


SIZES = [(1, 1), (1, 64), (3, 8), (2, 127), (5, 513), (4, 520), (9, 1536), (3, 2309), (2, 4104), (2, 6144), (1, 9000),
         (2, 16384), (2, 20011), (1, 24576), (1, 32768), (300, 264), (1025, 72), (520, 4616)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("pre,z", [("layer", BF), ("rms", F32), ("layer", FP8)])
def test_norm_before_a_block(m, d, pre, z):
    _run(m, d, pre=pre, z=z, mod=True, groups=min(m, 2))


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("post,pre,z", [("rms", "rms", FP8), ("layer", "none", BF), ("none", "layer", F32)])
def test_boundary(m, d, post, pre, z):
    _run(m, d, parts=2, bias=True, post=post, gate=True, pre=pre, z=z, mod=pre != "none", affine=True, groups=min(m, 3),
         x=F32 if z == F32 else BF)


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("part", [BF, F32])
@pytest.mark.parametrize("table", [BF, F32])
@pytest.mark.parametrize("z", [BF, F32, FP8])
def test_types(x, part, table, z):
    _run(11, 768, x=x, parts=1, part=part, table=table, z=z, gate=True, mod=True, residual=0.75)


@pytest.mark.parametrize("parts", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("d", [768, 1001])
def test_part_counts(parts, d):
    _run(13, d, parts=parts, bias=parts % 2 == 1, gate=parts != 3, mod=True)


@pytest.mark.parametrize("z", [BF, FP8])
def test_rows_without_a_group_keep_their_residual_whatever_the_branch_holds(z):
    """Index -1 and an index past the tables: no modulation, and NaN in the branch does not reach h."""
    index = [0, 2, -1, 1, 3, 2, 7, -5, 1]

    def edit(t):
        t["parts"][0][2] = float("nan")
        t["parts"][0][6, 3] = float("inf")

    h, _ = _run(9, 384, parts=1, gate=True, mod=True, groups=3, index=index, z=z, edit=edit)
    assert torch.isfinite(h[[2, 4, 6, 7]].float()).all()


def test_index_with_scale_and_shift_only():
    _run(6, 256, pre="rms", mod=True, groups=2, index=[1, 0, -1, 1, 2, 0])


@pytest.mark.parametrize("m,rows,groups", [(10, 3, 4), (10, 10, 1), (10, 16, 1), (7, 1, 7), (8, 3, 5)])
def test_group_rows(m, rows, groups):
    _run(m, 320, parts=1, gate=True, mod=True, groups=groups, group_rows=rows)


@pytest.mark.parametrize("d", [768, 770, 6144])
def test_in_place_residual(d):
    h, _ = _run(19, d, parts=3, bias=True, gate=True, mod=True, in_place=True)


def test_nan_row_stays_in_its_row():
    def edit(t):
        t["x"][3, 5] = float("nan")
    _, z = _run(8, 512, edit=edit)
    assert torch.equal(torch.isnan(z.cpu().float()).any(1), torch.arange(8) == 3)


def test_constant_rows_and_zero_rows():
    """A constant row has variance 0: 0 / sqrt(eps) is 0.  A zero row quantizes to zero with scale 1."""
    def edit(t):
        t["x"][0] = 3.0
        t["x"][1] = 0.0
    _, z = _run(2, 256, edit=edit, z=F32)
    assert (z.cpu() == 0).all()
    _, (c, s) = _run(2, 256, edit=edit, z=FP8)
    assert (c.cpu().float() == 0).all() and (s.cpu().contiguous().view(torch.uint8) == 127).all()


def test_large_mean_does_not_cancel():
    """Mean 1000, deviation about 2: the variance is taken about the mean (the bound holds)."""
    def edit(t):
        t["x"] += 1000.0
    _run(5, 4096, x=F32, z=F32, edit=edit)


def test_strided_tables_rows_and_outputs():
    """gate, scale and shift are column slices of one projection's output; x, parts, h and z are slices
    of wider rows at odd offsets, and the elements around the outputs stay."""
    g = torch.Generator().manual_seed(1)
    m, d = 21, 333
    mod = torch.randn(3, 6 * d, generator=g).to(BF)
    wide = lambda dt: torch.randn(m, d + 30, generator=g).to(dt)  # noqa: E731
    x, p0, p1 = wide(BF), wide(F32), wide(F32)
    sl = slice(7, 7 + d)
    tabs = [mod[:, i * d:(i + 1) * d] for i in (2, 3, 5)]
    md = mod.cuda()
    dtabs = [md[:, i * d:(i + 1) * d] for i in (2, 3, 5)]
    hb, zb = torch.full((m, d + 9), 5.0, dtype=BF, device="cuda"), torch.full((m, d + 9), 5.0, device="cuda")
    h, z = tsl.tp_block_norm(x.cuda()[:, sl], [p0.cuda()[:, sl], p1.cuda()[:, sl]], gate=dtabs[0], scale=dtabs[1],
                             shift=dtabs[2], h_out=hb[:, 3:3 + d], z_out=zb[:, 5:5 + d], z_dtype=F32)
    group = torch.arange(m) // 7
    (wh, eh), (wz, ez) = ref.block_norm(x[:, sl], [p0[:, sl], p1[:, sl]], None, ("none", None, None), tabs[0], 1.0,
                                        ("layer", None, None), tabs[1], tabs[2], EPS, group)
    ref.check(h, wh, eh)
    ref.check(z, wz, ez)
    hb[:, 3:3 + d] = 5
    zb[:, 5:5 + d] = 5
    assert (hb == 5).all() and (zb == 5).all()


def test_more_rows_than_one_launch_and_offsets_beyond_32_bits():
    """2^21 + 77 short rows (two launches), and rows that lie 2^30 and more elements apart."""
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn((1 << 21) + 77, 8, generator=g, device="cuda")
    p = torch.randn(x.shape, generator=g, device="cuda")
    index = torch.arange(x.shape[0], dtype=torch.int32, device="cuda") % 3
    gate = torch.randn(3, 8, generator=g, device="cuda").to(BF)
    h, z = tsl.tp_block_norm(x, [p], gate=gate, group_index=index, z_dtype=F32)
    for s in (slice(0, 50), slice((1 << 21) - 50, None)):
        (wh, eh), (wz, ez) = ref.block_norm(x[s], [p[s]], None, ("none", None, None), gate, 1.0, ("layer", None, None),
                                            None, None, EPS, index[s].long().cpu())
        ref.check(h[s], wh, eh)
        ref.check(z[s], wz, ez)
    d, ld = 640, (1 << 30) + 640
    bufs = [torch.empty(3 * ld, dtype=BF, device="cuda").as_strided((3, d), (ld, 1)) for _ in range(3)]
    for i, b in enumerate(bufs):
        b.copy_(torch.randn(3, d, generator=torch.Generator().manual_seed(i)).to(BF))
    x, p = bufs[0].clone(), bufs[1].clone()
    h, z = tsl.tp_block_norm(bufs[0], [bufs[1]], h_out=bufs[0], z_out=bufs[2])
    wh, wz = tsl.tp_block_norm(x, [p])
    assert torch.equal(h, wh) and torch.equal(z, wz)


def test_one_group_vectors_and_empty():
    x = torch.randn(4, 96, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    s = torch.randn(96, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    a = tsl.tp_block_norm(x, scale=s)[1]
    b = tsl.tp_block_norm(x, scale=s.unsqueeze(0))[1]
    assert torch.equal(a, b)
    h, z = tsl.tp_block_norm(x[:0], [x[:0]], gate=s, group_rows=1, z_dtype=FP8)
    assert h.shape == (0, 96) and z[0].shape == (0, 128)


def test_sum_equals_the_combine():
    """With no norm and no gate, h is the SUM combine plus the residual: on integers, exactly."""
    g = torch.Generator().manual_seed(4)
    parts = [torch.randint(-50, 50, (30, 640), generator=g).float().cuda() for _ in range(4)]
    b = torch.randint(-8, 8, (640,), generator=g).to(BF).cuda()
    x = torch.randint(-50, 50, (30, 640), generator=g).float().cuda()
    h, z = tsl.tp_block_norm(x, parts, bias=b, pre_norm="none")
    assert z is None and torch.equal(h, tsl.tp_partial_combine(parts, "sum", bias=b) + x)
