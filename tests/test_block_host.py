"""Host-side tests of include/tp_block.h: exported symbols, and bad arguments refused before any
device work.  CPU only: every call fails validation or is an M == 0 no-op."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import tensor_sharded_linear_amd as tsl
from tensor_sharded_linear_amd import _binding as B
from tensor_sharded_linear_amd import _block as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tp_block.h")
A = 0x7F0000000000   # fake, well-aligned device addresses: validation never dereferences them
INV, UNS = B.TP_ERR_INVALID_ARG, B.TP_ERR_UNSUPPORTED


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    syms = set(re.findall(r"\btp_status (tp_[a-z0-9_]+)\s*\(", text))
    assert syms == set(K.SIGNATURES)
    lib = K._library()
    for s in syms:
        assert hasattr(lib, s) and hasattr(tsl, s) and s in tsl.__all__


def test_struct_layout_matches_a_c_compiler(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("no host C compiler or ROCm headers")
    names = [f[0] for f in K._BlockNormArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "tp_block.h"\nint main(void) {\n' +
                   "".join(f'    printf("%zu\\n", offsetof(tp_block_norm_args, {n}));\n' for n in names) +
                   '    printf("%zu\\n", sizeof(tp_block_norm_args));\n    return 0;\n}\n')
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(K._BlockNormArgs, n).offset for n in names] + [ctypes.sizeof(K._BlockNormArgs)]


def quantize(**kw):
    a = dict(x=A, ldx=300, dt=0, codes=A, ldc=384, scales=A, lds=4, M=8, K=300, stream=None)
    a.update(kw)
    return K._library().tp_quantize_fp8(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), INV), (dict(M=-1), INV), (dict(dt=2), INV), (dict(ldx=299), INV), (dict(x=None), INV), (dict(x=A + 1), INV),
    (dict(x=A + 2, dt=1), INV), (dict(codes=None), INV), (dict(codes=A + 8), INV), (dict(ldc=376), INV), (dict(ldc=256), INV),
    (dict(scales=None), INV), (dict(scales=A + 2), INV), (dict(lds=2), INV), (dict(lds=6), INV), (dict(M=1 << 31), UNS),
    (dict(K=1 << 31), UNS), (dict(ldx=1 << 62), UNS), (dict(ldc=1 << 62), UNS), (dict(lds=1 << 62), UNS)])
def test_quantize_refusals(kw, status):
    assert quantize(**kw) == status
    assert tsl.tp_last_error().startswith("tp_quantize_fp8")


def linear(fn="tp_linear_colwise_fp8", **kw):
    a = dict(x=A, ldx=256, xs=A, ldxs=4, w=A, ldw=256, ws=A, ldws=4, bias=None, y=A, ldy=512, y_dtype=0, act=0, M=64,
             N=512, K=256, stream=None)
    a.update(kw)
    if fn.endswith("rowwise_fp8"):
        for k in ("bias", "y_dtype", "act"):
            a.pop(k)
    return getattr(K._library(), fn)(*a.values())


@pytest.mark.parametrize("fn", ["tp_linear_colwise_fp8", "tp_linear_rowwise_fp8"])
@pytest.mark.parametrize("kw,status", [
    (dict(K=192), UNS), (dict(N=500), UNS), (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(ldx=128), INV),
    (dict(ldx=264), INV), (dict(ldw=128), INV), (dict(ldw=264), INV), (dict(ldxs=1), INV), (dict(ldxs=6), INV),
    (dict(ldws=1), INV), (dict(ldws=6), INV), (dict(ldy=500), INV), (dict(ldy=513), INV), (dict(x=None), INV),
    (dict(xs=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(y=None), INV), (dict(x=A + 8), INV),
    (dict(w=A + 8), INV), (dict(xs=A + 2), INV), (dict(ws=A + 1), INV), (dict(y=A + 8), INV), (dict(M=1 << 31), UNS),
    (dict(N=1 << 31), UNS), (dict(K=1 << 31), UNS), (dict(ldx=1 << 62), UNS), (dict(ldw=1 << 62), UNS),
    (dict(ldy=1 << 62), UNS), (dict(ldxs=1 << 62), UNS), (dict(ldws=1 << 62), UNS),
    (dict(M=1 << 21, ldx=1 << 10, K=1 << 10, ldw=1 << 10, ldxs=8, ldws=8), UNS),       # 2 GiB of activations
    (dict(N=1 << 21, ldy=1 << 21, ldw=1 << 10, ldx=1 << 10, K=1 << 10, ldxs=8, ldws=8), UNS),   # 2 GiB of weights
    (dict(M=1 << 21, N=1 << 21, ldy=1 << 21, ldx=128, ldw=128, K=128), UNS)])          # more than 2^22 tiles
def test_linear_refusals(fn, kw, status):
    assert linear(fn, **kw) == status
    assert tsl.tp_last_error().startswith(fn)


def test_colwise_refusals():
    assert linear(bias=A + 4) == INV
    assert linear(y_dtype=2) == INV
    assert linear(act=3) == INV
    n, k = 1 << 18, 1 << 12   # n rows fit in 2 GiB, the 2 n of a [gate; up] weight do not
    assert linear(N=n, ldy=n, K=k, ldx=k, ldw=k, ldxs=32, ldws=32, act=B.TP_ACT_SWIGLU) == UNS
    assert "2 GiB" in tsl.tp_last_error()


def test_tile_shape_query():
    assert tsl.tp_linear_fp8_tile_shape(1, 9216, 6144) == (16, 36)
    assert tsl.tp_linear_fp8_tile_shape(96, 9216, 6144, "none", torch.float32) == (96, 36)
    assert tsl.tp_linear_fp8_tile_shape(0, 64, 128)[1] in range(4, 49)
    # one round of the split-K kernel's workgroups covers a small output, whatever its rows
    for out in (torch.bfloat16, torch.float32):
        rows, cols = tsl.tp_linear_fp8_tile_shape(500, 256, 9216, "none", out)
        assert rows in (16, 32, 48) and cols in (16, 32, 48)
    assert tsl.tp_linear_fp8_tile_shape(1 << 30, 1 << 30, 128) == (256, 256)
    rows, cols = tsl.tp_linear_fp8_tile_shape(4608, 9216, 6144, "gelu_tanh")
    assert rows in (192, 224, 256) and cols in (192, 256)
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(k=1 << 31), dict(act="relu"), dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            tsl.tp_linear_fp8_tile_shape(**{**dict(m=4, n=64, k=128), **bad})
    one = ctypes.c_int64()
    assert K._library().tp_linear_fp8_tile_shape(4, 64, 128, 0, 0, None, ctypes.byref(one)) == INV
    assert tsl.tp_last_error().startswith("tp_linear_fp8_tile_shape")


def test_empty_is_a_no_op():
    assert quantize(M=0, x=None, codes=None, scales=None) == B.TP_OK
    assert linear(M=0, x=None, xs=None, y=None) == B.TP_OK
    assert linear("tp_linear_rowwise_fp8", M=0, x=None, xs=None, y=None) == B.TP_OK
    assert norm(M=0, x=None, z=None) == B.TP_OK
    assert tsl.tp_last_error() == ""


def norm(parts=None, **kw):
    a = K._BlockNormArgs(M=8, D=256, x=A, ldx=256, pre_norm=1, z=A, ldz=256, residual_scale=1.0, eps=1e-6)
    if parts is not None:
        a.parts = (ctypes.c_void_p * max(1, len(parts)))(*parts)
        a.num_parts, a.ld_part, a.part_dtype = len(parts), 256, 1
        a.h, a.ldh = A, 256
    for k, v in kw.items():
        setattr(a, k, v)
    return K._library().tp_block_norm(ctypes.byref(a), None)


MOD = dict(scale=A, ld_scale=256, groups=1, group_rows=8)


@pytest.mark.parametrize("kw,status", [
    (dict(D=0), INV), (dict(M=-1), INV), (dict(M=1 << 31), UNS), (dict(D=32769, ldx=40000, ldz=40000), UNS),
    (dict(x_dtype=2), INV), (dict(part_dtype=5), INV), (dict(h_dtype=-1), INV), (dict(mod_dtype=2), INV),
    (dict(pre_norm=3), INV), (dict(post_norm=-1), INV), (dict(z_rows=3), INV), (dict(num_parts=-1), INV),
    (dict(num_parts=17), INV), (dict(x=None), INV), (dict(x=A + 1), INV), (dict(ldx=255), INV), (dict(ldx=1 << 62), UNS),
    (dict(z=None), INV), (dict(z=A + 1), INV), (dict(ldz=255), INV), (dict(z_scale=A), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(residual_scale=float("inf")), INV),
    (dict(residual_scale=2.0), INV), (dict(h=A, ldh=256), INV), (dict(bias=A), INV), (dict(post_norm=1), INV),
    (dict(post_weight=A), INV), (dict(pre_norm=0), INV), (dict(pre_norm=0, z=None), INV),
    (dict(z_rows=2, z_scale=None), INV), (dict(z_rows=2, z_scale=A + 1, ldzs=4), INV), (dict(z_rows=2, z_scale=A, ldzs=1), INV),
    (dict(z_rows=2, z_scale=A, ldzs=6), INV), (dict(z_rows=2, z_scale=A, ldzs=4, z=A + 8), INV),
    (dict(z_rows=2, z_scale=A, ldzs=4, ldz=248), INV), (dict(pre_weight=A + 1), INV), (dict(MOD, groups=0), INV),
    (dict(MOD, groups=2, group_rows=3), INV), (dict(MOD, group_rows=0), INV), (dict(MOD, ld_scale=255), INV),
    (dict(MOD, scale=A + 1), INV), (dict(MOD, group_index=A + 2), INV), (dict(group_index=A), INV),
    (dict(MOD, gate=A, ld_gate=256), INV), (dict(MOD, groups=1 << 31), INV)])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status
    assert tsl.tp_last_error().startswith("tp_block_norm")


@pytest.mark.parametrize("parts,kw", [
    ([A], dict(h=None)), ([A], dict(ldh=255)), ([A], dict(h=A + 1)), ([A], dict(ld_part=255)), ([None], {}), ([A, A + 2], {}),
    ([A], dict(parts_null=True)), ([A], dict(post_weight=A)), ([A], dict(pre_norm=0)),
    ([A], dict(pre_norm=0, z=None, pre_bias=A)), ([A], dict(MOD, pre_norm=0, z=None)), ([A], dict(bias=A + 1))])
def test_norm_refusals_with_parts(parts, kw):
    if kw.pop("parts_null", False):
        kw = dict(num_parts=1, ld_part=256, h=A, ldh=256)
        parts = None
    assert norm(parts, **kw) == INV
    assert tsl.tp_last_error().startswith("tp_block_norm")


def test_null_args():
    assert K._library().tp_block_norm(None, None) == INV


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tsl.tp_quantize_fp8(x)
    with pytest.raises(TypeError):
        tsl.tp_linear_rowwise_fp8(x, x, x, x)
    with pytest.raises(TypeError):
        tsl.tp_block_norm(x)


@pytest.mark.gpu
def test_binding_refusals_on_the_gpu():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    q, s = tsl.tp_quantize_fp8(x)
    for bad in (lambda: tsl.tp_quantize_fp8(x.half()), lambda: tsl.tp_quantize_fp8(x, codes=q),
                lambda: tsl.tp_quantize_fp8(x[:3], codes=q, scales=s), lambda: tsl.tp_quantize_fp8(x[:, :0]),
                lambda: tsl.tp_linear_colwise_fp8(q, s, q[:, :128], s[:, :1]), lambda: tsl.tp_linear_colwise_fp8(q, s[:3], q, s),
                lambda: tsl.tp_linear_colwise_fp8(q, s, q, s, act="relu"), lambda: tsl.tp_linear_colwise_fp8(q, s, q, s),
                lambda: tsl.tp_linear_rowwise_fp8(q.view(torch.uint8), s, q, s),
                lambda: tsl.tp_block_norm(x, []), lambda: tsl.tp_block_norm(x, [x[:3]]), lambda: tsl.tp_block_norm(x, h_out=x),
                lambda: tsl.tp_block_norm(x, pre_norm="batch"), lambda: tsl.tp_block_norm(x, z_dtype=torch.float16),
                lambda: tsl.tp_block_norm(x, scale=x[:3]), lambda: tsl.tp_block_norm(x, scale=x[:2], shift=x[:1]),
                lambda: tsl.tp_block_norm(x, scale=x[:1], shift=x[:1].float()),
                lambda: tsl.tp_block_norm(x, scale=x[:1], group_index=torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: tsl.tp_block_norm(x, group_index=torch.zeros(4, dtype=torch.int32, device="cuda")),
                lambda: tsl.tp_block_norm(x, scale=x[:1], group_rows=4, group_index=torch.zeros(4, dtype=torch.int32, device="cuda")),
                lambda: tsl.tp_block_norm(x, pre_weight=x[0, :255]), lambda: tsl.tp_block_norm(x, z_out=x[:3])):
        with pytest.raises((ValueError, TypeError)):
            bad()
