"""ctypes binding of the second part of libtp_linear.so (include/tp_block.h): quantized rows,
their products, and the norm at the boundary between two blocks.

Argument marshalling only, as in ``_binding``: outputs are allocated where none is passed, and
every step of the computation runs in the HIP kernels behind the C ABI.

Quantized rows are a pair ``(codes, scales)``: codes ``[rows, K8]`` ``torch.float8_e4m3fn`` with
K8 = K rounded up to a multiple of 128 (zero codes past K), scales ``[rows, K8 / 128]``
``torch.float8_e8m0fnu`` (powers of two).  Scale rows start at whole dwords: their row stride is a
multiple of 4, as :func:`tp_quantize_fp8` lays them out.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence

import torch

from . import _binding as _b
from ._binding import _check, _dev2d, _ld, _ptr, _vec

BLOCK = 128
CODES = torch.float8_e4m3fn
SCALES = torch.float8_e8m0fnu

_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_ROWS = {torch.bfloat16: 0, torch.float32: 1, CODES: 2}
_DT = _b._DT
_ACTS = {"none": _b.TP_ACT_NONE, "gelu_tanh": _b.TP_ACT_GELU_TANH, "swiglu": _b.TP_ACT_SWIGLU}


class _BlockNormArgs(ctypes.Structure):
    """tp_block_norm_args of include/tp_block.h."""
    _fields_ = [
        ("M", _I64), ("D", _I64), ("x", _P), ("ldx", _I64), ("x_dtype", _I), ("part_dtype", _I),
        ("parts", ctypes.POINTER(_P)), ("ld_part", _I64), ("num_parts", _I), ("post_norm", _I), ("bias", _P),
        ("post_weight", _P), ("post_bias", _P), ("h", _P), ("ldh", _I64), ("h_dtype", _I), ("pre_norm", _I),
        ("pre_weight", _P), ("pre_bias", _P), ("z", _P), ("ldz", _I64), ("z_scale", _P), ("ldzs", _I64),
        ("z_rows", _I), ("mod_dtype", _I), ("gate", _P), ("scale", _P), ("shift", _P), ("ld_gate", _I64),
        ("ld_scale", _I64), ("ld_shift", _I64), ("groups", _I64), ("group_rows", _I64), ("group_index", _P),
        ("residual_scale", _F), ("eps", _F)]


# The same layout for struct.pack: one call fills all fields, where setting 38 ctypes fields one by one
# took longer than the kernel of a few rows runs.
_PACK = struct.Struct("@qqPqiiPqiiPPPPqiiPPPqPqiiPPPqqqqqPff")
assert _PACK.size == ctypes.sizeof(_BlockNormArgs)

# Every symbol include/tp_block.h declares, with its ctypes signature.
SIGNATURES = {
    "tp_quantize_fp8": (_I, [_P, _I64, _I, _P, _I64, _P, _I64, _I64, _I64, _P]),
    "tp_linear_colwise_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I, _I, _I64, _I64, _I64, _P]),
    "tp_linear_rowwise_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P]),
    "tp_linear_fp8_tile_shape": (_I, [_I64, _I64, _I64, _I, _I, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "tp_block_norm": (_I, [_P, _P]),
}

_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = _b.load_library()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _call(fn, x: torch.Tensor, stream, *args) -> None:
    """Call an entry point on `stream` (default: the current one) with x's device current (the
    library launches on the current device)."""
    index = x.get_device()
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status:
        _check(status)


def _same_device(x: torch.Tensor, **others: Optional[torch.Tensor]) -> None:
    for name, t in others.items():
        if t is not None and t.get_device() != x.get_device():
            raise ValueError(f"{name} is on {t.device}, not on {x.device}")


def _empty_codes(m: int, k: int, device):
    """Codes and scales for m rows of k features; scale rows start at whole dwords.  (A product reads the
    last row's last dword whole: its last bytes may lie past the tensor, never past its allocation,
    whose granularity is a multiple of four.)"""
    kb = -(-k // BLOCK)
    return torch.empty_strided((m, kb * BLOCK), (kb * BLOCK, 1), dtype=CODES, device=device), \
        torch.empty_strided((m, kb), ((kb + 3) & -4, 1), dtype=SCALES, device=device)


def _codes(t: torch.Tensor, s: torch.Tensor, name: str, m: Optional[int] = None, k8: Optional[int] = None) -> None:
    """Checks a (codes, scales) pair, against [m, k8] where given."""
    _dev2d(t, f"{name} codes", CODES)
    _dev2d(s, f"{name} scales", SCALES)
    if k8 is not None and tuple(t.shape) != (m, k8):
        raise ValueError(f"{name} codes must be [{m}, {k8}], got {tuple(t.shape)}")
    if t.shape[1] % BLOCK:
        raise ValueError(f"{name} codes must have a multiple of {BLOCK} columns, got {t.shape[1]}")
    if tuple(s.shape) != (t.shape[0], t.shape[1] // BLOCK):
        raise ValueError(f"{name} scales must be [{t.shape[0]}, {t.shape[1] // BLOCK}], got {tuple(s.shape)}")


def _lds(s: torch.Tensor) -> int:
    """Row stride of scales; a single row's is its width rounded up to whole dwords."""
    if s.shape[0] > 1:
        return s.stride(0)
    return -(-max(s.stride(0), s.shape[1]) // 4) * 4


def _input(x: torch.Tensor):
    """(dtype number, device index, shape, address, row stride) of the matrix x."""
    try:
        shape, (ld, c) = x.shape, x.stride()
        (m, k), dtype, index = shape, _DT.get(x.dtype), x.get_device()
        good = dtype is not None and index >= 0 and k > 0 and (c == 1 or k == 1)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _dev2d(x, "x")   # names what is wrong, unless the type or the width is
        if x.dtype not in _DT:
            raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
        raise ValueError("x has no columns")
    return dtype, index, shape, x.data_ptr(), ld if m > 1 else k


def _place(t: torch.Tensor, name: str, shape, index: int):
    """(address, row stride) of a row-major matrix of this shape on cuda:`index`."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be a [{shape[0]}, {shape[1]}] tensor on cuda:{index}")
    ld, c = t.stride()
    if c != 1 and shape[1] > 1:
        _dev2d(t, name)   # raises
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def tp_quantize_fp8(x: torch.Tensor, *, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None, stream=None):
    """Quantize the rows of ``x`` [M, K] (bf16 or fp32, any K) to e4m3 codes with one
    power-of-two scale for each 128 features of a row.  Returns ``(codes, scales)``.

    Scale: the least 2^e, e >= -126, with max|x| <= 448 2^e (1 for an all-zero block); codes:
    x / 2^e rounded to nearest even.  A block with an infinity or a NaN becomes NaN."""
    lib = _library()
    dtype, _, (m, k), address, ld = _input(x)
    if (codes is None) != (scales is None):
        raise ValueError("pass both codes and scales, or neither")
    if codes is None:
        codes, scales = _empty_codes(m, k, x.device)
    else:
        _codes(codes, scales, "output", m, -(-k // BLOCK) * BLOCK)
        _same_device(x, codes=codes, scales=scales)
    _call(lib.tp_quantize_fp8, x, stream, address, ld, dtype, codes.data_ptr(), _ld(codes), scales.data_ptr(),
          _lds(scales), m, k)
    return codes, scales


def _rows(t: torch.Tensor, s: torch.Tensor, name: str):
    """(rows, features, code row stride, scale row stride) of a (codes, scales) operand."""
    try:
        (m, k), (ld, c) = t.shape, t.stride()
        (ms, kb), (lds, cs) = s.shape, s.stride()
        good = t.dtype == CODES and s.dtype == SCALES and t.is_cuda and s.is_cuda and c == 1 and ms == m and \
            kb * BLOCK == k and (cs == 1 or kb == 1)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _codes(t, s, name)   # names what is wrong; what it allows beyond the above is a single column
        raise ValueError(f"{name} has no columns")
    return m, k, ld if m > 1 else k, lds if m > 1 else -(-kb // 4) * 4


def _operands(x, x_scale, w, w_scale, x_name="x"):
    m, k, ldx, ldxs = _rows(x, x_scale, x_name)
    rows, kw, ldw, ldws = _rows(w, w_scale, "w_shard")
    if kw != k:
        raise ValueError(f"{x_name} is [M, {k}] but w_shard is {tuple(w.shape)}")
    index = x.get_device()
    if not index == x_scale.get_device() == w.get_device() == w_scale.get_device():
        raise ValueError(f"{x_name}, w_shard and their scales must be on one device")
    return m, rows, k, (x.data_ptr(), ldx, x_scale.data_ptr(), ldxs, w.data_ptr(), ldw, w_scale.data_ptr(), ldws)


def tp_linear_colwise_fp8(x: torch.Tensor, x_scale: torch.Tensor, w_shard: torch.Tensor, w_scale: torch.Tensor,
                          bias: Optional[torch.Tensor] = None, *, act: str = "none",
                          out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                          stream=None) -> torch.Tensor:
    """Colwise shard of quantized rows: ``out = act(x @ w_shard.T + bias)``, fp32 accumulation
    (fp32 output: exact products; large bf16 outputs of more than 96 rows: the 8-bit matrix cores).

    ``x``/``x_scale`` and ``w_shard``/``w_scale`` as :func:`tp_quantize_fp8` gives them; ``act``,
    ``bias`` and ``out`` as :func:`tp_linear_colwise` (``"swiglu"``: a packed [gate; up] shard)."""
    lib = _library()
    m, rows, k, operands = _operands(x, x_scale, w_shard, w_scale)
    if act not in _ACTS:
        raise ValueError("act must be 'none', 'gelu_tanh' or 'swiglu'")
    a = _ACTS[act]
    if a == _b.TP_ACT_SWIGLU and rows % 2:
        raise ValueError(f"a SwiGLU shard has an even number of rows [gate; up], got {rows}")
    n = rows // 2 if a == _b.TP_ACT_SWIGLU else rows
    bias = _vec(bias, "bias", rows)
    if out is None:
        if out_dtype not in _DT:
            raise ValueError("out_dtype must be bf16 or fp32")
        out = torch.empty_strided((m, n), (n, 1), dtype=out_dtype, device=x.device)
    else:
        _dev2d(out, "out")
        if tuple(out.shape) != (m, n) or out.dtype not in _DT:
            raise ValueError(f"out must be [{m}, {n}] bf16 or fp32")
    _same_device(x, bias=bias, out=out)
    _call(lib.tp_linear_colwise_fp8, x, stream, *operands, _ptr(bias), out.data_ptr(), _ld(out), _DT[out.dtype], a,
          m, n, k)
    return out


def tp_linear_rowwise_fp8(x_shard: torch.Tensor, x_scale: torch.Tensor, w_shard: torch.Tensor,
                          w_scale: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rowwise shard of quantized rows: fp32 partial ``out = x_shard @ w_shard.T`` (no bias)."""
    lib = _library()
    m, n, k, operands = _operands(x_shard, x_scale, w_shard, w_scale, "x_shard")
    if out is None:
        out = torch.empty_strided((m, n), (n, 1), dtype=torch.float32, device=x_shard.device)
    else:
        _dev2d(out, "out", torch.float32)
        if tuple(out.shape) != (m, n):
            raise ValueError(f"out must be [{m}, {n}]")
        _same_device(x_shard, out=out)
    _call(lib.tp_linear_rowwise_fp8, x_shard, stream, *operands, out.data_ptr(), _ld(out), m, n, k)
    return out


def tp_linear_fp8_tile_shape(m: int, n: int, k: int, act: str = "none",
                             out_dtype: torch.dtype = torch.bfloat16) -> tuple:
    """(rows, cols) of the output tile that the products of quantized rows use for an [m, k] x
    [n, k]^T problem on the current device; where the split-K kernel runs (up to 96 rows, and small
    outputs) the rows that a workgroup's instance holds and its output columns.  For ``act="swiglu"`` n counts the outputs.
    Host-only query: no device work."""
    if act not in _ACTS:
        raise ValueError("act must be 'none', 'gelu_tanh' or 'swiglu'")
    if out_dtype not in _DT:
        raise ValueError("out_dtype must be bf16 or fp32")
    rows, cols = _I64(), _I64()
    _check(_library().tp_linear_fp8_tile_shape(m, n, k, _ACTS[act], _DT[out_dtype], ctypes.byref(rows), ctypes.byref(cols)))
    return rows.value, cols.value


def _feature_vec(t: torch.Tensor, name: str, d: int, index: int) -> int:
    if t.get_device() != index or t.dtype != torch.bfloat16 or t.shape != (d,) or (d > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous bf16 vector of length {d} on cuda:{index}")
    return t.data_ptr()


def _table(t: torch.Tensor, name: str, like: torch.Tensor, groups: int, d: int, index: int):
    """(address, row stride) of a modulation table [groups, d], or [d] for one group."""
    shape, strides = t.shape, t.stride()
    if len(shape) not in (1, 2) or shape[-1] != d or t.dtype not in _DT or t.get_device() != index or \
            (strides[-1] != 1 and d > 1):
        raise ValueError(f"{name} must be [groups, {d}] bf16 or fp32 on cuda:{index}, with unit column stride")
    if t.dtype != like.dtype or (shape[0] if len(shape) == 2 else 1) != groups:
        raise ValueError("gate, scale and shift must have one dtype and one number of groups")
    return t.data_ptr(), strides[0] if groups > 1 else d


def tp_block_norm(x: torch.Tensor, parts: Optional[Sequence[torch.Tensor]] = None, *,
                  bias: Optional[torch.Tensor] = None, post_norm: str = "none",
                  post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0, pre_norm: str = "layer",
                  pre_weight: Optional[torch.Tensor] = None, pre_bias: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  group_rows: Optional[int] = None, group_index: Optional[torch.Tensor] = None,
                  h_out: Optional[torch.Tensor] = None, z_out=None,
                  z_dtype: torch.dtype = torch.bfloat16, stream=None):
    """The boundary between two blocks, one pass over the rows of ``x`` [M, D]::

        y = sum(parts) + bias                       # the block's output, fp32 adds in order
        h = residual_scale * x + gate * post(y)     # the residual stream
        z = pre(h) * (1 + scale) + shift            # the next block's input

    ``post_norm`` / ``pre_norm``: ``"none"``, ``"layer"`` or ``"rms"``, with bf16 [D] weights and
    biases.  ``gate``, ``scale``, ``shift``: [groups, D] tables (or [D] for one group) of one
    dtype; row r takes group ``r // group_rows`` (default: M / groups, which must divide) or
    ``group_index[r]`` (int32 [M]; outside [0, groups): no modulation, and no gated branch).
    ``parts``: fp32 or bf16 partials, or None: then only z is computed and h is ``x``.
    Returns ``(h, z)``: h of ``x``'s dtype (``h_out`` may be ``x`` itself), z of ``z_dtype`` (bf16,
    fp32, or ``torch.float8_e4m3fn`` for a ``(codes, scales)`` pair), None for ``pre_norm="none"``."""
    lib = _library()
    x_dt, index, shape, x_p, ldx = _input(x)
    m, d = shape
    post, pre = _NORMS.get(post_norm), _NORMS.get(pre_norm)
    if post is None or pre is None:
        raise ValueError("post_norm and pre_norm must be 'none', 'layer' or 'rms'")
    h, z = x, None
    part_array = parts_p = num_parts = ldp = part_dt = h_p = ldh = h_dt = 0
    if parts is not None:
        num_parts = len(parts)
        if not num_parts:
            raise ValueError("no parts (pass None for a norm without a block's output)")
        dtype, addresses = parts[0].dtype, []
        for i, p in enumerate(parts):
            address, ld = _place(p, f"parts[{i}]", shape, index)
            addresses.append(address)
            if i == 0:
                ldp = ld
            if p.dtype != dtype or ld != ldp:
                raise ValueError("all parts must be of one dtype and row stride")
        if dtype not in _DT:
            raise TypeError(f"parts must be bf16 or fp32, got {dtype}")
        part_array, part_dt = (_P * num_parts)(*addresses), _DT[dtype]
        parts_p = ctypes.addressof(part_array)
        if h_out is None:
            h = torch.empty_strided(shape, (d, 1), dtype=x.dtype, device=x.device)
            h_p, ldh, h_dt = h.data_ptr(), d, x_dt
        else:
            h = h_out
            h_p, ldh = _place(h, "h_out", shape, index)
            if h.dtype not in _DT:
                raise ValueError(f"h_out must be bf16 or fp32, got {h.dtype}")
            h_dt = _DT[h.dtype]
    elif h_out is not None:
        raise ValueError("h_out without parts")
    z_p = ldz = zs_p = ldzs = z_rows = 0
    if not pre:
        if z_out is not None:
            raise ValueError("z_out without pre_norm")
    elif z_dtype not in _ROWS:
        raise ValueError("z_dtype must be bf16, fp32 or float8_e4m3fn")
    else:
        z_rows = _ROWS[z_dtype]
        if z_dtype == CODES:
            if z_out is None:
                codes, scales = z = _empty_codes(m, d, x.device)
            else:
                codes, scales = z = z_out
                _codes(codes, scales, "z_out", m, -(-d // BLOCK) * BLOCK)
                _same_device(x, z_codes=codes, z_scales=scales)
            z_p, ldz, zs_p, ldzs = codes.data_ptr(), _ld(codes), scales.data_ptr(), _lds(scales)
        elif z_out is None:
            z = torch.empty_strided(shape, (d, 1), dtype=z_dtype, device=x.device)
            z_p, ldz = z.data_ptr(), d
        else:
            z = z_out
            z_p, ldz = _place(z, "z_out", shape, index)
            if z.dtype != z_dtype:
                raise TypeError(f"z_out must be {z_dtype}, got {z.dtype}")
    mod_dt = groups = index_p = gate_p = ld_gate = scale_p = ld_scale = shift_p = ld_shift = 0
    first = gate if gate is not None else scale if scale is not None else shift
    if first is not None:
        groups = first.shape[0] if first.dim() == 2 else 1
        if gate is not None:
            gate_p, ld_gate = _table(gate, "gate", first, groups, d, index)
        if scale is not None:
            scale_p, ld_scale = _table(scale, "scale", first, groups, d, index)
        if shift is not None:
            shift_p, ld_shift = _table(shift, "shift", first, groups, d, index)
        mod_dt = _DT[first.dtype]
        if group_index is not None:
            if group_rows is not None:
                raise ValueError("pass group_rows or group_index, not both")
            if group_index.get_device() != index or group_index.dtype != torch.int32 or group_index.shape != (m,) or \
                    (m > 1 and group_index.stride(0) != 1):
                raise ValueError(f"group_index must be a contiguous int32 vector of length {m} on cuda:{index}")
            index_p = group_index.data_ptr()
        elif group_rows is None:
            if groups == 0 or m % groups:
                raise ValueError(f"{groups} groups do not divide {m} rows: pass group_rows or group_index")
            group_rows = max(1, m // groups)
    elif group_index is not None:
        raise ValueError("group_index without a gate, scale or shift")
    bias_p = 0 if bias is None else _feature_vec(bias, "bias", d, index)
    post_w = 0 if post_weight is None else _feature_vec(post_weight, "post_weight", d, index)
    post_b = 0 if post_bias is None else _feature_vec(post_bias, "post_bias", d, index)
    pre_w = 0 if pre_weight is None else _feature_vec(pre_weight, "pre_weight", d, index)
    pre_b = 0 if pre_bias is None else _feature_vec(pre_bias, "pre_bias", d, index)
    args = _PACK.pack(m, d, x_p, ldx, x_dt, part_dt, parts_p, ldp, num_parts, post, bias_p, post_w, post_b, h_p, ldh, h_dt,
                      pre, pre_w, pre_b, z_p, ldz, zs_p, ldzs, z_rows, mod_dt, gate_p, scale_p, shift_p, ld_gate,
                      ld_scale, ld_shift, groups, group_rows or 0, index_p, residual_scale, eps)
    _call(lib.tp_block_norm, x, stream, args)   # part_array, which args points to, lives until here
    return h, z
