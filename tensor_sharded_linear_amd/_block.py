"""ctypes binding of the second part of libtp_linear.so (include/tp_block.h): quantized rows,
their products, and the norm at the boundary between two blocks.

Argument marshalling only, as in ``_binding``: outputs are allocated where none is passed, and
every step of the computation runs in the HIP kernels behind the C ABI.

Quantized rows are a pair ``(codes, scales)``: codes ``[rows, K8]`` ``torch.float8_e4m3fn`` with
K8 = K rounded up to a multiple of 128 (zero codes past K), scales ``[rows, K8 / 128]``
``torch.float8_e8m0fnu`` (powers of two).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _binding as _b
from ._binding import _check, _dev2d, _ld, _ptr, _stream, _vec

BLOCK = 128
CODES = torch.float8_e4m3fn
SCALES = torch.float8_e8m0fnu

_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_ROWS = {torch.bfloat16: 0, torch.float32: 1, CODES: 2}
_DT = _b._DT


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


# Every symbol include/tp_block.h declares, with its ctypes signature.
SIGNATURES = {
    "tp_quantize_fp8": (_I, [_P, _I64, _I, _P, _I64, _P, _I64, _I64, _I64, _P]),
    "tp_linear_colwise_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I, _I, _I64, _I64, _I64, _P]),
    "tp_linear_rowwise_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P]),
    "tp_block_norm": (_I, [ctypes.POINTER(_BlockNormArgs), _P]),
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


def _call(fn, device, *args) -> None:
    """Call an entry point with `device` current (the library launches on the current device)."""
    if device.index == torch.cuda.current_device():
        _check(fn(*args))
    else:
        with torch.cuda.device(device):
            _check(fn(*args))


def _same_device(x: torch.Tensor, **others: Optional[torch.Tensor]) -> None:
    for name, t in others.items():
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, not on {x.device}")


def _empty_codes(m: int, k: int, device):
    """Codes and scales for m rows of k features; scale rows padded to whole dwords."""
    kb = -(-k // BLOCK)
    codes = torch.empty((m, kb * BLOCK), dtype=CODES, device=device)
    scales = torch.empty((m, -(-kb // 4) * 4), dtype=SCALES, device=device)
    return codes, scales[:, :kb]


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


def tp_quantize_fp8(x: torch.Tensor, *, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None, stream=None):
    """Quantize the rows of ``x`` [M, K] (bf16 or fp32, any K) to e4m3 codes with one
    power-of-two scale for each 128 features of a row.  Returns ``(codes, scales)``.

    Scale: the least 2^e, e >= -126, with max|x| <= 448 2^e (1 for an all-zero block); codes:
    x / 2^e rounded to nearest even.  A block with an infinity or a NaN becomes NaN."""
    lib = _library()
    x = _dev2d(x, "x")
    if x.dtype not in _DT:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    m, k = x.shape
    if k == 0:
        raise ValueError("x has no columns")
    if (codes is None) != (scales is None):
        raise ValueError("pass both codes and scales, or neither")
    if codes is None:
        codes, scales = _empty_codes(m, k, x.device)
    else:
        _codes(codes, scales, "output", m, -(-k // BLOCK) * BLOCK)
        _same_device(x, codes=codes, scales=scales)
    _call(lib.tp_quantize_fp8, x.device, x.data_ptr(), _ld(x), _DT[x.dtype], codes.data_ptr(), _ld(codes),
          scales.data_ptr(), _lds(scales), m, k, _stream(stream, x))
    return codes, scales


def _operands(x, x_scale, w, w_scale):
    _codes(x, x_scale, "x")
    _codes(w, w_scale, "w_shard")
    if w.shape[1] != x.shape[1]:
        raise ValueError(f"x is [M, {x.shape[1]}] but w_shard is {tuple(w.shape)}")
    _same_device(x, x_scale=x_scale, w_shard=w, w_scale=w_scale)


def tp_linear_colwise_fp8(x: torch.Tensor, x_scale: torch.Tensor, w_shard: torch.Tensor, w_scale: torch.Tensor,
                          bias: Optional[torch.Tensor] = None, *, act: str = "none",
                          out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                          stream=None) -> torch.Tensor:
    """Colwise shard of quantized rows: ``out = act(x @ w_shard.T + bias)``, fp32 accumulation.

    ``x``/``x_scale`` and ``w_shard``/``w_scale`` as :func:`tp_quantize_fp8` gives them; ``act``,
    ``bias`` and ``out`` as :func:`tp_linear_colwise` (``"swiglu"``: a packed [gate; up] shard)."""
    lib = _library()
    _operands(x, x_scale, w_shard, w_scale)
    try:
        a = {"none": _b.TP_ACT_NONE, "gelu_tanh": _b.TP_ACT_GELU_TANH, "swiglu": _b.TP_ACT_SWIGLU}[act]
    except KeyError:
        raise ValueError("act must be 'none', 'gelu_tanh' or 'swiglu'") from None
    m, k = x.shape
    rows = w_shard.shape[0]
    if a == _b.TP_ACT_SWIGLU and rows % 2:
        raise ValueError(f"a SwiGLU shard has an even number of rows [gate; up], got {rows}")
    n = rows // 2 if a == _b.TP_ACT_SWIGLU else rows
    bias = _vec(bias, "bias", rows)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
    out = _dev2d(out, "out")
    if tuple(out.shape) != (m, n) or out.dtype not in _DT:
        raise ValueError(f"out must be [{m}, {n}] bf16 or fp32")
    _same_device(x, bias=bias, out=out)
    _call(lib.tp_linear_colwise_fp8, x.device, x.data_ptr(), _ld(x), x_scale.data_ptr(), _lds(x_scale),
          w_shard.data_ptr(), _ld(w_shard), w_scale.data_ptr(), _lds(w_scale), _ptr(bias), out.data_ptr(), _ld(out),
          _DT[out.dtype], a, m, n, k, _stream(stream, x))
    return out


def tp_linear_rowwise_fp8(x_shard: torch.Tensor, x_scale: torch.Tensor, w_shard: torch.Tensor,
                          w_scale: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rowwise shard of quantized rows: fp32 partial ``out = x_shard @ w_shard.T`` (no bias)."""
    lib = _library()
    _operands(x_shard, x_scale, w_shard, w_scale)
    m, k = x_shard.shape
    n = w_shard.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x_shard.device)
    out = _dev2d(out, "out", torch.float32)
    if tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}]")
    _same_device(x_shard, out=out)
    _call(lib.tp_linear_rowwise_fp8, x_shard.device, x_shard.data_ptr(), _ld(x_shard), x_scale.data_ptr(),
          _lds(x_scale), w_shard.data_ptr(), _ld(w_shard), w_scale.data_ptr(), _lds(w_scale), out.data_ptr(), _ld(out),
          m, n, k, _stream(stream, x_shard))
    return out


def _feature_vec(t: Optional[torch.Tensor], name: str, x: torch.Tensor) -> Optional[int]:
    if t is None:
        return None
    _vec(t, name, x.shape[1])
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, not on {x.device}")
    return t.data_ptr()


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
    x = _dev2d(x, "x")
    if x.dtype not in _DT:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    m, d = x.shape
    if d == 0:
        raise ValueError("x has no columns")
    if post_norm not in _NORMS or pre_norm not in _NORMS:
        raise ValueError("post_norm and pre_norm must be 'none', 'layer' or 'rms'")
    a = _BlockNormArgs(M=m, D=d, x=x.data_ptr(), ldx=_ld(x), x_dtype=_DT[x.dtype], post_norm=_NORMS[post_norm],
                       pre_norm=_NORMS[pre_norm], residual_scale=residual_scale, eps=eps)
    h, z = x, None
    if parts is not None:
        parts = list(parts)
        if not parts:
            raise ValueError("no parts (pass None for a norm without a block's output)")
        p0 = _dev2d(parts[0], "parts[0]")
        ldp = _ld(p0)
        if p0.dtype not in _DT:
            raise TypeError(f"parts must be bf16 or fp32, got {p0.dtype}")
        for i, p in enumerate(parts):
            _dev2d(p, f"parts[{i}]", p0.dtype)
            if tuple(p.shape) != (m, d) or _ld(p) != ldp:
                raise ValueError(f"all parts must be [{m}, {d}] with one row stride")
            if p.device != x.device:
                raise ValueError(f"parts[{i}] is on {p.device}, not on {x.device}")
        h = h_out if h_out is not None else torch.empty((m, d), dtype=x.dtype, device=x.device)
        _dev2d(h, "h_out")
        if tuple(h.shape) != (m, d) or h.dtype not in _DT:
            raise ValueError(f"h_out must be [{m}, {d}] bf16 or fp32")
        a.parts = (_P * len(parts))(*[p.data_ptr() for p in parts])
        a.num_parts, a.ld_part, a.part_dtype = len(parts), ldp, _DT[p0.dtype]
        a.h, a.ldh, a.h_dtype = h.data_ptr(), _ld(h), _DT[h.dtype]
    elif h_out is not None:
        raise ValueError("h_out without parts")
    if pre_norm == "none":
        if z_out is not None:
            raise ValueError("z_out without pre_norm")
    elif z_dtype == CODES:
        z = z_out if z_out is not None else _empty_codes(m, d, x.device)
        codes, scales = z
        _codes(codes, scales, "z_out", m, -(-d // BLOCK) * BLOCK)
        _same_device(x, z_codes=codes, z_scales=scales)
        a.z, a.ldz, a.z_scale, a.ldzs = codes.data_ptr(), _ld(codes), scales.data_ptr(), _lds(scales)
        a.z_rows = _ROWS[CODES]
    else:
        if z_dtype not in _ROWS:
            raise ValueError("z_dtype must be bf16, fp32 or float8_e4m3fn")
        z = z_out if z_out is not None else torch.empty((m, d), dtype=z_dtype, device=x.device)
        _dev2d(z, "z_out", z_dtype)
        if tuple(z.shape) != (m, d):
            raise ValueError(f"z_out must be [{m}, {d}]")
        a.z, a.ldz, a.z_rows = z.data_ptr(), _ld(z), _ROWS[z_dtype]
    a.bias = _feature_vec(bias, "bias", x)
    a.post_weight, a.post_bias = _feature_vec(post_weight, "post_weight", x), _feature_vec(post_bias, "post_bias", x)
    a.pre_weight, a.pre_bias = _feature_vec(pre_weight, "pre_weight", x), _feature_vec(pre_bias, "pre_bias", x)
    tables = {}
    for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
        if t is None:
            continue
        t = _dev2d(t.unsqueeze(0) if isinstance(t, torch.Tensor) and t.dim() == 1 else t, name)
        if t.shape[1] != d or t.dtype not in _DT:
            raise ValueError(f"{name} must be [groups, {d}] bf16 or fp32")
        tables[name] = t
        setattr(a, name, t.data_ptr())
        setattr(a, "ld_" + name, _ld(t))
    if tables:
        t0 = next(iter(tables.values()))
        if any(t.dtype != t0.dtype or t.shape[0] != t0.shape[0] for t in tables.values()):
            raise ValueError("gate, scale and shift must have one dtype and one number of groups")
        a.mod_dtype, a.groups = _DT[t0.dtype], t0.shape[0]
        if group_index is not None:
            if group_rows is not None:
                raise ValueError("pass group_rows or group_index, not both")
            if not group_index.is_cuda or group_index.dtype != torch.int32 or tuple(group_index.shape) != (m,) or \
                    (m > 1 and group_index.stride(0) != 1):
                raise ValueError(f"group_index must be a contiguous int32 GPU vector of length {m}")
            a.group_index = group_index.data_ptr()
        else:
            if group_rows is None:
                if a.groups == 0 or m % a.groups:
                    raise ValueError(f"{a.groups} groups do not divide {m} rows: pass group_rows or group_index")
                group_rows = max(1, m // a.groups)
            a.group_rows = group_rows
    elif group_index is not None:
        raise ValueError("group_index without a gate, scale or shift")
    _same_device(x, h_out=h, group_index=group_index, **tables)
    _call(lib.tp_block_norm, x.device, ctypes.byref(a), _stream(stream, x))
    return h, z
