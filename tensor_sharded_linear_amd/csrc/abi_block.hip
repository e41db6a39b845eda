// abi_block.hip -- the extern "C" entry points of include/tp_block.h: quantized rows, their
// products, and the block boundary.  Every argument is checked before any HIP call; nothing is
// allocated and no state is kept between calls.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "tp_block_internal.h"

namespace {

__attribute__((format(printf, 2, 3))) tp_status fail(tp_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(tpl::last_error_buffer(), tpl::kLastErrorBytes, fmt, ap);
    va_end(ap);
    return s;
}

tp_status hip_status(hipError_t e, const char *what)
{
    if (e == hipSuccess)
        return TP_OK;
    return fail(TP_ERR_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool is_dtype(int d) { return d == TP_BF16 || d == TP_F32; }
int size_of(int d) { return d == TP_F32 ? 4 : 2; }

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxLd = (int64_t)1 << 31;
constexpr int64_t kMaxOperandBytes = (int64_t)1 << 31;
constexpr int64_t kMaxTiles = (int64_t)1 << 22;

int64_t blocks_of(int64_t k) { return (k + tpl::kQBlock - 1) / tpl::kQBlock; }

// Codes and scales that are written: [M, kb * 128] and [M, kb].
tp_status check_codes(const char *fn, const void *codes, int64_t ldc, const void *scales, int64_t lds, int64_t kb)
{
    if (ldc > kMaxLd || lds > kMaxLd)
        return fail(TP_ERR_UNSUPPORTED, "%s: row strides above 2^31 are not supported", fn);
    if (!codes || !aligned(codes, 16) || ldc < kb * tpl::kQBlock || ldc % 16 != 0)
        return fail(TP_ERR_INVALID_ARG,
                    "%s: codes must be 16-byte aligned, their row stride %lld a multiple of 16 and >= %lld", fn,
                    (long long)ldc, (long long)(kb * tpl::kQBlock));
    if (!scales || !aligned(scales, 4) || lds < kb || lds % 4 != 0)
        return fail(TP_ERR_INVALID_ARG,
                    "%s: scales must be 4-byte aligned, their row stride %lld a multiple of 4 and >= %lld", fn,
                    (long long)lds, (long long)kb);
    return TP_OK;
}

tp_status check_fp8(const char *fn, const tpl::Fp8Problem &p, int y_es)
{
    const int64_t rows = p.swiglu ? 2 * p.N : p.N;
    if (p.M < 0 || p.N <= 0 || p.K <= 0)
        return fail(TP_ERR_INVALID_ARG, "%s: need M >= 0, N > 0, K > 0 (got M=%lld N=%lld K=%lld)", fn,
                    (long long)p.M, (long long)p.N, (long long)p.K);
    if (p.M > kMaxDim || p.N > kMaxDim || p.K > kMaxDim)
        return fail(TP_ERR_UNSUPPORTED, "%s: dimensions above 2^30 are not supported", fn);
    if (p.ldx > kMaxLd || p.ldw > kMaxLd || p.ldy > kMaxLd || p.ldxs > kMaxLd || p.ldws > kMaxLd)
        return fail(TP_ERR_UNSUPPORTED, "%s: row strides above 2^31 are not supported", fn);
    if (p.K % tpl::kQBlock != 0)
        return fail(TP_ERR_UNSUPPORTED, "%s: K=%lld must be a multiple of 128", fn, (long long)p.K);
    if (p.N % 16 != 0)
        return fail(TP_ERR_UNSUPPORTED, "%s: N=%lld must be a multiple of 16", fn, (long long)p.N);
    if (p.ldx < p.K || p.ldx % 16 != 0 || p.ldw < p.K || p.ldw % 16 != 0)
        return fail(TP_ERR_INVALID_ARG, "%s: ldx=%lld and ldw=%lld must be >= K=%lld and multiples of 16", fn,
                    (long long)p.ldx, (long long)p.ldw, (long long)p.K);
    const int64_t kb = p.K / tpl::kQBlock;
    if (p.ldxs < kb || p.ldxs % 4 != 0 || p.ldws < kb || p.ldws % 4 != 0)
        return fail(TP_ERR_INVALID_ARG,
                    "%s: scale row strides %lld and %lld must be >= K/128=%lld and multiples of 4", fn,
                    (long long)p.ldxs, (long long)p.ldws, (long long)kb);
    if (p.ldy < p.N || (p.ldy * y_es) % 16 != 0)
        return fail(TP_ERR_INVALID_ARG, "%s: ldy=%lld must be >= N=%lld and a multiple of 16 bytes", fn,
                    (long long)p.ldy, (long long)p.N);
    // The kernels address each operand by 32-bit byte offsets from its base.
    if ((rows - 1) * p.ldw + p.K >= kMaxOperandBytes || rows * p.ldws >= kMaxOperandBytes ||
        (p.M > 0 && ((p.M - 1) * p.ldx + p.K >= kMaxOperandBytes || p.M * p.ldxs >= kMaxOperandBytes)))
        return fail(TP_ERR_UNSUPPORTED, "%s: an operand spans 2 GiB or more", fn);
    if ((p.M + 191) / 192 * ((p.N + 255) / 256) > kMaxTiles)
        return fail(TP_ERR_UNSUPPORTED, "%s: an output of %lld x %lld needs more than 2^22 tiles", fn,
                    (long long)p.M, (long long)p.N);
    if (!p.w || !aligned(p.w, 16) || !p.ws || !aligned(p.ws, 4))
        return fail(TP_ERR_INVALID_ARG, "%s: weight codes / scales are null or not 16 / 4-byte aligned", fn);
    if (p.bias && !aligned(p.bias, 8))
        return fail(TP_ERR_INVALID_ARG, "%s: bias pointer is not 8-byte aligned", fn);
    if (p.M > 0 && (!p.x || !aligned(p.x, 16) || !p.xs || !aligned(p.xs, 4)))
        return fail(TP_ERR_INVALID_ARG, "%s: activation codes / scales are null or not 16 / 4-byte aligned", fn);
    if (p.M > 0 && (!p.y || !aligned(p.y, 16)))
        return fail(TP_ERR_INVALID_ARG, "%s: output pointer is null or not 16-byte aligned", fn);
    return TP_OK;
}

tp_status run_fp8(const char *fn, const tpl::Fp8Problem &p, int y_es, hipStream_t stream)
{
    const tp_status s = check_fp8(fn, p, y_es);
    if (s != TP_OK || p.M == 0)
        return s;
    return hip_status(tpl::launch_gemm_fp8(p, stream), fn);
}

bool is_norm(int k) { return k == TP_NORM_NONE || k == TP_NORM_LAYER || k == TP_NORM_RMS; }

}  // namespace

extern "C" {

tp_status tp_quantize_fp8(const void *x, int64_t ldx, tp_dtype x_dtype, void *codes, int64_t ldc, void *scales,
                          int64_t lds, int64_t M, int64_t K, hipStream_t stream)
{
    const char *fn = "tp_quantize_fp8";
    tpl::last_error_buffer()[0] = 0;
    if (!is_dtype(x_dtype))
        return fail(TP_ERR_INVALID_ARG, "%s: x_dtype must be TP_BF16 or TP_F32", fn);
    if (M < 0 || K < 1)
        return fail(TP_ERR_INVALID_ARG, "%s: need M >= 0 and K >= 1 (got M=%lld K=%lld)", fn, (long long)M,
                    (long long)K);
    if (M > kMaxDim || K > kMaxDim || ldx > kMaxLd)
        return fail(TP_ERR_UNSUPPORTED, "%s: dimensions above 2^30 or strides above 2^31 are not supported", fn);
    if (ldx < K)
        return fail(TP_ERR_INVALID_ARG, "%s: ldx=%lld must be >= K=%lld", fn, (long long)ldx, (long long)K);
    if (M == 0)
        return TP_OK;
    if (!x || !aligned(x, size_of(x_dtype)))
        return fail(TP_ERR_INVALID_ARG, "%s: x is null or not aligned to its elements", fn);
    const tp_status s = check_codes(fn, codes, ldc, scales, lds, blocks_of(K));
    if (s != TP_OK)
        return s;
    const tpl::QuantProblem p{x, ldx, x_dtype == TP_F32, (uint8_t *)codes, ldc, (uint8_t *)scales, lds, M, K};
    return hip_status(tpl::launch_quantize(p, stream), fn);
}

tp_status tp_linear_colwise_fp8(const void *x, int64_t ldx, const void *x_scale, int64_t ldxs, const void *w,
                                int64_t ldw, const void *w_scale, int64_t ldws, const void *bias, void *y,
                                int64_t ldy, tp_dtype y_dtype, tp_act act, int64_t M, int64_t n_shard, int64_t K,
                                hipStream_t stream)
{
    const char *fn = "tp_linear_colwise_fp8";
    tpl::last_error_buffer()[0] = 0;
    if (!is_dtype(y_dtype))
        return fail(TP_ERR_INVALID_ARG, "%s: y_dtype must be TP_BF16 or TP_F32", fn);
    if (act != TP_ACT_NONE && act != TP_ACT_GELU_TANH && act != TP_ACT_SWIGLU)
        return fail(TP_ERR_INVALID_ARG, "%s: act must be TP_ACT_NONE, TP_ACT_GELU_TANH or TP_ACT_SWIGLU", fn);
    const tpl::Fp8Problem p{(const uint8_t *)x, (const uint8_t *)x_scale, (const uint8_t *)w,
                            (const uint8_t *)w_scale, ldx, ldxs, ldw, ldws, (const uint16_t *)bias, y, ldy, M,
                            n_shard, K, y_dtype == TP_BF16, act == TP_ACT_GELU_TANH, act == TP_ACT_SWIGLU};
    return run_fp8(fn, p, size_of(y_dtype), stream);
}

tp_status tp_linear_rowwise_fp8(const void *x, int64_t ldx, const void *x_scale, int64_t ldxs, const void *w,
                                int64_t ldw, const void *w_scale, int64_t ldws, float *partial, int64_t ldp,
                                int64_t M, int64_t N, int64_t k_shard, hipStream_t stream)
{
    const char *fn = "tp_linear_rowwise_fp8";
    tpl::last_error_buffer()[0] = 0;
    const tpl::Fp8Problem p{(const uint8_t *)x, (const uint8_t *)x_scale, (const uint8_t *)w,
                            (const uint8_t *)w_scale, ldx, ldxs, ldw, ldws, nullptr, partial, ldp, M, N, k_shard,
                            false, false, false};
    return run_fp8(fn, p, 4, stream);
}

tp_status tp_linear_fp8_tile_shape(int64_t M, int64_t N, int64_t K, tp_act act, tp_dtype y_dtype,
                                   int64_t *tile_rows, int64_t *tile_cols)
{
    const char *fn = "tp_linear_fp8_tile_shape";
    tpl::last_error_buffer()[0] = 0;
    if (!tile_rows || !tile_cols)
        return fail(TP_ERR_INVALID_ARG, "%s: tile_rows and tile_cols must be non-null", fn);
    if (act != TP_ACT_NONE && act != TP_ACT_GELU_TANH && act != TP_ACT_SWIGLU)
        return fail(TP_ERR_INVALID_ARG, "%s: act must be TP_ACT_NONE, TP_ACT_GELU_TANH or TP_ACT_SWIGLU", fn);
    if (!is_dtype(y_dtype))
        return fail(TP_ERR_INVALID_ARG, "%s: y_dtype must be TP_BF16 or TP_F32", fn);
    if (M < 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return fail(TP_ERR_INVALID_ARG, "%s: need 0 <= M, 0 < N, 0 < K, all at most 2^30", fn);
    tpl::Fp8Problem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.out_bf16 = y_dtype == TP_BF16;
    p.gelu = act == TP_ACT_GELU_TANH;
    p.swiglu = act == TP_ACT_SWIGLU;
    int rows = 0, cols = 0;
    tpl::gemm_fp8_tile_shape(p, &rows, &cols);
    *tile_rows = rows;
    *tile_cols = cols;
    return TP_OK;
}

tp_status tp_block_norm(const tp_block_norm_args *args, hipStream_t stream)
{
    const char *fn = "tp_block_norm";
    tpl::last_error_buffer()[0] = 0;
    if (!args)
        return fail(TP_ERR_INVALID_ARG, "%s: args is null", fn);
    const tp_block_norm_args &a = *args;
    if (a.M < 0 || a.D < 1)
        return fail(TP_ERR_INVALID_ARG, "%s: need M >= 0 and D >= 1 (got M=%lld D=%lld)", fn, (long long)a.M,
                    (long long)a.D);
    if (!is_dtype(a.x_dtype) || !is_dtype(a.part_dtype) || !is_dtype(a.h_dtype) || !is_dtype(a.mod_dtype))
        return fail(TP_ERR_INVALID_ARG, "%s: x, part, h and mod dtypes must be TP_BF16 or TP_F32", fn);
    if (!is_norm(a.post_norm) || !is_norm(a.pre_norm))
        return fail(TP_ERR_INVALID_ARG, "%s: post_norm and pre_norm must be TP_NORM_NONE, LAYER or RMS", fn);
    if (a.z_rows != TP_ROWS_BF16 && a.z_rows != TP_ROWS_F32 && a.z_rows != TP_ROWS_FP8)
        return fail(TP_ERR_INVALID_ARG, "%s: z_rows must be TP_ROWS_BF16, TP_ROWS_F32 or TP_ROWS_FP8", fn);
    if (a.num_parts < 0 || a.num_parts > tpl::kMaxParts)
        return fail(TP_ERR_INVALID_ARG, "%s: num_parts=%d must be in [0, %d]", fn, a.num_parts, tpl::kMaxParts);
    if (a.M > kMaxDim || a.D > tpl::kNormMaxD)
        return fail(TP_ERR_UNSUPPORTED, "%s: M above 2^30 or D above %lld is not supported", fn,
                    (long long)tpl::kNormMaxD);
    for (const int64_t ld : {a.ldx, a.ld_part, a.ldh, a.ldz, a.ldzs, a.ld_gate, a.ld_scale, a.ld_shift})
        if (ld > kMaxLd)
            return fail(TP_ERR_UNSUPPORTED, "%s: row strides above 2^31 are not supported", fn);
    if (!isfinite(a.eps) || a.eps < 0 || !isfinite(a.residual_scale))
        return fail(TP_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, residual_scale finite", fn);
    const bool branch = a.num_parts > 0, next = a.pre_norm != TP_NORM_NONE;
    if (!branch && !next)
        return fail(TP_ERR_INVALID_ARG, "%s: neither parts nor pre_norm: nothing to compute", fn);
    if (!branch && (a.h || a.bias || a.gate || a.post_norm != TP_NORM_NONE || a.residual_scale != 1.0f))
        return fail(TP_ERR_INVALID_ARG,
                    "%s: without parts, h, bias and gate must be null, post_norm NONE and residual_scale 1", fn);
    if (!next && (a.z || a.z_scale || a.scale || a.shift))
        return fail(TP_ERR_INVALID_ARG, "%s: with pre_norm NONE, z, z_scale, scale and shift must be null", fn);
    if ((a.post_norm == TP_NORM_NONE && (a.post_weight || a.post_bias)) || (!next && (a.pre_weight || a.pre_bias)))
        return fail(TP_ERR_INVALID_ARG, "%s: a norm's weight or bias without the norm", fn);
    if (a.gate || a.scale || a.shift) {
        if (a.groups < 1 || a.groups > kMaxDim)
            return fail(TP_ERR_INVALID_ARG, "%s: groups=%lld must be in [1, 2^30]", fn, (long long)a.groups);
        if (!a.group_index && (a.group_rows < 1 || a.group_rows > kMaxDim || a.groups * a.group_rows < a.M))
            return fail(TP_ERR_INVALID_ARG, "%s: %lld groups of %lld rows do not cover M=%lld rows", fn,
                        (long long)a.groups, (long long)a.group_rows, (long long)a.M);
        if (a.group_index && !aligned(a.group_index, 4))
            return fail(TP_ERR_INVALID_ARG, "%s: group_index is not 4-byte aligned", fn);
    } else if (a.group_index) {
        return fail(TP_ERR_INVALID_ARG, "%s: group_index without a gate, scale or shift", fn);
    }
    const struct { const char *name; const void *p; int64_t ld; int64_t es; bool need; } rows[] = {
        {"x", a.x, a.ldx, size_of(a.x_dtype), true},
        {"h", a.h, a.ldh, size_of(a.h_dtype), branch},
        {"z", a.z, a.ldz, a.z_rows == TP_ROWS_F32 ? 4 : 2, next && a.z_rows != TP_ROWS_FP8},
        {"gate", a.gate, a.ld_gate, size_of(a.mod_dtype), a.gate != nullptr},
        {"scale", a.scale, a.ld_scale, size_of(a.mod_dtype), a.scale != nullptr},
        {"shift", a.shift, a.ld_shift, size_of(a.mod_dtype), a.shift != nullptr}};
    for (const auto &r : rows) {
        if (!r.need)
            continue;
        if (r.ld < a.D)
            return fail(TP_ERR_INVALID_ARG, "%s: the row stride %lld of %s must be >= D=%lld", fn, (long long)r.ld,
                        r.name, (long long)a.D);
        if (a.M > 0 && (!r.p || !aligned(r.p, (uintptr_t)r.es)))
            return fail(TP_ERR_INVALID_ARG, "%s: %s is null or not aligned to its elements", fn, r.name);
    }
    for (const void *v : {a.bias, a.post_weight, a.post_bias, a.pre_weight, a.pre_bias})
        if (!aligned(v, 2))
            return fail(TP_ERR_INVALID_ARG, "%s: a weight or bias is not aligned to its elements", fn);
    if (branch) {
        if (!a.parts)
            return fail(TP_ERR_INVALID_ARG, "%s: parts is null", fn);
        if (a.ld_part < a.D)
            return fail(TP_ERR_INVALID_ARG, "%s: the row stride %lld of the parts must be >= D=%lld", fn,
                        (long long)a.ld_part, (long long)a.D);
        for (int i = 0; i < a.num_parts; ++i)
            if (a.M > 0 && (!a.parts[i] || !aligned(a.parts[i], (uintptr_t)size_of(a.part_dtype))))
                return fail(TP_ERR_INVALID_ARG, "%s: parts[%d] is null or not aligned to its elements", fn, i);
    }
    if (next && a.z_rows != TP_ROWS_FP8 && a.z_scale)
        return fail(TP_ERR_INVALID_ARG, "%s: z_scale is for TP_ROWS_FP8 only", fn);
    if (a.M == 0)
        return TP_OK;
    if (next && a.z_rows == TP_ROWS_FP8) {
        const tp_status s = check_codes(fn, a.z, a.ldz, a.z_scale, a.ldzs, blocks_of(a.D));
        if (s != TP_OK)
            return s;
    }
    return hip_status(tpl::launch_block_norm(a, stream), fn);
}

}  // extern "C"
