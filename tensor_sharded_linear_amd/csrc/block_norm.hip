// block_norm.hip -- the boundary between two blocks: sum of partials and bias, norm after the
// block, gate and residual, norm before the next block, modulation, quantization.
//
//   y = ((p_0 + p_1) + ...) + b,   h = r x + g * post(y),   z = pre(h) (1 + s) + t
//
// HBM-bound: each row is read once, kept in registers through both norms, and h and z are
// written once.  A row belongs to one workgroup of 1 to 16 waves; a lane owns U units of 8
// consecutive features (16 bytes of bf16), so a 128-feature scale block of a quantized z is 16
// neighbouring lanes.  The variance is taken about the mean from the registers (two passes over
// registers, none over memory), so it does not cancel.  All sums are fp32: partial sums of a lane,
// then lanes of a wave by DPP and swizzle, then waves through LDS in wave order, the same
// order on every call.
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxWaves = 16;

struct NormParams {
    int64_t row0;  // first row of this launch
    int D, D8;  // features, and rounded up to what is written of a row (to 128 for codes)
    const void *x;
    const void *parts[kMaxParts];
    int num_parts;
    const uint16_t *bias, *post_w, *post_b, *pre_w, *pre_b;
    void *h, *z;
    uint8_t *z_scale;
    const void *gate, *scale, *shift;
    const int32_t *index;
    int64_t ldx, ld_part, ldh, ldz, ldzs, ld_gate, ld_scale, ld_shift, groups, group_rows;
    int post, pre, z_rows;
    bool x_f32, part_f32, h_f32, mod_f32;
    float residual, eps;
};

// Eight features at column c of a row that starts at element `row` of t.  VEC: rows start at
// 16-byte addresses, so whole units are one or two 16-byte loads.  Features past D are 0.
template <bool VEC>
__device__ __forceinline__ void load8(const void *t, bool f32, int64_t row, int c, int D, float (&v)[8])
{
    if (VEC && c + 8 <= D) {
        if (f32) {
            const f32x4 *s = (const f32x4 *)((const float *)t + row + c);
            const f32x4 a = s[0], b = s[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
            const u32x4 a = *(const u32x4 *)((const uint16_t *)t + row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0.f;
        if (c + i < D)
            v[i] = f32 ? ((const float *)t)[row + c + i]
                       : __uint_as_float((uint32_t)((const uint16_t *)t)[row + c + i] << 16);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(void *t, bool f32, int64_t row, int c, int D, const float (&v)[8])
{
    if (VEC && c + 8 <= D) {
        if (f32) {
            f32x4 *d = (f32x4 *)((float *)t + row + c);
            d[0] = f32x4{v[0], v[1], v[2], v[3]};
            d[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            bf16x8 b;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[i] = (__bf16)v[i];
            *(bf16x8 *)((uint16_t *)t + row + c) = b;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < D) {
            if (f32)
                ((float *)t)[row + c + i] = v[i];
            else
                ((__bf16 *)t)[row + c + i] = (__bf16)v[i];
        }
}

// Sum over the workgroup, the same value in every lane.  `slot` is this call's own LDS row, so
// one barrier per call suffices.
__device__ __forceinline__ float group_sum(float v, float *slot)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
        v += __shfl_xor(v, o, 64);
    const int waves = blockDim.x >> 6;
    if (waves == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
    for (int w = 1; w < waves; ++w)
        v += slot[w];
    return v;
}

template <int U, bool VEC>
__device__ __forceinline__ void normalise(float (&v)[U][8], const NormParams &p, int kind, const uint16_t *w,
                                          const uint16_t *b, float *slots)
{
    const float inv = 1.0f / (float)p.D;
    float mean = 0.f;
    if (kind == TP_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s += v[u][i];
        mean = group_sum(s, slots) * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = 8 * ((int)threadIdx.x + u * (int)blockDim.x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[u][i] = c + i < p.D ? v[u][i] - mean : 0.f;
            q += v[u][i] * v[u][i];
        }
    }
    const float r = 1.0f / sqrtf(group_sum(q, slots + kMaxWaves) * inv + p.eps);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = 8 * ((int)threadIdx.x + u * (int)blockDim.x);
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[u][i] *= r;
        if (w) {
            load8<VEC>(w, false, 0, c, p.D, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] *= g[i];
        }
        if (b) {
            load8<VEC>(b, false, 0, c, p.D, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] += g[i];
        }
    }
}

template <int U, bool VEC>
__global__ __launch_bounds__(1024) void block_norm_kernel(NormParams p)
{
    __shared__ float slots[4 * kMaxWaves];
    const int64_t row = p.row0 + blockIdx.x;
    const int64_t group = p.index ? (int64_t)p.index[row] : row / p.group_rows;
    const bool modulated = group >= 0 && group < p.groups;
    float h[U][8], t[8];
#pragma unroll
    for (int u = 0; u < U; ++u)
        load8<VEC>(p.x, p.x_f32, row * p.ldx, 8 * ((int)threadIdx.x + u * (int)blockDim.x), p.D, h[u]);
    if (p.num_parts) {
        float y[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = 8 * ((int)threadIdx.x + u * (int)blockDim.x);
            load8<VEC>(p.parts[0], p.part_f32, row * p.ld_part, c, p.D, y[u]);
            for (int q = 1; q < p.num_parts; ++q) {
                load8<VEC>(p.parts[q], p.part_f32, row * p.ld_part, c, p.D, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[u][i] += t[i];
            }
            if (p.bias) {
                load8<VEC>(p.bias, false, 0, c, p.D, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[u][i] += t[i];
            }
        }
        if (p.post != TP_NORM_NONE)
            normalise<U, VEC>(y, p, p.post, p.post_w, p.post_b, slots);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = 8 * ((int)threadIdx.x + u * (int)blockDim.x);
            if (p.gate && modulated) {
                load8<VEC>(p.gate, p.mod_f32, group * p.ld_gate, c, p.D, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[u][i] *= t[i];
            }
            const bool branch = !p.gate || modulated;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[u][i] = p.residual * h[u][i] + (branch ? y[u][i] : 0.f);
            store8<VEC>(p.h, p.h_f32, row * p.ldh, c, p.D, h[u]);
        }
    }
    if (p.pre == TP_NORM_NONE)
        return;
    normalise<U, VEC>(h, p, p.pre, p.pre_w, p.pre_b, slots + 2 * kMaxWaves);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = 8 * ((int)threadIdx.x + u * (int)blockDim.x);
        if (p.scale && modulated) {
            load8<VEC>(p.scale, p.mod_f32, group * p.ld_scale, c, p.D, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[u][i] *= 1.0f + t[i];
        }
        if (p.shift && modulated) {
            load8<VEC>(p.shift, p.mod_f32, group * p.ld_shift, c, p.D, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[u][i] += t[i];
        }
        if (p.z_rows != TP_ROWS_FP8) {
            store8<VEC>(p.z, p.z_rows == TP_ROWS_F32, row * p.ldz, c, p.D, h[u]);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[u][i] = c + i < p.D ? h[u][i] : 0.f;
                m = max(m, __float_as_uint(h[u][i]) & 0x7fffffffu);
            }
            const int s = scale_byte(row16_max(m));
            if (c < p.D8) {
                *(uint2 *)((uint8_t *)p.z + row * p.ldz + c) = quantize8(h[u], s);
                if ((threadIdx.x & 15) == 0)
                    p.z_scale[row * p.ldzs + c / kQBlock] = (uint8_t)s;
            }
        }
    }
}

// One workgroup per row; rows beyond what one launch's thread count (below 2^32) can hold go
// into further launches.
constexpr int64_t kRowsPerLaunch = (int64_t)1 << 21;

template <int U>
void launch_u(NormParams p, int64_t M, bool vec, int waves, hipStream_t stream)
{
    const dim3 block(64 * waves);
    for (p.row0 = 0; p.row0 < M; p.row0 += kRowsPerLaunch) {
        const dim3 grid((unsigned)(M - p.row0 < kRowsPerLaunch ? M - p.row0 : kRowsPerLaunch));
        if (vec)
            hipLaunchKernelGGL((block_norm_kernel<U, true>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((block_norm_kernel<U, false>), grid, block, 0, stream, p);
    }
}

}  // namespace

hipError_t launch_block_norm(const tp_block_norm_args &a, hipStream_t stream)
{
    NormParams p{};
    p.D = (int)a.D;
    p.D8 = a.z_rows == TP_ROWS_FP8 && a.z ? (int)((a.D + kQBlock - 1) / kQBlock * kQBlock) : p.D;
    p.x = a.x;
    p.num_parts = a.num_parts;
    bool vec = true;
    const auto rows = [&](const void *t, int64_t ld, int es) {
        vec = vec && (uintptr_t)t % 16 == 0 && ld * es % 16 == 0;
    };
    for (int i = 0; i < a.num_parts; ++i) {
        p.parts[i] = a.parts[i];
        rows(a.parts[i], a.ld_part, a.part_dtype == TP_F32 ? 4 : 2);
    }
    rows(a.x, a.ldx, a.x_dtype == TP_F32 ? 4 : 2);
    for (const void *v : {a.bias, a.post_weight, a.post_bias, a.pre_weight, a.pre_bias})
        rows(v, 0, 2);
    if (a.num_parts)
        rows(a.h, a.ldh, a.h_dtype == TP_F32 ? 4 : 2);
    if (a.z && a.z_rows != TP_ROWS_FP8)
        rows(a.z, a.ldz, a.z_rows == TP_ROWS_F32 ? 4 : 2);
    const int ms = a.mod_dtype == TP_F32 ? 4 : 2;
    if (a.gate)
        rows(a.gate, a.ld_gate, ms);
    if (a.scale)
        rows(a.scale, a.ld_scale, ms);
    if (a.shift)
        rows(a.shift, a.ld_shift, ms);
    p.bias = (const uint16_t *)a.bias;
    p.post_w = (const uint16_t *)a.post_weight;
    p.post_b = (const uint16_t *)a.post_bias;
    p.pre_w = (const uint16_t *)a.pre_weight;
    p.pre_b = (const uint16_t *)a.pre_bias;
    p.h = a.h;
    p.z = a.z;
    p.z_scale = (uint8_t *)a.z_scale;
    p.gate = a.gate;
    p.scale = a.scale;
    p.shift = a.shift;
    p.index = a.group_index;
    p.ldx = a.ldx;
    p.ld_part = a.ld_part;
    p.ldh = a.ldh;
    p.ldz = a.ldz;
    p.ldzs = a.ldzs;
    p.ld_gate = a.ld_gate;
    p.ld_scale = a.ld_scale;
    p.ld_shift = a.ld_shift;
    p.groups = a.gate || a.scale || a.shift ? a.groups : 0;
    p.group_rows = a.group_rows > 0 ? a.group_rows : 1;
    p.post = a.post_norm;
    p.pre = a.pre_norm;
    p.z_rows = a.z_rows;
    p.x_f32 = a.x_dtype == TP_F32;
    p.part_f32 = a.part_dtype == TP_F32;
    p.h_f32 = a.h_dtype == TP_F32;
    p.mod_f32 = a.mod_dtype == TP_F32;
    p.residual = a.residual_scale;
    p.eps = a.eps;
    // Units of 8 features per row; the fewest waves that hold a row in at most 4 units a lane.
    const int units = (p.D8 + 7) / 8;
    int waves = 1;
    while (waves < kMaxWaves && units > 4 * 64 * waves)
        waves *= 2;
    switch ((units + 64 * waves - 1) / (64 * waves)) {
    case 1: launch_u<1>(p, a.M, vec, waves, stream); break;
    case 2: launch_u<2>(p, a.M, vec, waves, stream); break;
    case 3: launch_u<3>(p, a.M, vec, waves, stream); break;
    default: launch_u<4>(p, a.M, vec, waves, stream); break;
    }
    return hipGetLastError();
}

}  // namespace tpl
