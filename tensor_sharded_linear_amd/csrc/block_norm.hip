// block_norm.hip -- the boundary between two blocks: sum of partials and bias, norm after the
// block, gate and residual, norm before the next block, modulation, quantization.
//
//   y = ((p_0 + p_1) + ...) + b,   h = r x + g * post(y),   z = pre(h) (1 + s) + t
//
// HBM-bound: each row is read once, kept in registers through both norms, and h and z are
// written once.  4608 x 6144 with four fp32 partials, bias, gate, modulation and quantized z takes
// 113 us: 5.3 TB/s of 595 MB, where a large copy reaches 5.05 TB/s.  A row belongs to one workgroup of
// 1 to 16 waves; a lane owns U units of 8 consecutive features (16 bytes of bf16), so a
// 128-feature scale block of a quantized z is 16 neighbouring lanes.  The variance is taken about
// the mean from the registers (two passes over registers, none over memory), so it does not cancel.
// All sums are fp32: partial sums of a lane, then lanes of a wave by DPP, then waves through LDS,
// the same order on every call.
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

// Rows need only start at an element: the memory system takes wide accesses at any address.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef bf16x8 __attribute__((aligned(2))) bf16x8_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

// Eight features as they lie in memory: bf16 in a, fp32 in a and b.  The type is a uniform run-time
// flag that guards the second load only, so all loads of a row go out before the first is awaited.
struct Raw {
    u32x4 a, b;
};

template <bool TAIL>
__device__ __forceinline__ Raw load8(const void *t, bool f32, int64_t row, int c, int D)
{
    Raw r{u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
    if (c + 8 <= D) {
        const char *p = (const char *)t + (row + c) * (f32 ? 4 : 2);
        r.a = *(const u32x4_any *)p;
        if (f32)
            r.b = *(const u32x4_any *)(p + 16);
    } else if (TAIL && c < D) {  // D % 8 features, one by one
        for (int i = 0; i < D - c; ++i) {
            if (f32) {
                const uint32_t v = ((const uint32_t *)t)[row + c + i];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    r.a[k] = i == k ? v : r.a[k];
                    r.b[k] = i == 4 + k ? v : r.b[k];
                }
            } else {
                const uint32_t v = (uint32_t)((const uint16_t *)t)[row + c + i] << (16 * (i & 1));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    r.a[k] |= i / 2 == k ? v : 0;
            }
        }
    }
    return r;
}

__device__ __forceinline__ void widen(const Raw &r, bool f32, float (&v)[8])
{
    if (f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(r.a[i]);
            v[4 + i] = __uint_as_float(r.b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r.a[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.a[i] & 0xffff0000u);
        }
    }
}

template <bool TAIL>
__device__ __forceinline__ void store8(void *t, bool f32, int64_t row, int c, int D, const float (&v)[8])
{
    if (c + 8 <= D) {
        if (f32) {
            float *d = (float *)t + row + c;
            *(f32x4_any *)d = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4_any *)(d + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            bf16x8 b;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[i] = (__bf16)v[i];
            *(bf16x8_any *)((uint16_t *)t + row + c) = b;
        }
    } else if (TAIL) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (c + i < D) {
                if (f32)
                    ((float *)t)[row + c + i] = v[i];
                else
                    ((__bf16 *)t)[row + c + i] = (__bf16)v[i];
            }
    }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}

// The sum over each row of 16 lanes in its lane 15.
__device__ __forceinline__ float row_sum(float v)
{
    v = dpp_add<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    return dpp_add<0x118, 0xf>(v);
}

// Sum over the workgroup, the same value in every lane: lanes of a wave by DPP, then the waves (at
// most 16) through LDS and once more by DPP.  `slot` is this call's own LDS row, so one barrier
// per call suffices.
__device__ __forceinline__ float group_sum(float v, float *slot)
{
    v = row_sum(v);
    v = dpp_add<0x142, 0xa>(v);  // row_bcast 15, 31
    v = dpp_add<0x143, 0xc>(v);
    const float wave = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
    const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
    if (waves == 1)
        return wave;
    if (lane == 0)
        slot[threadIdx.x >> 6] = wave;
    __syncthreads();
    const float w = row_sum(lane < waves ? slot[lane] : 0.f);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), 15));
}

// PRE: the weight and bias are loaded before the sums, so their latency passes beside the reductions.
template <int U, bool TAIL, bool PRE>
__device__ __forceinline__ void normalise(float (&v)[U][8], const NormParams &p, int kind, const uint16_t *w,
                                          const uint16_t *b, float *slots)
{
    const float inv = 1.0f / (float)p.D;
    Raw rw[U], rb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = 8 * ((int)threadIdx.x + u * (int)blockDim.x);
        if (PRE && w)
            rw[u] = load8<TAIL>(w, false, 0, c, p.D);
        if (PRE && b)
            rb[u] = load8<TAIL>(b, false, 0, c, p.D);
    }
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
            v[u][i] = c + (TAIL ? i : 0) < p.D ? v[u][i] - mean : 0.f;
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
            widen(PRE ? rw[u] : load8<TAIL>(w, false, 0, c, p.D), false, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] *= g[i];
        }
        if (b) {
            widen(PRE ? rb[u] : load8<TAIL>(b, false, 0, c, p.D), false, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] += g[i];
        }
    }
}

// One row per workgroup.  NP: the number of parts, or -1 for any.  TAIL: D is no multiple of 8.
// With one unit a lane everything that a row reads is loaded ahead of its use; more units leave no room
// for that in the 128 registers of a lane of 16 waves.
template <int U, int NP, bool TAIL>
__global__ __launch_bounds__(64 * kMaxWaves) void block_norm_kernel(NormParams p)
{
    constexpr bool PRE = U == 1;
    __shared__ float slots[4 * kMaxWaves];
    const int64_t row = p.row0 + blockIdx.x;
    const int parts = NP >= 0 ? NP : p.num_parts;
    const int64_t group = p.index ? (int64_t)p.index[row] : row / p.group_rows;
    const bool modulated = group >= 0 && group < p.groups;
    const auto col = [&](int u) { return 8 * ((int)threadIdx.x + u * (int)blockDim.x); };
    float h[U][8], t[8];
    Raw rx[U];
    if (PRE || NP == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            rx[u] = load8<TAIL>(p.x, p.x_f32, row * p.ldx, col(u), p.D);
    }
    if (NP != 0) {
        float y[U][8];
        constexpr int kAtOnce = NP > 0 ? NP : 1;
        Raw rp[kAtOnce][U];
        Raw rbias[U], rgate[U];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
            for (int u = 0; u < U; ++u)
                rp[q][u] = load8<TAIL>(p.parts[q], p.part_f32, row * p.ld_part, col(u), p.D);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (PRE && p.bias)
                rbias[u] = load8<TAIL>(p.bias, false, 0, col(u), p.D);
            if (PRE && p.gate && modulated)
                rgate[u] = load8<TAIL>(p.gate, p.mod_f32, group * p.ld_gate, col(u), p.D);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            widen(rp[0][u], p.part_f32, y[u]);
        if (NP > 0) {
#pragma unroll
            for (int q = 1; q < kAtOnce; ++q)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    widen(rp[q][u], p.part_f32, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[u][i] += t[i];
                }
        } else {
            for (int q = 1; q < parts; ++q) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    rp[0][u] = load8<TAIL>(p.parts[q], p.part_f32, row * p.ld_part, col(u), p.D);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    widen(rp[0][u], p.part_f32, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[u][i] += t[i];
                }
            }
        }
        if (p.bias) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                widen(PRE ? rbias[u] : load8<TAIL>(p.bias, false, 0, col(u), p.D), false, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[u][i] += t[i];
            }
        }
        if (p.post != TP_NORM_NONE)
            normalise<U, TAIL, PRE>(y, p, p.post, p.post_w, p.post_b, slots);
        const bool branch = !p.gate || modulated;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p.gate && modulated) {
                widen(PRE ? rgate[u] : load8<TAIL>(p.gate, p.mod_f32, group * p.ld_gate, col(u), p.D), p.mod_f32, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[u][i] *= t[i];
            }
            widen(PRE ? rx[u] : load8<TAIL>(p.x, p.x_f32, row * p.ldx, col(u), p.D), p.x_f32, h[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[u][i] = p.residual * h[u][i] + (branch ? y[u][i] : 0.f);
            store8<TAIL>(p.h, p.h_f32, row * p.ldh, col(u), p.D, h[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
            widen(rx[u], p.x_f32, h[u]);
    }
    if (p.pre == TP_NORM_NONE)
        return;
    const bool scaled = p.scale && modulated, shifted = p.shift && modulated;
    Raw rs[U], rt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (PRE && scaled)
            rs[u] = load8<TAIL>(p.scale, p.mod_f32, group * p.ld_scale, col(u), p.D);
        if (PRE && shifted)
            rt[u] = load8<TAIL>(p.shift, p.mod_f32, group * p.ld_shift, col(u), p.D);
    }
    normalise<U, TAIL, PRE>(h, p, p.pre, p.pre_w, p.pre_b, slots + 2 * kMaxWaves);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = col(u);
        if (scaled) {
            widen(PRE ? rs[u] : load8<TAIL>(p.scale, p.mod_f32, group * p.ld_scale, c, p.D), p.mod_f32, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[u][i] *= 1.0f + t[i];
        }
        if (shifted) {
            widen(PRE ? rt[u] : load8<TAIL>(p.shift, p.mod_f32, group * p.ld_shift, c, p.D), p.mod_f32, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[u][i] += t[i];
        }
        if (p.z_rows != TP_ROWS_FP8) {
            store8<TAIL>(p.z, p.z_rows == TP_ROWS_F32, row * p.ldz, c, p.D, h[u]);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[u][i] = c + (TAIL ? i : 0) < p.D ? h[u][i] : 0.f;
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

typedef void (*NormKernel)(NormParams);

// One unit a lane: everything ahead; the common part counts unrolled.
NormKernel eager_kernel(int parts, bool tail)
{
    if (tail)
        return parts == 0 ? block_norm_kernel<1, 0, true> : block_norm_kernel<1, -1, true>;
    switch (parts) {
    case 0: return block_norm_kernel<1, 0, false>;
    case 1: return block_norm_kernel<1, 1, false>;
    case 2: return block_norm_kernel<1, 2, false>;
    case 4: return block_norm_kernel<1, 4, false>;
    default: return block_norm_kernel<1, -1, false>;
    }
}

template <int U>
NormKernel lean_kernel(int parts, bool tail)
{
    if (tail)
        return parts == 0 ? block_norm_kernel<U, 0, true> : block_norm_kernel<U, -1, true>;
    return parts == 0 ? block_norm_kernel<U, 0, false> : block_norm_kernel<U, -1, false>;
}

}  // namespace

hipError_t launch_block_norm(const tp_block_norm_args &a, hipStream_t stream)
{
    NormParams p{};
    p.D = (int)a.D;
    p.D8 = a.z_rows == TP_ROWS_FP8 && a.z ? (int)((a.D + kQBlock - 1) / kQBlock * kQBlock) : p.D;
    p.x = a.x;
    p.num_parts = a.num_parts;
    for (int i = 0; i < a.num_parts; ++i)
        p.parts[i] = a.parts[i];
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
    // Units of 8 features per lane, and waves per row.  One unit and as many waves as that takes is the
    // fastest almost everywhere: the loads of many short waves overlap best (4608 x 6144, four parts,
    // quantized z: 112 us against 119, 123 and 132 with two to four units; 7 rows of 6144: 4.0 us
    // against 4.5 to 5.1).  Many long rows of at most one part do better with two (1024 x 6144: 18.5
    // us against 21.2), and beyond 16 waves there is no choice.
    const int units = (p.D8 + 7) / 8;
    const auto waves_of = [&](int u) { return (units + 64 * u - 1) / (64 * u); };
    int u = a.num_parts <= 1 && waves_of(1) > 8 && a.M > 2 * cu_count() ? 2 : 1;
    while (waves_of(u) > kMaxWaves)
        ++u;
    const int waves = waves_of(u);
    const bool tail = p.D % 8 != 0;
    const NormKernel kernel = u == 1   ? eager_kernel(p.num_parts, tail)
                              : u == 2 ? lean_kernel<2>(p.num_parts, tail)
                              : u == 3 ? lean_kernel<3>(p.num_parts, tail)
                                       : lean_kernel<4>(p.num_parts, tail);
    for (p.row0 = 0; p.row0 < a.M; p.row0 += kRowsPerLaunch) {
        const dim3 grid((unsigned)(a.M - p.row0 < kRowsPerLaunch ? a.M - p.row0 : kRowsPerLaunch));
        hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace tpl
