// gemm_fp8.hip -- Y = epilogue(X . W^T) on quantized rows (e4m3 codes, e8m0 scale per 128 features).
//
//   y[m, n] = sum_b 2^(sx[m,b] + sw[n,b]) sum_{k in block b} x[m,k] w[n,k]
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 covers 16 rows of each operand and one scale block of
// 128 features, and multiplies the products by both rows' scales inside the matrix core: each
// lane passes the scale byte of the operand row that it holds.
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float gelu_tanh(float v)
{
    const float a = -2.0f * 0.7978845608028654f * 1.4426950408889634f;
    const float b = 0.044715f * a;
    const float e = __builtin_amdgcn_exp2f(v * __builtin_fmaf(b, v * v, a));
    return v * __builtin_amdgcn_rcpf(1.0f + e);
}

__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// One wave per 16 x 16 outputs (and the matching up rows): operands straight from memory.
__global__ __launch_bounds__(256) void gemm_fp8_kernel(Fp8Problem p)
{
    const int lane = threadIdx.x & 63;
    const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t tn = p.N / 16, tm = (p.M + 15) / 16;
    if (tile >= tn * tm)
        return;
    const int64_t n0 = tile % tn * 16, m0 = tile / tn * 16;
    const int64_t xr = min(m0 + (lane & 15), p.M - 1), wr = n0 + (lane & 15);
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    const int halves = p.swiglu ? 2 : 1;
    for (int64_t b = 0; b < p.K / kQBlock; ++b) {
        const int64_t k = b * kQBlock + 32 * (lane >> 4);
        const i32x8 fx = *(const i32x8 *)(p.x + xr * p.ldx + k);
        const int sx = p.xs[xr * p.ldxs + b];
        for (int h = 0; h < halves; ++h) {
            const i32x8 fw = *(const i32x8 *)(p.w + (wr + h * p.N) * p.ldw + k);
            const int sw = p.ws[(wr + h * p.N) * p.ldws + b];
            acc[h] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fx, acc[h], 0, 0, 0, sw, 0, sx);
        }
    }
    const int64_t m = m0 + (lane & 15), n = n0 + 4 * (lane >> 4);
    if (m >= p.M)
        return;
    for (int i = 0; i < 4; ++i) {
        float v = acc[0][i], u = acc[1][i];
        if (p.bias) {
            v += (float)((const __bf16 *)p.bias)[n + i];
            if (p.swiglu)
                u += (float)((const __bf16 *)p.bias)[p.N + n + i];
        }
        v = p.gelu ? gelu_tanh(v) : (p.swiglu ? silu(v) * u : v);
        if (p.out_bf16)
            ((__bf16 *)p.y)[m * p.ldy + n + i] = (__bf16)v;
        else
            ((float *)p.y)[m * p.ldy + n + i] = v;
    }
}

}  // namespace

hipError_t launch_gemm_fp8(const Fp8Problem &p, hipStream_t stream)
{
    if (p.out_bf16 && p.M > 128)
        return launch_gemm_fp8_tiled(p, stream);
    const int64_t tiles = p.N / 16 * ((p.M + 15) / 16);
    hipLaunchKernelGGL(gemm_fp8_kernel, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace tpl
