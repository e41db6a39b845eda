// tp_block_internal.h -- declarations shared by the kernels behind include/tp_block.h.
#pragma once

#include "tp_block.h"
#include "tp_internal.h"

namespace tpl {

// ---- quantized rows ------------------------------------------------------------------
constexpr int kQBlock = 128;   // features per scale

// Scale byte of a block from the bits of its largest |x| (integer maximum of the sign-less
// bits, so an infinity or a NaN wins): amax = 1.m 2^x, and 448 = 1.75 2^8, so the least e with
// amax <= 448 2^e is x - 8, or x - 7 where 1.m > 1.75.  Kept at or above 1 (e >= -126), so the
// reciprocal 2^-e below is a normal number; 127 (scale 1) for zero, 255 (NaN) for non-finite.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits)
{
    const int ex = (int)(amax_bits >> 23);
    int s = ex - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    s = s < 1 ? 1 : s;
    s = amax_bits == 0 ? 127 : s;
    return ex == 255 ? 255 : s;
}

// 2^-(s - 127) for a finite scale byte (1 .. 247).
__device__ __forceinline__ float scale_inverse(int s) { return __uint_as_float((uint32_t)(254 - s) << 23); }

// Maximum over the 16 lanes of a DPP row (one 128-feature block at 8 features per lane).
__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    const auto rot = [](uint32_t a, auto N) {
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x120 + decltype(N)::value, 0xf, 0xf, false);
    };
    struct N8 { enum { value = 8 }; };
    struct N4 { enum { value = 4 }; };
    struct N2 { enum { value = 2 }; };
    struct N1 { enum { value = 1 }; };
    v = max(v, rot(v, N8{}));
    v = max(v, rot(v, N4{}));
    v = max(v, rot(v, N2{}));
    return max(v, rot(v, N1{}));
}

// Eight features of a block to codes: one conversion instruction per pair, nearest even.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], int s)
{
    if (s == 255)
        return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    const float r = scale_inverse(s);
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * r, v[1] * r, 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * r, v[3] * r, a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * r, v[5] * r, 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * r, v[7] * r, b, true);
    return make_uint2((uint32_t)a, (uint32_t)b);
}

struct QuantProblem {
    const void *x;
    int64_t ldx;
    bool x_f32;
    uint8_t *codes;
    int64_t ldc;
    uint8_t *scales;
    int64_t lds;
    int64_t M, K;
};
hipError_t launch_quantize(const QuantProblem &p, hipStream_t stream);

// ---- products of quantized rows --------------------------------------------------------
// Y = epilogue(X . W^T), X [M, K], W [N, K] (2 N rows [gate; up] with swiglu), K % 128 == 0.
struct Fp8Problem {
    const uint8_t *x, *xs, *w, *ws;
    int64_t ldx, ldxs, ldw, ldws;
    const uint16_t *bias;
    void *y;
    int64_t ldy;
    int64_t M, N, K;
    bool out_bf16, gelu, swiglu;
};
hipError_t launch_gemm_fp8(const Fp8Problem &p, hipStream_t stream);
void gemm_fp8_tile_shape(const Fp8Problem &p, int *rows, int *cols);

// Up to this many rows the kernel for few rows runs.
constexpr int64_t kFp8NarrowMaxM = 96;
hipError_t launch_gemm_fp8_narrow(const Fp8Problem &p, hipStream_t stream);
bool gemm_fp8_narrow_takes(const Fp8Problem &p);
void gemm_fp8_narrow_shape(const Fp8Problem &p, int *rows, int *cols);  // of a workgroup
// Four-wave tiles of 32 nxb x 32 nwb; eight-wave tiles of 32 nxb x 128.
hipError_t launch_gemm_fp8_tiled(const Fp8Problem &p, int nxb, int nwb, hipStream_t stream);
hipError_t launch_gemm_fp8_small(const Fp8Problem &p, int nxb, hipStream_t stream);

// ---- block boundary ---------------------------------------------------------------------
constexpr int64_t kNormMaxD = 32768;
hipError_t launch_block_norm(const tp_block_norm_args &a, hipStream_t stream);

}  // namespace tpl
