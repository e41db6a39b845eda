// quant_fp8.hip -- rows of bf16 or fp32 to e4m3 codes with an e8m0 scale per 128 features.
//
// For each block of 128 features of a row: a = max |x|, 2^e the least power of two with
// a <= 448 2^e, codes = e4m3(x 2^-e).  The scaling is exact (a power of two), so the one
// rounding is the conversion's.
//
// HBM-bound: a lane owns 8 features (one 16-byte load of bf16, two of fp32; one 8-byte store),
// 16 lanes a block, and the block's maximum is four DPP steps, so nothing passes through LDS.
// Blocks are numbered through all rows, so short rows fill a workgroup as well as long ones.
// 4608 x 6144 bf16 takes 15.5 us: 5.5 TB/s of the 85 MB that it reads and writes, where a large copy
// reaches 5.05 TB/s.
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Rows need only start at an element: the memory system takes wide accesses at any address.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 16;  // blocks per workgroup and step

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantProblem p, int kb, int64_t wg0, int64_t units)
{
    const int64_t first = (wg0 + blockIdx.x) * kUnits;  // uniform
    const int64_t row0 = first / kb;
    const int c = (int)(first - row0 * kb) + ((int)threadIdx.x >> 4);
    const int dr = c / kb;
    const int blk = c - dr * kb;
    const int64_t row = row0 + dr;
    if (first + (threadIdx.x >> 4) >= units)
        return;  // whole 16-lane groups
    const int64_t k = (int64_t)blk * kQBlock + 8 * (threadIdx.x & 15);
    float v[8];
    if (k + 8 <= p.K) {
        if (F32) {
            const float *src = (const float *)p.x + row * p.ldx + k;
            const u32x4 a = *(const u32x4_any *)src, b = *(const u32x4_any *)(src + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(a[i]);
                v[4 + i] = __uint_as_float(b[i]);
            }
        } else {
            const u32x4 a = *(const u32x4_any *)((const uint16_t *)p.x + row * p.ldx + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.f;
            if (k + i < p.K)
                v[i] = F32 ? ((const float *)p.x)[row * p.ldx + k + i]
                           : bf16_f32(((const uint16_t *)p.x)[row * p.ldx + k + i]);
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    const int s = scale_byte(row16_max(m));
    *(uint2 *)(p.codes + row * p.ldc + k) = quantize8(v, s);
    if ((threadIdx.x & 15) == 0)
        p.scales[row * p.lds + blk] = (uint8_t)s;
}

}  // namespace

hipError_t launch_quantize(const QuantProblem &p, hipStream_t stream)
{
    const int kb = (int)((p.K + kQBlock - 1) / kQBlock);
    const int64_t units = p.M * kb;
    const int64_t wgs = (units + kUnits - 1) / kUnits;
    const auto kernel = p.x_f32 ? quantize_kernel<true> : quantize_kernel<false>;
    // A launch holds fewer than 2^32 threads; more blocks go into further launches.
    constexpr int64_t kPerLaunch = (int64_t)1 << 23;
    for (int64_t wg0 = 0; wg0 < wgs; wg0 += kPerLaunch) {
        const dim3 grid((unsigned)(wgs - wg0 < kPerLaunch ? wgs - wg0 : kPerLaunch)), block(kThreads);
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, p, kb, wg0, units);
    }
    return hipGetLastError();
}

}  // namespace tpl
