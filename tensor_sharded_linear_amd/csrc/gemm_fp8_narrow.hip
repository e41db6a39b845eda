// gemm_fp8_narrow.hip -- product of quantized rows for few rows or few outputs: split-K, exact products.
//
// With few rows the weight stream sets the time: 9216 x 6144 codes and their scales are 57 MB, 7 us at
// 8 TB/s.  So a workgroup of 4 waves owns all M rows or a chunk of them, as MB blocks of 16, and a run
// of output columns (weight rows, NB blocks of 16) sized so that every CU streams about the same
// number of lines, and its waves split K: wave w takes the scale blocks w, w + 4, ... of 128
// features.  Wave w's step i then needs byte w of the i-th dword of every scale row.
//
//  * Each wave feeds itself: a private LDS ring of D steps, filled by direct-to-LDS loads of whole
//    128-byte lines (8 lanes a line); a step's slot is refilled as soon as its codes are in
//    registers, and there is no barrier.  D fills the 160 KiB of LDS (8 steps for one row block and one
//    column block, 2 for 6 and 3), which holds several times the bytes in flight that the registers
//    of the wave could.
//  * The fragments are read from LDS as 16-byte chunks (chunk c of row r at c ^ ((r >> 1) & 7)), widened
//    to bf16 times their scale (exact) and multiplied by v_mfma_f32_16x16x32_bf16: few rows leave the
//    matrix cores idle, so the products cost nothing by being exact, whatever the output type.
//  * The waves' fp32 partial tiles meet in LDS and are added in wave order, so each output is the same
//    sum whatever N is; one item per lane then applies bias, GELU or SwiGLU and rounding.
//
// 1 row x 9216 x 6144 takes 11 us (5.2 TB/s, a large copy's rate), 77 x 4608 x 6144 13.4 us and 96 x 9216
// x 6144 27 us.  From a few dozen rows on the activation re-reads through each CU bound it: without
// the products 64 x 9216 x 6144 takes 20.5 of 22.6 us, the weight alone 15.6, the activations alone 14.1.
#include <type_traits>

#include "gemm_tile.h"
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreadsN = 256;
constexpr int kWavesN4 = 4;
constexpr int kLdsBytes = 160 * 1024;

// Kept short: arguments beyond their second 64-byte line cost a small launch 0.2 us.
struct NarrowParams {
    const uint8_t *x, *w, *xs, *ws;
    const uint16_t *bias;
    void *y;
    uint32_t ldx, ldw, ldxs, ldws, ldy;  // at most 2^31
    int M, N, K;
    int rows;    // output columns per workgroup, a multiple of 4
    int m_rows;  // activation rows per workgroup
    int grid, minor;  // runs of columns x chunks of rows, and the smaller of the two counts
    uint32_t inverse;  // ceil(2^32 / minor): id * inverse >> 32 is id / minor while grid * minor < 2^32
    bool runs_minor;
    bool gelu;
};

template <int MB, int NB>
struct Ring {
    static constexpr int kBlocks = NB + MB;
    static constexpr int kScaleLoads = (kBlocks + 3) / 4;  // 64 rows each
    static constexpr int kStep = kBlocks * 2048 + kScaleLoads * 256;
    static constexpr int kLoads = 2 * kBlocks + kScaleLoads;  // per wave and step
    static constexpr int kFit = kLdsBytes / (kWavesN4 * kStep);
    static constexpr int kByCount = 60 / kLoads + 1;  // (D - 1) steps of loads fit the wait counter
    static constexpr int D = kFit < kByCount ? (kFit < 8 ? kFit : 8) : (kByCount < 8 ? kByCount : 8);
    static constexpr int kReduce = kWavesN4 * MB * NB * 1024;
    static constexpr int kBytes = kWavesN4 * D * kStep > kReduce ? kWavesN4 * D * kStep : kReduce;
    static_assert(D >= 2 && kBytes <= kLdsBytes, "two steps and the partial tiles fit in LDS");
};

// Four bytes a lane straight to LDS (lane l writes dst + 4 l), from the lane's own address.
__device__ __forceinline__ void dma4_lane(const char *src, char *dst)
{
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 4, 0, 0);
}

// Eight codes to bf16, times a power of two (exact).
__device__ __forceinline__ bf16x8 widen8(int a, int b, float s)
{
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
    return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

__device__ __forceinline__ f32x4 bias4(const uint16_t *b, int n)
{
    const bf16x4 v = *reinterpret_cast<const bf16x4 *>(b + n);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// NB blocks of 16 weight rows cover the workgroup's p.rows output columns (GATED: the first half of the
// blocks holds gate rows, the second the matching up rows).
template <int MB, int NB, bool GATED, bool OUT_BF16>
__global__ __launch_bounds__(kThreadsN) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_narrow_kernel(NarrowParams p)
{
    typedef Ring<MB, NB> R;
    constexpr int D = R::D, kBlocks = R::kBlocks;
    static_assert(!GATED || NB % 2 == 0, "the gated form pairs gate and up blocks");
    constexpr int kHalf = GATED ? NB / 2 : NB;  // blocks of output columns
    __shared__ __attribute__((aligned(1024))) char lds[R::kBytes];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The chunks of a run, or the runs of a chunk where those are fewer, lie side by side on one XCD, so
    // that its L2 fetches the larger operand once (3908 x 256 x 2304 12.9 us against 15.4, 132 x 3456 x
    // 1664 8.3 against 9.4).
    int run = blockIdx.x, chunk = 0;
    if (p.minor > 1) {
        const int id = xcd_contiguous(blockIdx.x, p.grid);
        const int q = __umulhi(id, p.inverse), r = id - q * p.minor;
        run = p.runs_minor ? r : q;
        chunk = p.runs_minor ? q : r;
    } else if (p.runs_minor) {
        run = 0;
        chunk = blockIdx.x;
    }
    const int n0 = run * p.rows, n_end = min(n0 + p.rows, p.N);
    const int m0 = chunk * p.m_rows, m_end = min(m0 + p.m_rows, p.M);
    const int steps = (p.K / kQBlock - wave + kWavesN4 - 1) / kWavesN4;
    char *ring = lds + wave * (D * R::kStep);
    // Row r of block b, W blocks first; rows past the end repeat the last one.
    const auto wrow = [&](int b, int r) {
        return GATED ? b / kHalf * p.N + min(n0 + 16 * (b % kHalf) + r, n_end - 1) : min(n0 + 16 * b + r, n_end - 1);
    };
    const auto xrow = [&](int b, int r) { return min(m0 + 16 * (b - NB) + r, m_end - 1); };
    uint32_t off[kBlocks][2];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + (lane >> 3), chunk = (lane & 7) ^ ((r >> 1) & 7);
            off[b][h] = b < NB ? (uint32_t)wrow(b, r) * p.ldw + chunk * 16
                               : (uint32_t)xrow(b, r) * p.ldx + chunk * 16;
        }
    // Scale load s: lane l takes row l % 16 of block 4 s + l / 16; a lane's block is W or X, so its
    // base differs, and the loads take 64-bit lane addresses.
    const char *sptr[R::kScaleLoads];
#pragma unroll
    for (int s = 0; s < R::kScaleLoads; ++s) {
        const int b = min(4 * s + (lane >> 4), kBlocks - 1), r = lane & 15;
        sptr[s] = reinterpret_cast<const char *>(b < NB ? p.ws : p.xs) +
                  (b < NB ? (uint32_t)wrow(b, r) * p.ldws : (uint32_t)xrow(b, r) * p.ldxs);
    }
    const char *xbase = reinterpret_cast<const char *>(p.x), *wbase = reinterpret_cast<const char *>(p.w);
    // step i of the wave into ring slot `slot`; past the last step, the last one again
    auto issue = [&](int i, int slot) {
        const int u = min(i, steps - 1);
        const int k = (u * kWavesN4 + wave) * kQBlock;
        char *d = ring + slot * R::kStep;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                dma16_sbase((b < NB ? wbase : xbase) + k, off[b][h], reinterpret_cast<uint16_t *>(d + b * 2048 + h * 1024));
#pragma unroll
        for (int s = 0; s < R::kScaleLoads; ++s)
            dma4_lane(sptr[s] + 4 * u, d + kBlocks * 2048 + s * 256);
    };
    f32x4 acc[MB][NB];
    zero<MB, NB>(acc);
    const int fr = lane & 15, g = lane >> 4, swz = (lane >> 1) & 7;
    if (steps > 0) {
#pragma unroll
        for (int i = 0; i < D; ++i)
            issue(i, i);
        int slot = 0;
        for (int i = 0; i < steps; ++i) {
            wait_dma_keep<(D - 1) * R::kLoads>();
            const char *s = ring + slot * R::kStep;
            i32x4 raw[kBlocks][2];
            float f[kBlocks];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    raw[b][h] = *reinterpret_cast<const i32x4 *>(s + b * 2048 + fr * 128 + ((4 * h + g) ^ swz) * 16);
                const uint32_t d = *reinterpret_cast<const uint32_t *>(s + kBlocks * 2048 + (16 * b + fr) * 4);
                // the scale byte as an fp32 exponent: all that the conversion looks at
                f[b] = __uint_as_float((d >> (8 * wave)) << 23);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read: refill it
            issue(i + D, slot);
            slot = slot == D - 1 ? 0 : slot + 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 w[NB];
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    w[j] = widen8(raw[j][q / 2][q % 2 * 2], raw[j][q / 2][q % 2 * 2 + 1], f[j]);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const bf16x8 x = widen8(raw[NB + m][q / 2][q % 2 * 2], raw[NB + m][q / 2][q % 2 * 2 + 1], f[NB + m]);
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], x, acc[m][j], 0, 0, 0);
                }
            }
        }
    }
    wait_dma();       // the repeated loads of the last step
    __syncthreads();  // every wave is done with its ring
    f32x4 *red = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            red[(wave * MB * NB + m * NB + j) * 64 + lane] = acc[m][j];
    __syncthreads();
    typedef typename std::conditional<OUT_BF16, __bf16, float>::type OutT;
    // Item (block, l): lane l of every wave holds Y[16 m + l % 16][n .. n + 3], n = column base + 16 j +
    // 4 (l / 16); n and n_end are multiples of 4.
    constexpr int kItems = MB * kHalf * 64;
    const auto total = [&](int blk, int l) {
        f32x4 v = red[blk * 64 + l];
#pragma unroll
        for (int w = 1; w < kWavesN4; ++w)
            v += red[(w * MB * NB + blk) * 64 + l];
        return v;
    };
    for (int e = threadIdx.x; e < kItems; e += kThreadsN) {
        const int l = e & 63, mb = (e >> 6) / kHalf, jb = (e >> 6) % kHalf, blk = mb * NB + jb;
        const int m = m0 + 16 * mb + (l & 15), n = n0 + 16 * jb + 4 * (l >> 4);
        if (m >= m_end || n >= n_end)
            continue;
        f32x4 v = total(blk, l);
        if (p.bias)
            v += bias4(p.bias, n);
        if (p.gelu) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = gelu_tanh(v[i]);
        }
        if (GATED) {
            f32x4 u = total(blk + kHalf, l);
            if (p.bias)
                u += bias4(p.bias, p.N + n);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = silu(v[i]) * u[i];
        }
        OutT *dst = reinterpret_cast<OutT *>(p.y) + (int64_t)m * p.ldy + n;
        if (OUT_BF16)
            *reinterpret_cast<bf16x4 *>(dst) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        else
            *reinterpret_cast<f32x4 *>(dst) = v;
    }
}

template <int MB, int NB, bool GATED>
hipError_t launch_mb(const NarrowParams &np, bool out_bf16, hipStream_t stream)
{
    const dim3 grid(np.grid), block(kThreadsN);
    if (out_bf16)
        hipLaunchKernelGGL((gemm_fp8_narrow_kernel<MB, NB, GATED, true>), grid, block, 0, stream, np);
    else
        hipLaunchKernelGGL((gemm_fp8_narrow_kernel<MB, NB, GATED, false>), grid, block, 0, stream, np);
    return hipGetLastError();
}

template <int NB, bool GATED>
hipError_t launch_nb(const NarrowParams &np, bool out_bf16, hipStream_t stream)
{
    const int blocks = (np.m_rows + 15) / 16;
    switch (blocks) {
    case 1: return launch_mb<1, NB, GATED>(np, out_bf16, stream);
    case 2: return launch_mb<2, NB, GATED>(np, out_bf16, stream);
    case 3: return launch_mb<3, NB, GATED>(np, out_bf16, stream);
    }
    // pick_runs gives more than 48 rows at least two blocks of columns, and SwiGLU more than 80 rows two
    if constexpr (NB > 1) {
        if (blocks == 4)
            return launch_mb<4, NB, GATED>(np, out_bf16, stream);
        if (blocks == 5)
            return launch_mb<5, NB, GATED>(np, out_bf16, stream);
        if constexpr (NB <= 3)
            return launch_mb<6, NB, GATED>(np, out_bf16, stream);
    }
    return hipErrorInvalidValue;
}

// Output columns and activation rows per workgroup.  Every workgroup streams its weight rows (from
// HBM) and its activation rows (from L2, like weight rows that another workgroup reads too) through one
// CU, and the LDS ring leaves room for one workgroup per CU.  The cost of a choice is ceil(workgroups / CUs) x
// (32 + weight rows + 0.8 x activation rows): 32 for a round's start and end; activation rows are
// counted in whole blocks of 16, a partial block of weight rows as if half of what it lacks were there
// (rows past the end repeat the last one, which loads cheaply).  That chooses all rows together with few
// rows and many columns, 16 rows each with few columns, and between them what evens the CUs' loads: 77 x
// 4608 x 6144 takes two chunks of 39 rows by 36 columns (256 workgroups: 15.9 us against 17.8 for 231 of all
// rows by 20), 100 x 64 x 9216 seven of 15 by 4 (7.6 us against 8.8 in 32 by 16 and 18 in 96 by 16).  Ties go
// to fewer chunks, then to more columns.
struct Runs {
    int cols, m_rows;
    bool one_round;
    double cost;  // per round, without its start and end
};

Runs pick_runs(const Fp8Problem &p, int cus)
{
    Runs best{4, 16, false, 0};
    double best_cost = -1;
    const uint32_t M = p.M ? (uint32_t)p.M : 1, N = (uint32_t)p.N;
    for (uint32_t blocks = 6; blocks >= 1; --blocks) {
        const uint32_t chunks = (M + 16 * blocks - 1) / (16 * blocks), m_rows = (M + chunks - 1) / chunks;
        // MB + NB <= 9 blocks fit the ring: three, or with SwiGLU, which pairs them, four up to 80 rows
        const uint32_t max_cols = p.swiglu ? (m_rows <= 80 ? 32 : 16) : 48;
        const uint32_t min_cols = p.swiglu || m_rows <= 48 ? 4 : 20;  // many rows by one block of columns never paid
        for (uint32_t cols = max_cols; cols >= min_cols; cols -= 4) {
            const uint64_t wgs = (uint64_t)((N + cols - 1) / cols) * chunks;
            const uint32_t c16 = (cols + 15) / 16 * 16, m16 = (m_rows + 15) / 16 * 16;
            const double one = (p.swiglu ? 1.0 : 0.5) * (cols + c16) + 0.8 * m16;
            const double cost = (double)((wgs + cus - 1) / cus) * (one + 32);
            if (best_cost < 0 || cost < best_cost) {
                best = Runs{(int)cols, (int)m_rows, wgs <= (uint64_t)cus, one};
                best_cost = cost;
            }
        }
    }
    return best;
}

}  // namespace

// Up to kFp8NarrowMaxM rows this kernel runs every product.  Beyond, it runs those whose outputs are few
// enough for one round of workgroups, where the tiled kernels leave most CUs idle and do not split K
// (500 x 256 x 9216: 10 us against 25 bf16 and 44 fp32 in the tile of 64 x 128; 1500 x 64 x 768: 4.4 against 5.1
// and 6.7).  Its round takes about 2.3 + 0.13 K' + (0.027 + 0.012 K') cost us at K = 1000 K', that tile's 3.3 + 2.3
// K' with 8-bit products and 3.4 + 4.3 K' with exact ones: a costly round at a short K is for the tile (bf16:
// 333 x 2304 x 768 5.7 us against 7.1, at K = 9216 28 against 22.4; fp32: 2156 x 496 x 128 4.6 against 5.7).
bool gemm_fp8_narrow_takes(const Fp8Problem &p)
{
    if (p.M <= kFp8NarrowMaxM)
        return true;
    const int cus = cu_count();
    if (p.M * p.N > (int64_t)cus * 96 * 48)
        return false;  // more than one round whatever the choice
    const Runs r = pick_runs(p, cus);
    return r.one_round && r.cost <= (p.out_bf16 ? 64.0 + (double)p.K / 80 : 100.0 + (double)p.K / 32);
}

void gemm_fp8_narrow_shape(const Fp8Problem &p, int *rows, int *cols)
{
    const Runs r = pick_runs(p, cu_count());
    *rows = (r.m_rows + 15) / 16 * 16;
    *cols = r.cols;
}

hipError_t launch_gemm_fp8_narrow(const Fp8Problem &pr, hipStream_t stream)
{
    NarrowParams np;
    np.x = pr.x;
    np.w = pr.w;
    np.xs = pr.xs;
    np.ws = pr.ws;
    np.bias = pr.bias;
    np.y = pr.y;
    np.ldx = (uint32_t)pr.ldx;
    np.ldw = (uint32_t)pr.ldw;
    np.ldxs = (uint32_t)pr.ldxs;
    np.ldws = (uint32_t)pr.ldws;
    np.ldy = (uint32_t)pr.ldy;
    np.M = (int)pr.M;
    np.N = (int)pr.N;
    np.K = (int)pr.K;
    const Runs runs = pick_runs(pr, cu_count());
    np.rows = runs.cols;
    np.m_rows = runs.m_rows;
    const int num_runs = (np.N + np.rows - 1) / np.rows, chunks = (np.M + np.m_rows - 1) / np.m_rows;
    np.grid = num_runs * chunks;
    np.runs_minor = num_runs < chunks;
    np.minor = np.runs_minor ? num_runs : chunks;
    np.inverse = (uint32_t)((((uint64_t)1 << 32) + np.minor - 1) / np.minor);  // unused for 1
    np.gelu = pr.gelu;
    if (pr.swiglu)
        return np.rows <= 16 ? launch_nb<2, true>(np, pr.out_bf16, stream) : launch_nb<4, true>(np, pr.out_bf16, stream);
    switch ((np.rows + 15) / 16) {
    case 1: return launch_nb<1, false>(np, pr.out_bf16, stream);
    case 2: return launch_nb<2, false>(np, pr.out_bf16, stream);
    default: return launch_nb<3, false>(np, pr.out_bf16, stream);
    }
}

}  // namespace tpl
