// gemm_fp8_small.hip -- tiled product of quantized rows for a few hundred rows, eight waves a tile.
//
// Between the split-K kernel's 96 rows and the thousand or so that fill the CUs with the four-wave
// tiles, a launch is one partial round of tiles and its time is that of one tile: k-tiles times the
// latency and the feed of one CU.  So tiles are 128, 96 or 64 rows by 128 columns, four or five k-tiles are
// in flight in LDS, and two waves per SIMD cover each other: 8 waves in a 2 x 4 grid, scheduled
// by the compiler within a k-tile, whose codes and scales are read from LDS a k-tile ahead.  333 x
// 6144 x 4608 takes 21 us with bf16 output (8-bit products) and 33 with fp32 output (exact products,
// widened to bf16); the four-wave 192 x 192 tiles take 34 and 54.  Loads alone take 0.5 to 0.7 us a
// k-tile and CU (46 GB/s a CU), the exact products 0.4 to 0.7.
#include "gemm_tile.h"
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRow = 128;         // bytes of a row in an LDS tile: one scale block
constexpr int kThreadsS = 512;    // 8 waves in a 2 (M) x 4 (N) grid

struct SmallParams {
    const uint8_t *x, *w, *xs, *ws;
    const uint16_t *bias;
    void *y;
    int64_t ldx, ldw, ldxs, ldws, ldy;
    int M, N, K;
    int tiles_m, tiles_n, group_m;
};

template <int NXB, int NWB>
struct STile {
    static constexpr int WM = 16 * NXB, WN = 16 * NWB, BM = 2 * WM, BN = 4 * WN;
    static constexpr int kPer = (BM + BN + 63) / 64;  // loads per wave and k-tile: 64 rows each, X then W
    static constexpr int kStageBytes = kPer * 64 * kRow;
    static constexpr int kFit = (160 * 1024 - 4096) / kStageBytes;
    static constexpr int kStages = kFit > 5 ? 5 : kFit;
    static constexpr int kLdsBytes = kStages * kStageBytes + 4096;
};

// A scale byte as an fp32 exponent: all that the conversion below looks at (255 is NaN, 0 is 2^-127).
__device__ __forceinline__ float factor(uint32_t dword, int u) { return __uint_as_float((dword >> (8 * (u & 3))) << 23); }

// Eight codes to bf16, times a power of two (exact).
__device__ __forceinline__ bf16x8 widen8(int a, int b, float s)
{
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
    return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

__device__ __forceinline__ void dma_to_lds16(const char *src, char *dst)
{
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}
__device__ __forceinline__ void dma_to_lds4(const char *src, char *dst)
{
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 4, 0, 0);
}

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// EXACT: products of the codes widened to bf16; otherwise on the 8-bit matrix cores.
template <int NXB, int NWB, bool GATED, bool EXACT>
__device__ __forceinline__ void mainloop_small(const SmallParams &p, char *lds, const Ctx &c, int m0, int n0,
                                               f32x4 (&acc)[NXB][NWB])
{
    typedef STile<NXB, NWB> L;
    constexpr int BM = L::BM, BN = L::BN, S = L::kStages;
    constexpr int kPer = L::kPer;
    static_assert(S >= 2 && (S - 1) * kPer <= 60, "the wait count fits vmcnt");
    // weight row of a tile row; gated: a wave column's first half holds gate rows, its second up rows
    auto wrow = [&](int r) {
        if (!GATED)
            return min(n0 + r, p.N - 1);
        const int q = r / L::WN, o = r % L::WN;
        return (o / (L::WN / 2)) * p.N + min(n0 + q * (L::WN / 2) + o % (L::WN / 2), p.N - 1);
    };
    const int dma_row = c.wave * 8 + (c.lane >> 3);
    const int dma_chunk = (c.lane & 7) ^ ((((c.wave & 1) << 2) + (c.lane >> 4)) & 7);
    uint32_t off[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int r = 64 * j + dma_row;  // rows past the W tile (a last load of half the waves) repeat its last
        off[j] = r < BM ? (uint32_t)min(m0 + r, p.M - 1) * (uint32_t)p.ldx + dma_chunk * 16
                        : (uint32_t)wrow(min(r - BM, BN - 1)) * (uint32_t)p.ldw + dma_chunk * 16;
    }
    const int T = p.K / kRow, groups = (T + 3) / 4;
    const char *xbase = reinterpret_cast<const char *>(p.x), *wbase = reinterpret_cast<const char *>(p.w);
    auto issue = [&](int u, int stage) {
        const int k = min(u, T - 1) * kRow;
        char *d = lds + stage * L::kStageBytes + c.wave * 1024;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            dma_to_lds16((64 * j + 8 * c.wave < BM ? xbase : wbase) + k + off[j], d + j * 8192);
    };
    // Scales of four k-tiles, a dword a row: the X tile's rows, then the W tile's; two buffers.
    char *sl = lds + S * L::kStageBytes;
    const int srow = c.wave * 64 + c.lane;
    const char *sbase = reinterpret_cast<const char *>(srow < BM ? p.xs : p.ws);
    const uint32_t soff = srow < BM ? (uint32_t)min(m0 + srow, p.M - 1) * (uint32_t)p.ldxs
                                    : (uint32_t)wrow(min(srow - BM, BN - 1)) * (uint32_t)p.ldws;
    auto issue_scales = [&](int group) {
        dma_to_lds4(sbase + 4 * min(group, groups - 1) + soff, sl + (group & 1) * 2048 + c.wave * 256);
    };
    issue_scales(0);
#pragma unroll
    for (int u = 0; u < S; ++u)
        issue(u, u);
    const int fr = c.lane & 15, g = c.lane >> 4, swz = (c.lane >> 1) & 7;
    const int xrow = c.wave_m * L::WM + fr, wr0 = c.wave_n * L::WN + fr;
    // A k-tile's codes and scales in registers, read one k-tile ahead of the products that use them.
    struct Codes {
        i32x4 x[2][NXB], w[2][NWB];
        uint32_t sx[NXB], sw[NWB];
    };
    auto read = [&](int u, int stage, Codes &r) {
        const char *xs = lds + stage * L::kStageBytes, *ws = xs + BM * kRow;
        const char *sc = sl + ((u >> 2) & 1) * 2048;
#pragma unroll
        for (int i = 0; i < NXB; ++i)
            r.sx[i] = *reinterpret_cast<const uint32_t *>(sc + (xrow + 16 * i) * 4);
#pragma unroll
        for (int j = 0; j < NWB; ++j)
            r.sw[j] = *reinterpret_cast<const uint32_t *>(sc + (BM + wr0 + 16 * j) * 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int cpos = ((4 * h + g) ^ swz) * 16;
#pragma unroll
            for (int j = 0; j < NWB; ++j)
                r.w[h][j] = *reinterpret_cast<const i32x4 *>(ws + (wr0 + 16 * j) * kRow + cpos);
#pragma unroll
            for (int i = 0; i < NXB; ++i)
                r.x[h][i] = *reinterpret_cast<const i32x4 *>(xs + (xrow + 16 * i) * kRow + cpos);
        }
    };
    auto multiply = [&](int u, const Codes &r) {
        if constexpr (!EXACT) {
            const int byte = 8 * (u & 3);
#pragma unroll
            for (int i = 0; i < NXB; ++i)
#pragma unroll
                for (int j = 0; j < NWB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        join(r.w[0][j], r.w[1][j]), join(r.x[0][i], r.x[1][i]), acc[i][j], 0, 0, 0, r.sw[j] >> byte, 0,
                        r.sx[i] >> byte);
            return;
        }
        float fx[NXB], fw[NWB];
#pragma unroll
        for (int i = 0; i < NXB; ++i)
            fx[i] = factor(r.sx[i], u);
#pragma unroll
        for (int j = 0; j < NWB; ++j)
            fw[j] = factor(r.sw[j], u);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf16x8 w[NWB];
#pragma unroll
            for (int j = 0; j < NWB; ++j)
                w[j] = widen8(r.w[s / 2][j][s % 2 * 2], r.w[s / 2][j][s % 2 * 2 + 1], fw[j]);
#pragma unroll
            for (int i = 0; i < NXB; ++i) {
                const bf16x8 x = widen8(r.x[s / 2][i][s % 2 * 2], r.x[s / 2][i][s % 2 * 2 + 1], fx[i]);
#pragma unroll
                for (int j = 0; j < NWB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], x, acc[i][j], 0, 0, 0);
            }
        }
    };
    // k-tile u is in stage u % S.
    wait_dma_keep<(S - 1) * kPer>();
    barrier_only();
    Codes ca, cb;
    read(0, 0, ca);
    int stage = 0;  // of k-tile t
    // At the barrier of k-tile t, k-tile t + 1 has landed (the S - 2 after it stay in flight) and every
    // wave has k-tile t in registers, so its stage takes k-tile t + S.  The scales of the next group
    // of four k-tiles go out at a group's first k-tile, ahead of its loads, and are read three
    // k-tiles later, behind a wait that leaves at most S - 2 <= 3 k-tiles of loads in flight.
    auto body = [&](int t, const Codes &cur, Codes &nxt) {
        const int next = stage == S - 1 ? 0 : stage + 1;
        wait_dma_keep<(S - 2) * kPer>();
        barrier_only();
        if ((t & 3) == 0)
            issue_scales((t >> 2) + 1);
        issue(t + S, stage);
        // lgkmcnt(0) once more, in a form that the compiler sees: without it, it takes `cur` for still
        // on its way and waits for the reads below before the products
        __builtin_amdgcn_s_waitcnt(0xc07f);
        read(t + 1, next, nxt);
        __builtin_amdgcn_sched_barrier(0);  // the reads go out before the products, not after them
        multiply(t, cur);
        stage = next;
    };
    for (int t = 0;;) {
        body(t, ca, cb);
        if (++t == T)
            break;
        body(t, cb, ca);
        if (++t == T)
            break;
    }
    wait_dma();  // the repeated loads of the last k-tile, before the epilogue reuses the LDS
}

template <int NXB, int NWB, bool OUT_BF16, bool HAS_BIAS, int ACT>
__global__ __launch_bounds__(kThreadsS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gemm_fp8_small_kernel(SmallParams p)
{
    typedef STile<NXB, NWB> L;
    constexpr bool kGated = ACT == kActSwiglu;
    constexpr int kTileCols = kGated ? L::BN / 2 : L::BN;
    __shared__ __attribute__((aligned(1024))) char lds[L::kLdsBytes];
    Ctx c;
    c.lane = threadIdx.x & 63;
    c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c.wave_m = c.wave >> 2;
    c.wave_n = c.wave & 3;
    int tm, tn;
    tile_of(xcd_contiguous(blockIdx.x, p.tiles_m * p.tiles_n), p, tm, tn);
    f32x4 acc[NXB][NWB];
    zero<NXB, NWB>(acc);
    mainloop_small<NXB, NWB, kGated, !OUT_BF16>(p, lds, c, tm * L::BM, tn * kTileCols, acc);
    epilogue<NXB, NWB, OUT_BF16, HAS_BIAS, ACT, true>(p, reinterpret_cast<uint16_t *>(lds), c, tm * L::BM, tn * kTileCols, acc);
}

template <int NXB, int NWB, bool OUT_BF16, bool HAS_BIAS, int ACT>
hipError_t launch_tile(SmallParams gp, hipStream_t stream)
{
    typedef STile<NXB, NWB> L;
    const int cols = ACT == kActSwiglu ? L::BN / 2 : L::BN;
    gp.tiles_n = (gp.N + cols - 1) / cols;
    gp.tiles_m = (gp.M + L::BM - 1) / L::BM;
    gp.group_m = gp.tiles_m < 8 ? gp.tiles_m : 8;
    hipLaunchKernelGGL((gemm_fp8_small_kernel<NXB, NWB, OUT_BF16, HAS_BIAS, ACT>), dim3(gp.tiles_m * gp.tiles_n),
                       dim3(kThreadsS), 0, stream, gp);
    return hipGetLastError();
}

template <bool OUT_BF16, bool HAS_BIAS, int ACT>
hipError_t launch_shape(const SmallParams &gp, int nxb, hipStream_t stream)
{
    switch (nxb) {
    case 2: return launch_tile<2, 2, OUT_BF16, HAS_BIAS, ACT>(gp, stream);
    case 3: return launch_tile<3, 2, OUT_BF16, HAS_BIAS, ACT>(gp, stream);
    default: return launch_tile<4, 2, OUT_BF16, HAS_BIAS, ACT>(gp, stream);
    }
}

}  // namespace

hipError_t launch_gemm_fp8_small(const Fp8Problem &pr, int nxb, hipStream_t stream)
{
    SmallParams gp;
    gp.x = pr.x;
    gp.w = pr.w;
    gp.xs = pr.xs;
    gp.ws = pr.ws;
    gp.bias = pr.bias;
    gp.y = pr.y;
    gp.ldx = pr.ldx;
    gp.ldw = pr.ldw;
    gp.ldxs = pr.ldxs;
    gp.ldws = pr.ldws;
    gp.ldy = pr.ldy;
    gp.M = (int)pr.M;
    gp.N = (int)pr.N;
    gp.K = (int)pr.K;
    const int act = pr.swiglu ? kActSwiglu : (pr.gelu ? kActGelu : kActNone);
    switch ((pr.out_bf16 ? 6 : 0) + (pr.bias ? 3 : 0) + act) {
    case 0: return launch_shape<false, false, 0>(gp, nxb, stream);
    case 1: return launch_shape<false, false, 1>(gp, nxb, stream);
    case 2: return launch_shape<false, false, 2>(gp, nxb, stream);
    case 3: return launch_shape<false, true, 0>(gp, nxb, stream);
    case 4: return launch_shape<false, true, 1>(gp, nxb, stream);
    case 5: return launch_shape<false, true, 2>(gp, nxb, stream);
    case 6: return launch_shape<true, false, 0>(gp, nxb, stream);
    case 7: return launch_shape<true, false, 1>(gp, nxb, stream);
    case 8: return launch_shape<true, false, 2>(gp, nxb, stream);
    case 9: return launch_shape<true, true, 0>(gp, nxb, stream);
    case 10: return launch_shape<true, true, 1>(gp, nxb, stream);
    default: return launch_shape<true, true, 2>(gp, nxb, stream);
    }
}

}  // namespace tpl
