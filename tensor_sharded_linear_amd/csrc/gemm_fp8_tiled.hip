// gemm_fp8_tiled.hip -- tiled product of quantized rows on the 8-bit matrix cores, bf16 output.
#include "gemm_tile.h"
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kRow = 128;  // bytes of a row in an LDS tile: one scale block
constexpr int kThreads8 = 256;

struct Fp8Params {
    const uint8_t *x, *w, *xs, *ws;
    const uint16_t *bias;
    void *y;
    int64_t ldx, ldw, ldxs, ldws, ldy;
    int M, N, K;
    int tiles_m, tiles_n, group_m;
};

// f(0), f(1), ... with compile-time indexes: the main loop's body is longer than the loop unroller
// takes.
template <typename F, int... Q>
__device__ __forceinline__ void each(F &&f, std::integer_sequence<int, Q...>)
{
    (f(std::integral_constant<int, Q>{}), ...);
}

// dma16_sbase with 4 bytes a lane (lane l writes dst + 4 l).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4_sbase(const char *base, uint32_t off, char *dst)
{
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)dst;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(m0), "v"(off), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// acc += 2^(sw + sx - 254) w . x^T over 128 features, the scales byte BYTE of sw and sx.
template <int BYTE>
__device__ __forceinline__ void scaled_mfma(f32x4 &acc, const i32x8 &w, const i32x8 &x, uint32_t sw, uint32_t sx)
{
#define TPL_SCALED_MFMA(SEL)                                                                               \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL                            \
                 : "+a"(acc) : "v"(w), "v"(x), "v"(sw), "v"(sx) : "memory")
    if constexpr (BYTE == 0)
        TPL_SCALED_MFMA("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
    else if constexpr (BYTE == 1)
        TPL_SCALED_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
    else if constexpr (BYTE == 2)
        TPL_SCALED_MFMA("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
    else
        TPL_SCALED_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef TPL_SCALED_MFMA
}

template <int NXB, int NWB, bool GATED>
__device__ __forceinline__ void mainloop8(const Fp8Params &p, uint16_t *lds, const Ctx &c, int m0, int n0,
                                          f32x4 (&acc)[NXB][NWB])
{
    constexpr int WM = 16 * NXB, WN = 16 * NWB, BM = 2 * WM, BN = 2 * WN;
    constexpr int kXBytes = BM * kRow, kWBytes = BN * kRow;
    constexpr int kDmaX = BM / 32, kDmaW = BN / 32, kDma = kDmaX + kDmaW;
    constexpr int kMfma = NXB * NWB, kLast = kMfma - NXB;  // first MFMA of the last W block
    constexpr int RS = (NWB - 1) / 2;                      // X reads: one every RS MFMAs
    constexpr int DS = 2;                                  // loads: one every DS MFMAs after the barrier
    constexpr int kF = NXB / DS;                           // loads issued within the last W block
    static_assert(NWB % 2 == 0 && (2 * NXB - 1) * RS < kLast, "reads fit");
    static_assert(!GATED || NWB == 8, "the gated tile pairs four gate and four up blocks per wave");
    static_assert(NXB >= 5, "the scale reads are placed within a W block");
    char *base = reinterpret_cast<char *>(lds);
    const int dma_row = c.wave * 8 + (c.lane >> 3);
    const int dma_chunk = (c.lane & 7) ^ ((((c.wave & 1) << 2) + (c.lane >> 4)) & 7);
    const int fr = c.lane & 15, g = c.lane >> 4, swz = (c.lane >> 1) & 7;
    uint32_t xoff[kDmaX], woff[kDmaW];
#pragma unroll
    for (int j = 0; j < kDmaX; ++j)
        xoff[j] = (uint32_t)min(m0 + 32 * j + dma_row, p.M - 1) * (uint32_t)p.ldx + dma_chunk * 16;
#pragma unroll
    for (int j = 0; j < kDmaW; ++j) {
        const int gn = GATED ? ((j >> 1) & 1) * p.N + min(n0 + 64 * (j >> 2) + 32 * (j & 1) + dma_row, p.N - 1)
                             : min(n0 + 32 * j + dma_row, p.N - 1);
        woff[j] = (uint32_t)gn * (uint32_t)p.ldw + dma_chunk * 16;
    }
    const char *xbase = reinterpret_cast<const char *>(p.x);
    const char *wbase = reinterpret_cast<const char *>(p.w);
    const int T = p.K / kRow;
    auto kt = [&](int u) { return min(u, T - 1) * kRow; };
    auto dma_x = [&](int d, int u) {
        dma16_sbase(xbase + kt(u), xoff[d],
                    reinterpret_cast<uint16_t *>(base + (u & 1) * kXBytes + (d * 4 + c.wave) * 1024));
    };
    auto dma_w = [&](int d, int u) {
        dma16_sbase(wbase + kt(u), woff[d],
                    reinterpret_cast<uint16_t *>(base + 2 * kXBytes + (u & 1) * kWBytes + (d * 4 + c.wave) * 1024));
    };
    // load d of the step after barrier u: W of k-tile u + 2, X of k-tile u + 3
    auto dma = [&](int d, int u) {
        if (d < kDmaW)
            dma_w(d, u + 2);
        else
            dma_x(d - kDmaW, u + 3);
    };
    const char *xl = base + (c.wave_m * WM + fr) * kRow;
    const char *wl = base + 2 * kXBytes + (c.wave_n * WN + fr) * kRow;
    const int c0 = (g ^ swz) * 16, c1 = ((4 + g) ^ swz) * 16;
    auto read = [&](const char *t, int block, int half) {
        return *reinterpret_cast<const i32x4 *>(t + block * 16 * kRow + (half ? c1 : c0));
    };
    auto set = [](i32x8 &f, int half, i32x4 v) {
        if (half == 0)
            f = __builtin_shufflevector(__builtin_shufflevector(v, v, 0, 1, 2, 3, 0, 1, 2, 3), f, 0, 1, 2, 3, 12, 13, 14, 15);
        else
            f = __builtin_shufflevector(f, __builtin_shufflevector(v, v, 0, 1, 2, 3, 0, 1, 2, 3), 0, 1, 2, 3, 8, 9, 10, 11);
    };
    // Scales: a dword holds a row's scales of four k-tiles.  Lane l of wave w loads row 64 w + l of
    // the X tile and of the W tile, group u / 4 into buffer (u / 4) % 2.
    char *sl = base + 2 * (kXBytes + kWBytes);
    const int srow = c.wave * 64 + c.lane;
    const uint32_t xsoff = (uint32_t)min(m0 + min(srow, BM - 1), p.M - 1) * (uint32_t)p.ldxs;
    const int sn = min(srow, BN - 1);
    const uint32_t wsoff = (uint32_t)(GATED ? ((sn >> 6) & 1) * p.N + min(n0 + 64 * (sn >> 7) + (sn & 63), p.N - 1)
                                            : min(n0 + sn, p.N - 1)) * (uint32_t)p.ldws;
    auto dma_scales = [&](int group) {
        char *d = sl + (group & 1) * 2048 + c.wave * 256;
        dma4_sbase(reinterpret_cast<const char *>(p.xs) + 4 * group, xsoff, d);
        dma4_sbase(reinterpret_cast<const char *>(p.ws) + 4 * group, wsoff, d + 1024);
    };
    const char *xsl = sl + (c.wave_m * WM + fr) * 4, *wsl = sl + 1024 + (c.wave_n * WN + fr) * 4;
    auto scale = [](const char *t, int buf, int block) {
        return *reinterpret_cast<const uint32_t *>(t + buf * 2048 + block * 64);
    };
    const int groups = (T + 3) / 4;
    uint32_t sx[NXB], sw[NWB];

    // prologue
    i32x8 fa[NXB] = {}, fb[NXB] = {}, fw[2] = {};
#pragma unroll
    for (int d = 0; d < kDmaX; ++d)
        dma_x(d, 0);
#pragma unroll
    for (int d = 0; d < kDmaW; ++d)
        dma_w(d, 0);
#pragma unroll
    for (int d = 0; d < kDmaX; ++d)
        dma_x(d, 1);
    dma_scales(0);
    wait_dma_keep<0>();
    barrier_only();
#pragma unroll
    for (int i = 0; i < NXB; ++i) {
        set(fa[i], 0, read(xl, i, 0));
        set(fa[i], 1, read(xl, i, 1));
        sx[i] = scale(xsl, 0, i);
    }
    set(fw[0], 0, read(wl, 0, 0));
    set(fw[0], 1, read(wl, 0, 1));
#pragma unroll
    for (int j = 0; j < NWB; ++j)
        sw[j] = scale(wsl, 0, j);
    wait_dma_keep<0>();
    barrier_only();
#pragma unroll
    for (int d = 0; d < kF; ++d)
        dma(d, -1);
    int t = 0;
    // k-tile t, with S = t % 4
    auto body = [&](i32x8 (&cur)[NXB], i32x8 (&nxt)[NXB], auto S) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value, par = st & 1;
        const char *xn = xl + (par ^ 1) * kXBytes;          // X of k-tile t + 1
        const char *wc = wl + par * kWBytes, *wn = wl + (par ^ 1) * kWBytes;
        const int buf = (t >> 2) & 1;  // of this k-tile's scales
        each([&](auto Q) __attribute__((always_inline)) {
            constexpr int q = decltype(Q)::value, j = q / NXB, i = q % NXB;
            if constexpr (q == kLast) {
                wait_dma_keep<0>();
                barrier_only();
            }
            scaled_mfma<st>(acc[i][j], fw[j & 1], cur[i], sw[j], sx[i]);
            // loads: the rest of the step after the previous barrier, then the first of this one's
            if constexpr (q < kLast) {
                if constexpr (q % DS == 0 && kF + q / DS < kDma)
                    dma(kF + q / DS, t - 1);
            } else if constexpr ((q - kLast) % DS == 0 && (q - kLast) / DS < kF) {
                dma((q - kLast) / DS, t);
            }
            // fragments: X of the next k-tile, the next W block
            if constexpr (q % RS == 0 && q / RS < 2 * NXB)
                set(nxt[q / RS / 2], q / RS % 2, read(xn, q / RS / 2, q / RS % 2));
            if constexpr (i == 1 || i == 2) {
                if constexpr (j < NWB - 1)
                    set(fw[(j + 1) & 1], i - 1, read(wc, j + 1, i - 1));
                else
                    set(fw[0], i - 1, read(wn, 0, i - 1));
            }
            // scales of the next four k-tiles, each after the last use of these
            if constexpr (st == 0 && q == 0)
                sx[NXB - 1] = scale(xsl, buf, NXB - 1);
            if constexpr (st == 0 && q == 4)
                sw[NWB - 1] = scale(wsl, buf, NWB - 1);
            if constexpr (st == 3 && q > kLast)
                sx[i - 1] = scale(xsl, buf ^ 1, i - 1);
            if constexpr (st == 3 && j > 0 && i == 4)
                sw[j - 1] = scale(wsl, buf ^ 1, j - 1);
            if constexpr (st == 1 && q == NXB)
                dma_scales(min(t / 4 + 1, groups - 1));
        }, std::make_integer_sequence<int, kMfma>{});
    };
    for (;;) {
        body(fa, fb, std::integral_constant<int, 0>{});
        if (++t == T)
            break;
        body(fb, fa, std::integral_constant<int, 1>{});
        if (++t == T)
            break;
        body(fa, fb, std::integral_constant<int, 2>{});
        if (++t == T)
            break;
        body(fb, fa, std::integral_constant<int, 3>{});
        if (++t == T)
            break;
    }
    wait_dma();
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < NXB; ++i)
#pragma unroll
        for (int j = 0; j < NWB; ++j)
            asm volatile("" : "+a"(acc[i][j]));
}

template <int NXB, int NWB, bool HAS_BIAS, int ACT>
__global__ __launch_bounds__(kThreads8) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_nt_kernel(Fp8Params p)
{
    constexpr bool kGated = ACT == kActSwiglu;
    constexpr int BM = 32 * NXB, BN = 32 * NWB, kTileCols = kGated ? BN / 2 : BN;
    __shared__ __attribute__((aligned(1024))) uint16_t lds[(BM + BN) * kRow + 2048];  // two stages, two scale groups
    Ctx c;
    c.lane = threadIdx.x & 63;
    c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c.wave_m = c.wave >> 1;
    c.wave_n = c.wave & 1;
    int tm, tn;
    tile_of(xcd_contiguous(blockIdx.x, p.tiles_m * p.tiles_n), p, tm, tn);
    f32x4 acc[NXB][NWB];
    zero<NXB, NWB>(acc);
    mainloop8<NXB, NWB, kGated>(p, lds, c, tm * BM, tn * kTileCols, acc);
    epilogue<NXB, NWB, true, HAS_BIAS, ACT>(p, lds, c, tm * BM, tn * kTileCols, acc);
}

template <int NXB, int NWB, bool HAS_BIAS, int ACT>
hipError_t launch_tile(Fp8Params gp, hipStream_t stream)
{
    const int cols = ACT == kActSwiglu ? 16 * NWB : 32 * NWB;
    gp.tiles_n = (gp.N + cols - 1) / cols;
    gp.tiles_m = (gp.M + 32 * NXB - 1) / (32 * NXB);
    gp.group_m = gp.tiles_m < 8 ? gp.tiles_m : 8;
    hipLaunchKernelGGL((gemm_fp8_nt_kernel<NXB, NWB, HAS_BIAS, ACT>), dim3(gp.tiles_m * gp.tiles_n), dim3(kThreads8),
                       0, stream, gp);
    return hipGetLastError();
}

template <bool HAS_BIAS>
hipError_t launch_act(const Fp8Params &gp, int act, hipStream_t stream)
{
    switch (act) {
    case kActGelu: return launch_tile<8, 8, HAS_BIAS, kActGelu>(gp, stream);
    case kActSwiglu: return launch_tile<8, 8, HAS_BIAS, kActSwiglu>(gp, stream);
    default: return launch_tile<8, 8, HAS_BIAS, kActNone>(gp, stream);
    }
}

}  // namespace

hipError_t launch_gemm_fp8_tiled(const Fp8Problem &pr, hipStream_t stream)
{
    Fp8Params gp;
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
    return pr.bias ? launch_act<true>(gp, act, stream) : launch_act<false>(gp, act, stream);
}

}  // namespace tpl
