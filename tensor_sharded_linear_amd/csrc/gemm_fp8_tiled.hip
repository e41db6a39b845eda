// gemm_fp8_tiled.hip -- tiled product of quantized rows for many rows, four waves a tile.
//
//   y[m, n] = sum_b 2^(sx[m,b] + sw[n,b]) sum_{k in block b} x[m,k] w[n,k]
//
// Two main loops over the same LDS tiles:
//
//  * mainloop8 (bf16 output): v_mfma_scale_f32_16x16x128_f8f6f4, whose 128 features are one scale block, so
//    the matrix core multiplies by both rows' scales itself and the loop holds nothing but
//    MFMAs, fragment reads and loads.  Among the products of each 8 consecutive features that
//    instruction drops what lies 2^13 below the largest (found by products of chosen magnitudes), about
//    1.5e-5 of a result: a hundredth of the bf16 rounding, but 200 times an fp32 accumulation's error.
//  * mainloop_exact (fp32 output): the codes are widened to bf16 times their scale, which is exact,
//    and multiplied by v_mfma_f32_16x16x32_bf16 at half the rate.
//
// Bound by the matrix cores.  4608 x 9216 x 6144 takes 184 us (2.83 PF; about 200 with bias and GELU), where the
// vendor library's e4m3 product with one scale per tensor takes 188; 8192^3 369 us (2.98 PF).  fp32
// output: 4608 x 6144 x 4608 takes 174 to 182 us (1.50 PF; the vendor's bf16 product 169).  The matrix cores are
// busy 55 to 65% of a launch's cycles; the rest is the start and the epilogue of each tile (about 8 us of
// 62), the last round's gap, and loads that land late.
//
//  * 256 threads = 4 waves in a 2 x 2 grid, one wave per SIMD with 512 registers, each owning up to
//    128 x 128 outputs as 8 x 8 accumulators in the accumulation registers; 256, 224 or 192 rows by 256 or
//    192 columns.  MFMAs are written as assembly with their accumulators tied to those registers,
//    and the order of every instruction between them is written out (each()).
//  * An LDS row is the 128 bytes of one scale block of one row, so a k-tile is as many bytes as in the
//    bf16 kernel and the MFMAs of a k-tile take as many cycles.  X fragments are read a k-tile
//    ahead into a second set of registers, W fragments a block ahead; one barrier per k-tile, before its
//    last W block.
//  * Scales are loaded to LDS four k-tiles at a time (a dword a row) and read once per four k-tiles; the
//    MFMA picks the byte by an immediate, so the loop is unrolled by four.  Reading the byte itself
//    from LDS as an unaligned dword cost 40% (308 us for 4608 x 9216 x 6144 with GELU against 223).
#include "gemm_tile.h"
#include "tp_block_internal.h"

namespace tpl {
namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
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

// What both main loops share: S LDS stages of X and W tiles (rows of 128 codes, 16-byte chunk c of
// row r at c ^ ((r >> 1) & 7)), the loads that fill them, and the scales.  k-tile u is in stage
// u % S; past the last k-tile the loads repeat it into a stage that is never read again.
template <int NXB, int NWB, bool GATED, int S>
struct Feed {
    static constexpr int WM = 16 * NXB, WN = 16 * NWB, BM = 2 * WM, BN = 2 * WN;
    static constexpr int kXBytes = BM * kRow, kWBytes = BN * kRow;
    static constexpr int kDmaX = BM / 32, kDmaW = BN / 32, kDma = kDmaX + kDmaW;  // per lane and k-tile
    static constexpr int kLdsBytes = S * (kXBytes + kWBytes) + 4096;
    static_assert(!GATED || NWB == 8, "the gated tile pairs four gate and four up blocks per wave");

    char *base;
    const char *xbase, *wbase, *xsbase, *wsbase;
    uint32_t xoff[kDmaX], woff[kDmaW], xsoff, wsoff;
    int wave, T, groups;
    const char *xl, *wl, *xsl, *wsl;  // the lane's first row in the X and W tiles, and of its scales

    __device__ __forceinline__ Feed(const Fp8Params &p, char *lds, const Ctx &c, int m0, int n0)
    {
        base = lds;
        wave = c.wave;
        T = p.K / kRow;
        groups = (T + 3) / 4;
        xbase = reinterpret_cast<const char *>(p.x);
        wbase = reinterpret_cast<const char *>(p.w);
        xsbase = reinterpret_cast<const char *>(p.xs);
        wsbase = reinterpret_cast<const char *>(p.ws);
        // Load j of wave w fills tile rows 32 j + 8 w + [0, 8): lane l lands at row l / 8, position
        // l % 8, so it fetches chunk (l % 8) ^ ((row >> 1) & 7).  Rows past the end repeat the last
        // one (computed and discarded).
        const int row = c.wave * 8 + (c.lane >> 3);
        const int chunk = (c.lane & 7) ^ ((((c.wave & 1) << 2) + (c.lane >> 4)) & 7);
        // GATED: tile row 128 q + 64 h + i is W[h N + n0 + 64 q + i], so wave column q's blocks 0-3 hold
        // the gate rows and blocks 4-7 the up rows of outputs n0 + 64 q + [0, 64).
        const auto wrow = [&](int r) {
            return GATED ? ((r >> 6) & 1) * p.N + min(n0 + 64 * (r >> 7) + (r & 63), p.N - 1) : min(n0 + r, p.N - 1);
        };
#pragma unroll
        for (int j = 0; j < kDmaX; ++j)
            xoff[j] = (uint32_t)min(m0 + 32 * j + row, p.M - 1) * (uint32_t)p.ldx + chunk * 16;
#pragma unroll
        for (int j = 0; j < kDmaW; ++j)
            woff[j] = (uint32_t)wrow(32 * j + row) * (uint32_t)p.ldw + chunk * 16;
        // Scales: a dword holds a row's scales of four k-tiles.  Lane l of wave w loads row 64 w + l of
        // the X tile and of the W tile; group u / 4 goes into buffer (u / 4) % 2.
        const int srow = c.wave * 64 + c.lane;
        xsoff = (uint32_t)min(m0 + min(srow, BM - 1), p.M - 1) * (uint32_t)p.ldxs;
        wsoff = (uint32_t)wrow(min(srow, BN - 1)) * (uint32_t)p.ldws;
        const int fr = c.lane & 15;
        xl = base + (c.wave_m * WM + fr) * kRow;
        wl = base + S * kXBytes + (c.wave_n * WN + fr) * kRow;
        xsl = base + S * (kXBytes + kWBytes) + (c.wave_m * WM + fr) * 4;
        wsl = base + S * (kXBytes + kWBytes) + 1024 + (c.wave_n * WN + fr) * 4;
    }
    __device__ __forceinline__ void dma_x(int d, int u, int stage) const
    {
        dma16_sbase(xbase + min(u, T - 1) * kRow, xoff[d],
                    reinterpret_cast<uint16_t *>(base + stage * kXBytes + (d * 4 + wave) * 1024));
    }
    __device__ __forceinline__ void dma_w(int d, int u, int stage) const
    {
        dma16_sbase(wbase + min(u, T - 1) * kRow, woff[d],
                    reinterpret_cast<uint16_t *>(base + S * kXBytes + stage * kWBytes + (d * 4 + wave) * 1024));
    }
    __device__ __forceinline__ void dma_scales(int group) const
    {
        char *d = base + S * (kXBytes + kWBytes) + (group & 1) * 2048 + wave * 256;
        const int at = 4 * min(group, groups - 1);
        dma4_sbase(xsbase + at, xsoff, d);
        dma4_sbase(wsbase + at, wsoff, d + 1024);
    }
    // The scale dword of a block's row, from xsl or wsl.
    __device__ __forceinline__ static uint32_t scale(const char *t, int buf, int block)
    {
        return *reinterpret_cast<const uint32_t *>(t + buf * 2048 + block * 64);
    }
};

// An offset that the compiler cannot see through, so that it keeps this one value rather than an
// address for every block and stage that it is added to.
__device__ __forceinline__ int opaque(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// acc += X[m0 .., :] . W[n0 .., :]^T on the 8-bit matrix cores.
template <int NXB, int NWB, bool GATED, int S>
__device__ __forceinline__ void mainloop8(const Fp8Params &p, char *lds, const Ctx &c, int m0, int n0,
                                          f32x4 (&acc)[NXB][NWB])
{
    typedef Feed<NXB, NWB, GATED, S> F;
    constexpr int kDmaW = F::kDmaW, kDma = F::kDma;
    constexpr int kMfma = NXB * NWB, kLast = kMfma - NXB;  // first MFMA of the last W block
    constexpr int RS = (NWB - 1) / 2;                      // X reads: one every RS MFMAs
    constexpr int DS = 2;                                  // loads: one every DS MFMAs after the barrier
    constexpr int kF = NXB / DS;                           // loads issued within the last W block
    static_assert(NWB % 2 == 0 && (2 * NXB - 1) * RS < kLast, "reads fit");
    static_assert(NXB >= 5, "the scale reads are placed within a W block");
    const F f(p, lds, c, m0, n0);
    const int T = f.T;
    // load d of the step after barrier u: W of k-tile u + S into the stage of k-tile u, X of k-tile
    // u + S + 1 into that of k-tile u + 1 (whose X fragments every wave has read by then)
    auto dma = [&](int d, int u, int stage, int next) {
        if (d < kDmaW)
            f.dma_w(d, u + S, stage);
        else
            f.dma_x(d - kDmaW, u + S + 1, next);
    };
    // Fragments: lane l holds 32 codes of row l % 16 of a block, chunks l / 16 and 4 + l / 16.  Which
    // features these are does not matter, as both operands take the same ones.
    const int g = c.lane >> 4, swz = (c.lane >> 1) & 7;
    const int c0 = (g ^ swz) * 16, c1 = ((4 + g) ^ swz) * 16;
    // the lane's first chunks in a tile of a stage
    struct At {
        const char *half[2];
    };
    auto at = [&](const char *t, int stage, int bytes) {
        const int o = stage * bytes;
        return S > 2 ? At{{t + opaque(o + c0), t + opaque(o + c1)}} : At{{t + o + c0, t + o + c1}};
    };
    auto read = [&](const At &a, int block, int half) {
        return *reinterpret_cast<const i32x4 *>(a.half[half] + block * 16 * kRow);
    };
    auto set = [](i32x8 &f, int half, i32x4 v) {
        if (half == 0)
            f = __builtin_shufflevector(__builtin_shufflevector(v, v, 0, 1, 2, 3, 0, 1, 2, 3), f, 0, 1, 2, 3, 12, 13, 14, 15);
        else
            f = __builtin_shufflevector(f, __builtin_shufflevector(v, v, 0, 1, 2, 3, 0, 1, 2, 3), 0, 1, 2, 3, 8, 9, 10, 11);
    };
    uint32_t sx[NXB], sw[NWB];

    // prologue: what the first S - 1 k-tiles read
    i32x8 fa[NXB] = {}, fb[NXB] = {}, fw[2] = {};
    f.dma_scales(0);
#pragma unroll
    for (int d = 0; d < F::kDmaX; ++d)
        f.dma_x(d, 0, 0);
#pragma unroll
    for (int u = 0; u < S - 1; ++u) {
#pragma unroll
        for (int d = 0; d < kDmaW; ++d)
            f.dma_w(d, u, u);
#pragma unroll
        for (int d = 0; d < F::kDmaX; ++d)
            f.dma_x(d, u + 1, u + 1);
    }
    wait_dma_keep<(S - 2) * kDma>();
    barrier_only();
#pragma unroll
    for (int i = 0; i < NXB; ++i) {
        set(fa[i], 0, read(at(f.xl, 0, 0), i, 0));
        set(fa[i], 1, read(at(f.xl, 0, 0), i, 1));
        sx[i] = F::scale(f.xsl, 0, i);
    }
    set(fw[0], 0, read(at(f.wl, 0, 0), 0, 0));
    set(fw[0], 1, read(at(f.wl, 0, 0), 0, 1));
#pragma unroll
    for (int j = 0; j < NWB; ++j)
        sw[j] = F::scale(f.wsl, 0, j);
    wait_dma_keep<(S - 2) * kDma>();
    barrier_only();
#pragma unroll
    for (int d = 0; d < kF; ++d)
        dma(d, -1, S - 1, 0);
    int before = S - 1, stage = 0, after = 1;  // stages of k-tiles t - 1, t, t + 1
    int t = 0;
    // k-tile t, with T4 = t % 4
    auto body = [&](i32x8 (&cur)[NXB], i32x8 (&nxt)[NXB], auto T4) __attribute__((always_inline)) {
        constexpr int st = decltype(T4)::value;
        // three stages: uniform values that the compiler has to be told are uniform
        const int s0 = S == 2 ? st & 1 : __builtin_amdgcn_readfirstlane(stage);
        const int s1 = S == 2 ? (st & 1) ^ 1 : __builtin_amdgcn_readfirstlane(after);
        const int sb = S == 2 ? s1 : __builtin_amdgcn_readfirstlane(before);
        const At xn = at(f.xl, s1, F::kXBytes);  // X of k-tile t + 1
        const At wc = at(f.wl, s0, F::kWBytes), wn = at(f.wl, s1, F::kWBytes);
        const int buf = (t >> 2) & 1;  // of this k-tile's scales
        each([&](auto Q) __attribute__((always_inline)) {
            constexpr int q = decltype(Q)::value, j = q / NXB, i = q % NXB;
            if constexpr (q == kLast) {  // W of k-tile t + 1 and X of k-tile t + 2 have landed
                wait_dma_keep<(S - 2) * kDma>();
                barrier_only();
            }
            scaled_mfma<st>(acc[i][j], fw[j & 1], cur[i], sw[j], sx[i]);
            // loads: the rest of the step after the previous barrier, then the first of this one's
            if constexpr (q < kLast) {
                if constexpr (q % DS == 0 && kF + q / DS < kDma)
                    dma(kF + q / DS, t - 1, sb, s0);
            } else if constexpr ((q - kLast) % DS == 0 && (q - kLast) / DS < kF) {
                dma((q - kLast) / DS, t, s0, s1);
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
                sx[NXB - 1] = F::scale(f.xsl, buf, NXB - 1);
            if constexpr (st == 0 && q == 4)
                sw[NWB - 1] = F::scale(f.wsl, buf, NWB - 1);
            if constexpr (st == 3 && q > kLast)
                sx[i - 1] = F::scale(f.xsl, buf ^ 1, i - 1);
            if constexpr (st == 3 && j > 0 && i == 4)
                sw[j - 1] = F::scale(f.wsl, buf ^ 1, j - 1);
            if constexpr (st == 1 && q == NXB)
                f.dma_scales(t / 4 + 1);
        }, std::make_integer_sequence<int, kMfma>{});
        before = stage;
        stage = after;
        after = after == S - 1 ? 0 : after + 1;
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
}

// acc += w . x^T over 32 features in bf16.
__device__ __forceinline__ void exact_mfma(f32x4 &acc, const i32x4 &w, const i32x4 &x)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(w), "v"(x) : "memory");
}

// Features 2 E and 2 E + 1 of eight codes, times 2^(exponent of s), as bf16 (exact).
template <int E>
__device__ __forceinline__ void widen2(i32x4 &d, const i32x2 &codes, uint32_t s)
{
    int v;
    if constexpr (E % 2 == 0)
        asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2" : "=v"(v) : "v"(codes[E / 2]), "v"(s));
    else
        asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2 op_sel:[1,0,0]" : "=v"(v) : "v"(codes[E / 2]), "v"(s));
    d[E] = v;
}

// Which W fragment slot q of a step of the exact main loop converts: 2 b + half, or -1.  Fragment b
// takes the two slots from kCw + 2 b on, but not before the second after its last use (MFMA
// NXB (b + 1) - 1); the last fragment is converted elsewhere.
constexpr int w_conversion(int q, int nxb, int nwb, int kcw)
{
    for (int b = 0; b < nwb - 1; ++b) {
        const int from = kcw + 2 * b > nxb * (b + 1) + 1 ? kcw + 2 * b : nxb * (b + 1) + 1;
        if (q == from || q == from + 1)
            return 2 * b + (q - from);
    }
    return -1;
}

// acc += X[m0 .., :] . W[n0 .., :]^T with exact products: codes widened to bf16 times their scale (four
// significant bits and a power of two: exact), v_mfma_f32_16x16x32_bf16.
//
// A k-tile is four steps of 32 features; MFMA q of a step takes W block q / NXB and X block q % NXB.
// Beside the MFMAs a step reads the next step's codes (8 bytes a lane and block) and widens them: the
// X fragments into a second set of registers, each W fragment in place after its last use, the last
// one at the start of its own step.  Every instruction is placed by hand: an MFMA must not follow
// within two wait states of a conversion that writes its operand, which the compiler does not check
// for instructions written as assembly; here at least two MFMAs lie between them.
template <int NXB, int NWB, bool GATED>
__device__ __forceinline__ void mainloop_exact(const Fp8Params &p, char *lds, const Ctx &c, int m0, int n0,
                                               f32x4 (&acc)[NXB][NWB])
{
    typedef Feed<NXB, NWB, GATED, 2> F;
    constexpr int kDma = F::kDma, kDmaX = F::kDmaX, kMfma = NXB * NWB;
    constexpr int kCx = NXB + NWB - 4;                    // slot of the first X conversions, two a slot
    constexpr int kCw = kCx + 2 * NXB;                    // and of the W conversions
    constexpr int kD0 = kDma / 2, kD1 = kDma - kD0;       // loads of a k-tile in its step 3 and step 0
    static_assert(NXB >= 6 && NWB >= 6 && kCw + NXB + NWB <= kMfma, "the reads and conversions fit in a step");
    static_assert(w_conversion(NXB * (NWB - 1) + 2, NXB, NWB, kCw) == 2 * (NWB - 2) + 1 && NXB * (NWB - 1) + 2 < kMfma,
                  "the last in-place W conversion ends within the step");
    const F f(p, lds, c, m0, n0);
    const int T = f.T;
    auto dma = [&](int d, int u, int stage) {
        if (d < kDmaX)
            f.dma_x(d, u, stage);
        else
            f.dma_w(d - kDmaX, u, stage);
    };
    // Step s: lanes 16 g .. 16 g + 15 take half g % 2 of chunk 2 s + g / 2 of their rows, so 32 neighbouring
    // lanes read whole chunks and meet every LDS bank once.
    const int g = c.lane >> 4, swz = (c.lane >> 1) & 7;
    int at[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        at[s] = ((2 * s + (g >> 1)) ^ swz) * 16 + 8 * (g & 1);
    auto read_x = [&](int i, int s, int stage) {
        return *reinterpret_cast<const i32x2 *>(f.xl + at[s] + (stage * F::kXBytes + i * 16 * kRow));
    };
    auto read_w = [&](int j, int s, int stage) {
        return *reinterpret_cast<const i32x2 *>(f.wl + at[s] + (stage * F::kWBytes + j * 16 * kRow));
    };
    // the scale byte of k-tile u % 4 as an fp32 exponent (the conversion looks at nothing else)
    auto factor = [](uint32_t d, int u) { return (d >> (8 * (u & 3))) << 23; };
    i32x4 fa[NXB] = {}, fb[NXB] = {}, fw[NWB] = {};
    i32x2 rx[NXB], rw[NWB];
    uint32_t sx[NXB], sw[NWB], dx[NXB], dw[NWB];

#pragma unroll
    for (int d = 0; d < kDma; ++d)
        dma(d, 0, 0);
    f.dma_scales(0);
    wait_dma_keep<0>();
    barrier_only();
#pragma unroll
    for (int i = 0; i < NXB; ++i) {
        rx[i] = read_x(i, 0, 0);
        dx[i] = F::scale(f.xsl, 0, i);
        sx[i] = factor(dx[i], 0);
    }
#pragma unroll
    for (int j = 0; j < NWB; ++j) {
        rw[j] = read_w(j, 0, 0);
        dw[j] = F::scale(f.wsl, 0, j);
        sw[j] = factor(dw[j], 0);
    }
    each([&](auto E) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NXB; ++i)
            widen2<decltype(E)::value>(fa[i], rx[i], sx[i]);
#pragma unroll
        for (int j = 0; j < NWB - 1; ++j)
            widen2<decltype(E)::value>(fw[j], rw[j], sw[j]);
    }, std::make_integer_sequence<int, 4>{});
#pragma unroll
    for (int d = 0; d < kD0; ++d)
        dma(d, 1, 1);
    asm volatile("s_nop 1" ::: "memory");
    int t = 0;
    auto step = [&](i32x4 (&cur)[NXB], i32x4 (&nxt)[NXB], auto S, auto PAR) __attribute__((always_inline)) {
        constexpr int s = decltype(S)::value, par = decltype(PAR)::value;
        constexpr int sn = (s + 1) % 4, stage = s == 3 ? par ^ 1 : par;  // where the next step's codes are
        if constexpr (s == 3) {  // k-tile t + 1 has landed, and k-tile t has been read by every wave
            wait_dma_keep<0>();
            barrier_only();
        }
        if constexpr (s == 1) {
            if ((t & 3) == 1)
                f.dma_scales(t / 4 + 1);
        }
        each([&](auto Q) __attribute__((always_inline)) {
            constexpr int q = decltype(Q)::value, j = q / NXB, i = q % NXB;
            exact_mfma(acc[i][j], fw[j], cur[i]);
            // the next step's codes
            if constexpr (q < NXB)
                rx[q] = read_x(q, sn, stage);
            else if constexpr (q < NXB + NWB)
                rw[q - NXB] = read_w(q - NXB, sn, stage);
            // k-tile t + 2 into k-tile t's stage: half of the loads here, half in the next k-tile's step 0
            if constexpr (s == 3 && q % (kMfma / kD0) == 1 && q / (kMfma / kD0) < kD0)
                dma(q / (kMfma / kD0), t + 2, par);
            if constexpr (s == 0 && q % (kMfma / kD1) == 1 && q / (kMfma / kD1) < kD1)
                dma(kD0 + q / (kMfma / kD1), t + 1, par ^ 1);
            // the next k-tile's scales: dwords in step 2, factors in step 3
            if constexpr (s == 2 && q >= kCw && q < kCw + NXB)
                dx[q - kCw] = F::scale(f.xsl, ((t + 1) >> 2) & 1, q - kCw);
            if constexpr (s == 2 && q >= kCw + NXB && q < kCw + NXB + NWB)
                dw[q - kCw - NXB] = F::scale(f.wsl, ((t + 1) >> 2) & 1, q - kCw - NXB);
            if constexpr (s == 3 && q < NXB)
                sx[q] = factor(dx[q], t + 1);
            if constexpr (s == 3 && q >= NXB && q < NXB + NWB)
                sw[q - NXB] = factor(dw[q - NXB], t + 1);
            // conversions: the last W fragment of this step, then the next step's
            if constexpr (q < 4)
                widen2<q>(fw[NWB - 1], rw[NWB - 1], sw[NWB - 1]);
            if constexpr (q >= kCx && q < kCw) {
                constexpr int b = (q - kCx) / 2, e = (q - kCx) % 2 * 2;
                widen2<e>(nxt[b], rx[b], sx[b]);
                widen2<e + 1>(nxt[b], rx[b], sx[b]);
            }
            constexpr int wc = w_conversion(q, NXB, NWB, kCw);
            if constexpr (wc >= 0) {
                widen2<wc % 2 * 2>(fw[wc / 2], rw[wc / 2], sw[wc / 2]);
                widen2<wc % 2 * 2 + 1>(fw[wc / 2], rw[wc / 2], sw[wc / 2]);
            }
        }, std::make_integer_sequence<int, kMfma>{});
    };
    auto tile = [&](auto PAR) __attribute__((always_inline)) {
        step(fa, fb, std::integral_constant<int, 0>{}, PAR);
        step(fb, fa, std::integral_constant<int, 1>{}, PAR);
        step(fa, fb, std::integral_constant<int, 2>{}, PAR);
        step(fb, fa, std::integral_constant<int, 3>{}, PAR);
    };
    for (;;) {
        tile(std::integral_constant<int, 0>{});
        if (++t == T)
            break;
        tile(std::integral_constant<int, 1>{});
        if (++t == T)
            break;
    }
}

// The last loads and MFMAs of a main loop, before the LDS is reused and the accumulators are read as
// ordinary values; the empty statements keep every such read after the wait.
template <int NXB, int NWB>
__device__ __forceinline__ void finish(f32x4 (&acc)[NXB][NWB])
{
    wait_dma();
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < NXB; ++i)
#pragma unroll
        for (int j = 0; j < NWB; ++j)
            asm volatile("" : "+a"(acc[i][j]));
}

template <int NXB, int NWB, bool EXACT, bool HAS_BIAS, int ACT>
__global__ __launch_bounds__(kThreads8) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_nt_kernel(Fp8Params p)
{
    constexpr bool kGated = ACT == kActSwiglu;
    constexpr int BM = 32 * NXB, BN = 32 * NWB, kTileCols = kGated ? BN / 2 : BN;
    // Three stages where they fit in the 160 KiB of LDS (224 x 192 and 192 x 192: 512 x 9216 x 6144 in
    // 192 x 192 takes 46 us against 60 with two).  The exact products take twice as long to cover a
    // k-tile's loads, and gain nothing (1024 x 4608 x 6144 in 192 x 192: 73 us against 70).
    constexpr int S = !EXACT && Feed<NXB, NWB, kGated, 3>::kLdsBytes <= 160 * 1024 ? 3 : 2;
    __shared__ __attribute__((aligned(1024))) char lds[Feed<NXB, NWB, kGated, S>::kLdsBytes];
    Ctx c;
    c.lane = threadIdx.x & 63;
    c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c.wave_m = c.wave >> 1;
    c.wave_n = c.wave & 1;
    int tm, tn;
    tile_of(xcd_contiguous(blockIdx.x, p.tiles_m * p.tiles_n), p, tm, tn);
    f32x4 acc[NXB][NWB];
    zero<NXB, NWB>(acc);
    if constexpr (EXACT)
        mainloop_exact<NXB, NWB, kGated>(p, lds, c, tm * BM, tn * kTileCols, acc);
    else
        mainloop8<NXB, NWB, kGated, S>(p, lds, c, tm * BM, tn * kTileCols, acc);
    finish<NXB, NWB>(acc);
    epilogue<NXB, NWB, !EXACT, HAS_BIAS, ACT, true>(p, reinterpret_cast<uint16_t *>(lds), c, tm * BM, tn * kTileCols, acc);
}

template <int NXB, int NWB, bool EXACT, bool HAS_BIAS, int ACT>
hipError_t launch_tile(Fp8Params gp, hipStream_t stream)
{
    const int cols = ACT == kActSwiglu ? 16 * NWB : 32 * NWB;
    gp.tiles_n = (gp.N + cols - 1) / cols;
    gp.tiles_m = (gp.M + 32 * NXB - 1) / (32 * NXB);
    gp.group_m = gp.tiles_m < 8 ? gp.tiles_m : 8;
    hipLaunchKernelGGL((gemm_fp8_nt_kernel<NXB, NWB, EXACT, HAS_BIAS, ACT>), dim3(gp.tiles_m * gp.tiles_n), dim3(kThreads8),
                       0, stream, gp);
    return hipGetLastError();
}

// The shapes that exist: 256 x 256 and 224 x 256 for all, 192 x 192 and (8-bit) 224 x 192 without
// SwiGLU, 192 x 256 for 8-bit SwiGLU.
template <bool EXACT, bool HAS_BIAS, int ACT>
hipError_t launch_shape(const Fp8Params &gp, int nxb, int nwb, hipStream_t stream)
{
    if (nxb == 7 && nwb == 8)
        return launch_tile<7, 8, EXACT, HAS_BIAS, ACT>(gp, stream);
    if constexpr (ACT != kActSwiglu) {
        if (nxb == 6 && nwb == 6)
            return launch_tile<6, 6, EXACT, HAS_BIAS, ACT>(gp, stream);
        if constexpr (!EXACT)
            if (nxb == 7 && nwb == 6)
                return launch_tile<7, 6, EXACT, HAS_BIAS, ACT>(gp, stream);
    } else if constexpr (!EXACT) {
        if (nxb == 6 && nwb == 8)
            return launch_tile<6, 8, EXACT, HAS_BIAS, ACT>(gp, stream);
    }
    return launch_tile<8, 8, EXACT, HAS_BIAS, ACT>(gp, stream);
}

template <bool EXACT, bool HAS_BIAS>
hipError_t launch_act(const Fp8Params &gp, int act, int nxb, int nwb, hipStream_t stream)
{
    switch (act) {
    case kActGelu: return launch_shape<EXACT, HAS_BIAS, kActGelu>(gp, nxb, nwb, stream);
    case kActSwiglu: return launch_shape<EXACT, HAS_BIAS, kActSwiglu>(gp, nxb, nwb, stream);
    default: return launch_shape<EXACT, HAS_BIAS, kActNone>(gp, nxb, nwb, stream);
    }
}

}  // namespace

hipError_t launch_gemm_fp8_tiled(const Fp8Problem &pr, int nxb, int nwb, hipStream_t stream)
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
    if (pr.out_bf16)
        return pr.bias ? launch_act<false, true>(gp, act, nxb, nwb, stream) : launch_act<false, false>(gp, act, nxb, nwb, stream);
    return pr.bias ? launch_act<true, true>(gp, act, nxb, nwb, stream) : launch_act<true, false>(gp, act, nxb, nwb, stream);
}

}  // namespace tpl
