// gemm_tile.h -- pieces shared by the tiled GEMM kernels: tile order over the XCDs, activations,
// waits and direct-to-LDS loads of the main loops, and the epilogue through LDS.
#pragma once

#include <type_traits>

#include "tp_internal.h"

namespace tpl {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Workgroups are dealt round-robin to the 8 XCDs (block b runs on XCD b % 8).
// Renumber [0, total) so that each XCD's blocks get a contiguous run.
__device__ __forceinline__ int xcd_contiguous(int bid, int total)
{
    const int xcd = bid & 7;
    const int local = bid >> 3;
    const int per = (total + 7) >> 3;
    const int tall = total - (per - 1) * 8;  // XCDs that receive `per` blocks
    return xcd < tall ? xcd * per + local : tall * per + (xcd - tall) * (per - 1) + local;
}

// Linear tile index -> (tile row, tile column), grouped raster: group_m tile
// rows at a time, column-major inside the group.
template <typename Params>
__device__ __forceinline__ void tile_of(int lin, const Params &p, int &tm, int &tn)
{
    const int in_group = p.group_m * p.tiles_n;
    const int g = lin / in_group;
    const int first_m = g * p.group_m;
    const int gsz = min(p.tiles_m - first_m, p.group_m);
    const int r = lin - g * in_group;
    tm = first_m + r % gsz;
    tn = r / gsz;
}

// GELU, tanh form: g(v) = v/2 (1 + tanh(u)), u = sqrt(2/pi) (v + 0.044715 v^3).
// Uses 1 + tanh(u) = 2 / (1 + exp(-2u)), so g(v) = v / (1 + exp(-2u)), with
// exp(-2u) = 2^(v (a + b v^2)), a = -2 sqrt(2/pi) log2(e), b = 0.044715 a.
// The hardware exp2 and reciprocal (about 1 ulp each) replace the library
// exp and the IEEE divide: 7 instructions per element instead of about 19,
// which took 6% of a 4608 x 9216 x 6144 launch in the epilogue.  Both tails
// are exact limits (2^+inf gives v * 0 = -0, 2^-inf gives v).
__device__ __forceinline__ float gelu_tanh(float v)
{
    const float a = -2.0f * 0.7978845608028654f * 1.4426950408889634f;
    const float b = 0.044715f * a;
    const float e = __builtin_amdgcn_exp2f(v * __builtin_fmaf(b, v * v, a));
    return v * __builtin_amdgcn_rcpf(1.0f + e);
}

// SiLU (Swish): v * sigmoid(v) = v / (1 + exp(-v)) = v / (1 + 2^(-v log2(e))),
// with the hardware exp2 and reciprocal as in gelu_tanh; both tails are exact
// limits (2^+inf gives -0, 2^-inf gives v).
__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// Per-thread constants of the tile pipeline.
struct Ctx {
    int lane, wave, wave_m, wave_n;
    int dma_row, dma_chunk;       // DMA: row within a 64-row group, logical chunk
    int xrow_off, wrow_off;       // fragment row offsets inside an LDS tile
    int swz, kh;                  // fragment swizzle and k-quarter
};

// Waits until this wave's direct-to-LDS loads have written the LDS.  A
// barrier after it then publishes every wave's loads to the workgroup.  The
// compiler's own waits do not cover this in every loop shape: a k-step-32
// variant of this kernel compiled with no load wait before its barrier and read
// stale tiles.
__device__ __forceinline__ void wait_dma() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Waits until at most N of this wave's vector memory instructions are outstanding (they
// complete in issue order) and its LDS reads have returned: with N = the loads issued
// after a k-tile's, that k-tile has landed while the later ones stay in flight.
template <int N>
__device__ __forceinline__ void wait_dma_keep()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// A workgroup barrier without the release fence of __syncthreads(), which would wait for
// every outstanding load, the ones meant to stay in flight included.  The caller waits
// for what must be complete first; the empty asm statements keep the compiler from moving
// memory accesses across it.
__device__ __forceinline__ void barrier_only()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// One 16-byte direct-to-LDS load per lane in its scalar-base form: a wave-uniform base
// address plus the lane's 32-bit byte offset, with the LDS address of the wave's 1 KiB
// destination in M0 (lane l writes 16 l bytes after it).  The builtin forms a 64-bit lane
// address with two VALU instructions per load, which the single wave of a SIMD issues
// between its MFMAs.  The load writes no register; the caller waits for it with an explicit
// vmcnt wait before the barrier that publishes its data.  No other code of the kernel uses
// M0, so clobbering it here is safe.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_sbase(const char *base, uint32_t off, uint16_t *dst)
{
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t *)dst;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m0), "v"(off), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

template <int NXB, int NWB>
__device__ __forceinline__ void zero(f32x4 (&acc)[NXB][NWB])
{
#pragma unroll
    for (int i = 0; i < NXB; ++i)
#pragma unroll
        for (int j = 0; j < NWB; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Epilogue activations.
constexpr int kActNone = 0;
constexpr int kActGelu = 1;
constexpr int kActSwiglu = 2;  // W tile = interleaved [gate; up] 64-row blocks, see mainloop4

// Epilogue through LDS.  Lane l holds Y[m][n..n+3] for m = row base +
// 16 i + l%16 and n = column base + 16 j + 4 (l / 16).  For each of the
// wave's 16-row slices the wave writes its output values (after bias /
// activation / rounding) into a private LDS area with padded rows, then
// reads them back row-major and stores whole row segments.  A wave owns 16 NWB
// output columns, or 8 NWB with SwiGLU: there its blocks j < NWB / 2 hold the gate
// and j >= NWB / 2 the up projection of the same columns, and the output is
// silu(gate + b_gate) * (up + b_up), the bias being [b_gate; b_up] (2 N).
template <int NXB, int NWB, bool OUT_BF16, bool HAS_BIAS, int ACT, bool BIAS_AHEAD = false, typename Params>
__device__ __forceinline__ void epilogue(const Params &p, uint16_t *lds, const Ctx &c, int m0, int n0,
                                         const f32x4 (&acc)[NXB][NWB])
{
    __syncthreads();  // every wave is done reading the operand stages
    typedef typename std::conditional<OUT_BF16, __bf16, float>::type OutT;
    constexpr bool kGated = ACT == kActSwiglu;
    static_assert(!kGated || NWB % 2 == 0, "the gated epilogue pairs NWB / 2 gate and up blocks");
    constexpr int WNO = kGated ? 8 * NWB : 16 * NWB;  // output columns per wave
    constexpr int JO = WNO / 16;               // 16-column output blocks per wave
    constexpr int kOutEs = sizeof(OutT);
    constexpr int kRowElems = WNO + 16 / kOutEs;  // one 16-byte pad per row
    OutT *stage = reinterpret_cast<OutT *>(lds) + c.wave * 16 * kRowElems;
    // The lane's terms are derived here from an opaque copy of the thread index, so the
    // compiler cannot keep them live through the main loop (at 256 registers the 256-row
    // tiles would spill them).
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63;
    const int mrow = lane & 15;
    const int ncol = 4 * (lane >> 4);
    auto bias4 = [&](int e) {
        const bf16x4 bb = *reinterpret_cast<const bf16x4 *>(p.bias + e);
        return f32x4{(float)bb[0], (float)bb[1], (float)bb[2], (float)bb[3]};
    };
    // BIAS_AHEAD: the wave's bias values in registers before the first slice.  Loaded where they are
    // used, each slice waits for them again, as the output's stores might change them.  Columns past
    // the end take the last ones' and are added like the others, without a branch (4608 x 9216 x 6144
    // with GELU in 8-bit products: 3 us less in three rounds of tiles).
    bf16x4 bias_v[kGated ? 2 : 1][JO];
    if constexpr (HAS_BIAS && BIAS_AHEAD) {
#pragma unroll
        for (int j = 0; j < JO; ++j) {
            const int n = min(n0 + c.wave_n * WNO + j * 16 + ncol, p.N - 4);
            bias_v[0][j] = *reinterpret_cast<const bf16x4 *>(p.bias + n);
            if constexpr (kGated)
                bias_v[1][j] = *reinterpret_cast<const bf16x4 *>(p.bias + p.N + n);
        }
    }
    auto bias_of = [&](int up, int j, int n) {
        if constexpr (BIAS_AHEAD) {
            const bf16x4 bb = bias_v[up][j];
            return f32x4{(float)bb[0], (float)bb[1], (float)bb[2], (float)bb[3]};
        } else {
            return bias4(up * p.N + n);
        }
    };
    constexpr int kVec = 16 / kOutEs;              // elements per 16-byte vector
    constexpr int kVecPerRow = WNO / kVec;
    // When a pass of 64 lanes covers whole rows, each lane keeps its row and column for
    // every pass; otherwise (48 output columns per wave) a lane's position moves per pass.
    constexpr bool kWholeRows = 64 % kVecPerRow == 0;
    constexpr int kRowsPerPass = kWholeRows ? 64 / kVecPerRow : 1;  // over 16: lanes past row 15 sit out
    constexpr int kPasses = (16 * kVecPerRow + 63) / 64;
    const int rd_row = lane / kVecPerRow;
    const int rd_vec = lane % kVecPerRow;
    const int64_t lane_off = (int64_t)rd_row * p.ldy + rd_vec * kVec;
#pragma unroll
    for (int i = 0; i < NXB; ++i) {
#pragma unroll
        for (int j = 0; j < JO; ++j) {
            const int n = n0 + c.wave_n * WNO + j * 16 + ncol;  // N % 16 == 0: n < N covers n + 3
            f32x4 v = acc[i][j];
            if (HAS_BIAS && (BIAS_AHEAD || n < p.N))
                v = v + bias_of(0, j, n);
            if (ACT == kActGelu) {
                v[0] = gelu_tanh(v[0]);
                v[1] = gelu_tanh(v[1]);
                v[2] = gelu_tanh(v[2]);
                v[3] = gelu_tanh(v[3]);
            }
            if (kGated) {
                f32x4 u = acc[i][j + NWB / 2];
                if (HAS_BIAS && (BIAS_AHEAD || n < p.N))
                    u = u + bias_of(1, j, n);
                v[0] = silu(v[0]) * u[0];
                v[1] = silu(v[1]) * u[1];
                v[2] = silu(v[2]) * u[2];
                v[3] = silu(v[3]) * u[3];
            }
            OutT *dst = stage + mrow * kRowElems + j * 16 + ncol;
            if (OUT_BF16)
                *reinterpret_cast<bf16x4 *>(dst) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
            else
                *reinterpret_cast<f32x4 *>(dst) = v;
        }
        // Row r + rd_row of the slice: the row's base and bound are wave-uniform, the lane's
        // offset is fixed, so no per-row lane value stays live across the unrolled passes.
        const int mbase = m0 + c.wave_m * 16 * NXB + i * 16;
        OutT *ybase = reinterpret_cast<OutT *>(p.y) + n0 + c.wave_n * WNO;
        if constexpr (kWholeRows) {
            const bool col_ok = n0 + c.wave_n * WNO + rd_vec * kVec < p.N;
#pragma unroll
            for (int r = 0; r < 16; r += kRowsPerPass) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(stage + (r + (kRowsPerPass <= 16 ? rd_row : (rd_row & 15))) * kRowElems +
                                                                 rd_vec * kVec);
                // Non-temporal stores: about 1% faster than ordinary ones over a DiT block's
                // GEMMs, with the same fetched and written bytes.
                if ((kRowsPerPass <= 16 || rd_row < 16) && rd_row < p.M - (mbase + r) && col_ok)
                    __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(ybase + (int64_t)(mbase + r) * p.ldy + lane_off));
            }
        } else {
#pragma unroll
            for (int q = 0; q < kPasses; ++q) {
                const int e = lane + 64 * q;        // vector e of the slice: row e / kVecPerRow
                const int row = e / kVecPerRow;
                const int vec = e - row * kVecPerRow;
                if (row < 16) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(stage + row * kRowElems + vec * kVec);
                    if (row < p.M - mbase && n0 + c.wave_n * WNO + vec * kVec < p.N)
                        __builtin_nontemporal_store(
                            v, reinterpret_cast<f32x4 *>(ybase + (int64_t)(mbase + row) * p.ldy + vec * kVec));
                }
            }
        }
    }
}

}  // namespace
}  // namespace tpl
