// gemm_fp8.hip -- which kernel runs a product of quantized rows (e4m3 codes, e8m0 scale per 128
// features):
//
//   y[m, n] = sum_b 2^(sx[m,b] + sw[n,b]) sum_{k in block b} x[m,k] w[n,k]
//
// Few rows or few outputs take the split-K kernel (gemm_fp8_narrow.hip), a few hundred rows the
// eight-wave tiles (gemm_fp8_small.hip), more the four-wave tiles (gemm_fp8_tiled.hip).
#include "tp_block_internal.h"

namespace tpl {
namespace {

// Tiles for what the split-K kernel leaves: the candidate with the least
// (0.2 r + 0.8 ceil r) x (time of one round), r = rounds of tiles over the CUs, at least 1 (a partly
// filled last round runs a little faster than a full one).  The times are those of K = 6144 in us,
// between a lone round with its weights in HBM and full rounds; the choice was checked against sweeps of
// every shape, 97 to 8192 rows, K 640 to 8192.  bf16 output (8-bit products): 4608 x 9216 x 6144 takes
// 224 x 256 (2.95 rounds, 184 us against 190 in 256 x 256 and 219 in 192 x 192), 4608 x 2304 x 6144 224 x 192
// (one round, 57 us against 81 in 192 x 192), 8192^3 256 x 256 (369 against 393 in 224 x 256).  fp32 output (exact
// products): 4608 x 6144 x 4608 takes 224 x 256 (174 us against 183 in 256 x 256 and 182 in 192 x
// 192), 1024 x 4608 x 6144 192 x 192 (71 against 99 in 224 x 256 and 94 in 128 x 128).  The eight-wave
// tiles of 128, 96 and 64 rows by 128 columns run the few hundred rows that leave most CUs idle
// otherwise: 333 x 6144 x 4608 21 us in 96 x 128 against 24 in 128 x 128 and 34 in 192 x 192 (bf16; fp32 33,
// 38 and 54), 129 x 4608 x 6144 21 us in 64 x 128 against 44 in 192 x 192 (fp32 32 against 69).
struct TileChoice {
    int nxb, nwb;  // nwb == 2: the eight-wave kernel
};

TileChoice pick_tile(const Fp8Problem &p)
{
    struct Cand {
        int nxb, nwb;
        double time;
    };
    static const Cand kEight[] = {{8, 8, 68}, {7, 8, 64}, {7, 6, 53}, {6, 6, 45}, {4, 2, 33}, {3, 2, 28.5}, {2, 2, 24.5}};
    static const Cand kEightGated[] = {{8, 8, 68}, {7, 8, 64}, {6, 8, 62}, {4, 2, 31.5}, {3, 2, 28}, {2, 2, 24.5}};
    static const Cand kExact[] = {{8, 8, 109}, {7, 8, 99}, {6, 6, 70.5}, {4, 2, 49.5}, {3, 2, 41}, {2, 2, 33.5}};
    static const Cand kExactGated[] = {{8, 8, 109}, {7, 8, 99}, {4, 2, 49.5}, {3, 2, 41}, {2, 2, 33.5}};
    const Cand *first = p.out_bf16 ? (p.swiglu ? kEightGated : kEight) : (p.swiglu ? kExactGated : kExact);
    const int count = p.out_bf16 ? (p.swiglu ? 6 : 7) : (p.swiglu ? 5 : 6);
    const int cus = cu_count();
    TileChoice best{8, 8};
    double best_cost = -1;
    for (const Cand *c = first; c < first + count; ++c) {
        const int bm = 32 * c->nxb, bn = c->nwb == 2 ? 128 : 32 * c->nwb, cols = p.swiglu ? bn / 2 : bn;
        const int64_t tiles = (p.M + bm - 1) / bm * ((p.N + cols - 1) / cols);
        if (tiles > ((int64_t)1 << 22))
            continue;  // the launch's thread count must stay below 2^32 (256 x 256 always fits)
        const double r = tiles < cus ? 1.0 : (double)tiles / cus;
        const double cost = (0.2 * r + 0.8 * (double)((tiles + cus - 1) / cus)) * c->time;
        if (best_cost < 0 || cost < best_cost) {
            best = TileChoice{c->nxb, c->nwb};
            best_cost = cost;
        }
    }
    return best;
}

}  // namespace

void gemm_fp8_tile_shape(const Fp8Problem &p, int *rows, int *cols)
{
    if (gemm_fp8_narrow_takes(p)) {
        gemm_fp8_narrow_shape(p, rows, cols);
        return;
    }
    const TileChoice c = pick_tile(p);
    *rows = 32 * c.nxb;
    *cols = (c.nwb == 2 ? 128 : 32 * c.nwb) / (p.swiglu ? 2 : 1);
}

hipError_t launch_gemm_fp8(const Fp8Problem &p, hipStream_t stream)
{
    if (gemm_fp8_narrow_takes(p))
        return launch_gemm_fp8_narrow(p, stream);
    const TileChoice c = pick_tile(p);
    return c.nwb == 2 ? launch_gemm_fp8_small(p, c.nxb, stream) : launch_gemm_fp8_tiled(p, c.nxb, c.nwb, stream);
}

}  // namespace tpl
