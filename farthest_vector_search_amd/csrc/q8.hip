// q8.hip -- scores over a table held in 8 bits.
//
//   y[q][i] = xs[q] ts[i] sum_k xc[q][k] tc[i][k]
// The sum is a whole number below 2^31 (d <= 131,071 codes of -128 .. 127), taken
// exactly; it is rounded to fp32 once, multiplied by both scales there, and the
// result rounded to the output's type.  Bound by the matrix cores where queries are many
// (8,192 over 8,192 x 8,192, bf16 scores: 455 us, 383 at best, 2,870 Top/s), by reading the
// table where they are few (1 over 65,536 x 4,096: 51 us, 5.3 TB/s).
#include <type_traits>

#include "few.h"
#include "tile.h"
#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

template <typename O, int BM, int BN, int WM, int WN, int PIECE>
__global__ __launch_bounds__(WM *WN * 64, 2) void k_q8_scores(
    const int8_t *__restrict__ x, const float *__restrict__ xs, int64_t nq, int32_t d,
    const int8_t *__restrict__ t, const float *__restrict__ ts, int64_t nc, O *__restrict__ y) {
    using C = tile::Core<int8_t, BM, BN, WM, WN, false, false, PIECE>;
    __shared__ __attribute__((aligned(1024))) char bufs[2 * C::kBytes];
    const int64_t qt = (nq + BM - 1) / BM, it = (nc + BN - 1) / BN;
    tile::run_tiles<int8_t, O, C>(
        qt * it, bufs,
        [&](int64_t id, tile::Job<int8_t, O> &j) {
            int64_t at;
            if (!tile::xcd_tile(id, qt * it, at)) return false;
            const tile::Place pl = tile::place(at, qt, it);
            const int64_t q0 = pl.row * BM, i0 = pl.col * BN;
            j.depth = d;
            j.m = {x + q0 * d, d, (int)(nq - q0 < BM ? nq - q0 : BM)};
            j.n = {t + i0 * d, d, (int)(nc - i0 < BN ? nc - i0 : BN)};
            j.out = y + q0 * nc + i0;
            j.ld = nc;
            j.mscale = xs + q0;
            j.nscale = ts + i0;
            return true;
        });
}

// Few queries, 16 a turn, `groups` workgroups for each.
template <typename O, int NB>
__global__ __launch_bounds__(few::kWaves * 64) void k_q8_scores_few(
    const int8_t *__restrict__ x, const float *__restrict__ xs, int64_t nq, int32_t d,
    const int8_t *__restrict__ t, const float *__restrict__ ts, int64_t nc, O *__restrict__ y,
    int64_t groups, int share) {
    const int per = few::kWaves / share * NB * 16;
    const int64_t total = (nq + 15) / 16 * groups;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int64_t q0 = id / groups * 16, i0 = id % groups * per;
        const int qn = (int)(nq - q0 < 16 ? nq - q0 : 16);
        __syncthreads();  // the last turn's sums have been read
        few::products<int8_t, 1, NB>(
            x + q0 * d, qn, t, i0, nc, d, share, [&](int q, int64_t i, const tile::i32x4 &v) {
                const float s = xs[q0 + q];
                tile::f32x4 f;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    f[u] = (float)v[u] * s * ts[i + u < nc ? i + u : nc - 1];
                few::store4(y + (q0 + q) * nc, i, nc, f);
            });
    }
}

inline int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

template <typename O>
hipError_t q8_scores_few(const int8_t *x, const float *xs, int64_t nq, int32_t d, const int8_t *t,
                         const float *ts, int64_t nc, O *y, hipStream_t st, int n_cu) {
    const few::Deal e = few::deal(tiles_of(nc, 16), tiles_of(nq, 16), d, n_cu);
    const int64_t total = tiles_of(nq, 16) * e.groups, most = tile::kMostGroups;
    const dim3 grid((unsigned)(total < most ? total : most)), block(few::kWaves * 64);
    timing_before(st, "k_q8_scores_few");
    if (e.nb == 2)
        hipLaunchKernelGGL((k_q8_scores_few<O, 2>), grid, block, 0, st, x, xs, nq, d, t, ts, nc, y,
                           e.groups, e.share);
    else
        hipLaunchKernelGGL((k_q8_scores_few<O, 1>), grid, block, 0, st, x, xs, nq, d, t, ts, nc, y,
                           e.groups, e.share);
    timing_after(st);
    return hipGetLastError();
}

template <typename O, int BM, int BN, int WM, int WN>
hipError_t q8_scores(const int8_t *x, const float *xs, int64_t nq, int32_t d, const int8_t *t,
                     const float *ts, int64_t nc, int piece, O *y, hipStream_t st) {
    const dim3 grid(tile::grid_of(tiles_of(nq, BM) * tiles_of(nc, BN))), block(WM * WN * 64);
    auto go = [&](auto pc) {
        static const tile::FormName name("k_q8_scores", BM, BN, decltype(pc)::value);
        timing_before(st, name.text);
        hipLaunchKernelGGL((k_q8_scores<O, BM, BN, WM, WN, decltype(pc)::value>), grid, block, 0, st,
                           x, xs, nq, d, t, ts, nc, y);
        timing_after(st);
    };
    if constexpr (BM < 256) {  // the largest tile is for pieces of 16 only
        if (piece == 4) go(std::integral_constant<int, 4>());
        if (piece == 0) go(std::integral_constant<int, 0>());
    }
    if (piece == 16) go(std::integral_constant<int, 16>());
    return hipGetLastError();
}

}  // namespace

// Which kernel, in brackets us of it and of its neighbour:
//   few.h      reads the table once for every 16 queries.  Rows on 4-byte boundaries: up
//              to 4 queries (1 over 262,144 x 256: 15, 64 x 64 17); with rows of 1,024 codes
//              or more up to 16 (16 over 65,536 x 4,096: 59 and 67), and any number while
//              12,288 rows are read in all, since tiles leave most CUs idle there (256 over
//              300 x 2,048: 7.9, 64 x 64 8.4, over 1,000 x 8,192 27 and 33; 1,024 over 300 x
//              2,048: 17 and 8.4).  At other addresses its loads are the slower ones: while
//              8,192 rows are read in all, of 512 codes or more for up to 4 queries, of
//              1,024 for more (4 over 4,096 x 767: 8.0, 64 x 64 8.8, over 32,768 18 and 11.5,
//              over 4,096 x 255 9.0 and 5.7; 16 over 4,096 x 2,047: 12 and 18, over 32,768 48
//              and 24)
//   64 x 64    up to 64 queries (37 over 8,359 x 767: 10, 128 x 128 13), or too few
//              tiles of 128 x 128 for the GPU
//   128 x 128  96 over 65,536 x 4,096: 74, 64 x 64 85; 1,000 over 20,000 x 1,000: 53,
//              256 x 256 57
//   256 x 256  two tiles for every CU, rows on 16-byte boundaries (8,192 over 16,384 x
//              4,096: 500, 128 x 128 604)
hipError_t launch_q8_scores(const int8_t *x, const float *xs, int64_t nq, int32_t d,
                            const int8_t *table, const float *ts, int64_t nc, int out_dtype,
                            void *y, hipStream_t st, int n_cu) {
    // the bytes that rows move in, by the boundaries they lie on
    const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(table) |
                         (uintptr_t)d;
    const int piece = (at & 15) == 0 ? 16 : (at & 3) == 0 ? 4 : 0;
    auto tiles = [&](int b) { return tiles_of(nq, b) * tiles_of(nc, b); };
    auto go = [&](auto o) {
        using O = decltype(o);
        const int64_t reads = tiles_of(nq, 16) * nc;  // rows of the table, with few.h
        if (piece ? nq <= 4 || (d >= 1024 && (nq <= 16 || reads <= 12288))
                  : d >= (nq <= 4 ? 512 : 1024) && reads <= 8192)
            return q8_scores_few<O>(x, xs, nq, d, table, ts, nc, (O *)y, st, n_cu);
        if (piece == 16 && nq >= 192 && tiles(256) >= 2 * (int64_t)n_cu)
            return q8_scores<O, 256, 256, 2, 4>(x, xs, nq, d, table, ts, nc, piece, (O *)y, st);
        if (nq > 64 && tiles(128) >= n_cu)
            return q8_scores<O, 128, 128, 2, 2>(x, xs, nq, d, table, ts, nc, piece, (O *)y, st);
        return q8_scores<O, 64, 64, 2, 2>(x, xs, nq, d, table, ts, nc, piece, (O *)y, st);
    };
    switch (out_dtype) {
    case kF32: return go(float());
    case kF16: return go(_Float16());
    default: return go(__bf16());
    }
}

}  // namespace vs
