// q8.hip -- scores over a table held in 8 bits.
//
//   y[q][i] = xs[q] ts[i] sum_k xc[q][k] tc[i][k]
// The sum is a whole number below 2^31 (d <= 131,071 codes of -128 .. 127), taken
// exactly; it is rounded to fp32 once, multiplied by both scales there, and the
// result rounded to the output's type.
#include <type_traits>

#include "tile.h"
#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

template <typename O, int BM, int BN, int WM, int WN, bool ALIGNED>
__global__ __launch_bounds__(WM *WN * 64, BM * BN > 128 * 128 ? 1 : 2) void k_q8_scores(
    const int8_t *__restrict__ x, const float *__restrict__ xs, int64_t nq, int32_t d,
    const int8_t *__restrict__ t, const float *__restrict__ ts, int64_t nc, O *__restrict__ y,
    bool whole) {
    using C = tile::Core<int8_t, BM, BN, WM, WN, false, false, ALIGNED>;
    __shared__ __attribute__((aligned(1024))) char bufs[2 * C::kBytes];
    const int64_t qt = (nq + BM - 1) / BM, it = (nc + BN - 1) / BN, total = qt * it;
    for (int64_t id = blockIdx.x; id < (total + 7) / 8 * 8; id += gridDim.x) {
        const int64_t at = tile::xcd_order(id, total);
        if (at >= total) continue;
        const tile::Place pl = tile::place(at, qt, it);
        const int64_t q0 = pl.row * BM, i0 = pl.col * BN;
        const int64_t qn = nq - q0 < BM ? nq - q0 : BM, in = nc - i0 < BN ? nc - i0 : BN;
        C core;
        core.run({x + q0 * d, d, (int)qn}, {t + i0 * d, d, (int)in}, d, bufs);
        core.each([&](int q, int i, const tile::i32x4 &v) {
            if (q >= qn) return;
            const float s = xs[q0 + q];
            O *row = y + (q0 + q) * nc + i0;
            if (whole && i + 4 <= in) {
                Vec<O, 4> o;
#pragma unroll
                for (int u = 0; u < 4; ++u) o.v[u] = narrow<O>((float)v[u] * s * ts[i0 + i + u]);
                *reinterpret_cast<Vec<O, 4> *>(row + i) = o;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i + u < in) row[i + u] = narrow<O>((float)v[u] * s * ts[i0 + i + u]);
            }
        });
    }
}

template <typename O, int BM, int BN, int WM, int WN>
hipError_t q8_scores(const int8_t *x, const float *xs, int64_t nq, int32_t d, const int8_t *t,
                     const float *ts, int64_t nc, O *y, hipStream_t st) {
    const dim3 grid(tile::grid_of(((nq + BM - 1) / BM) * ((nc + BN - 1) / BN)));
    const dim3 block(WM * WN * 64);
    const bool aligned =
        ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(t) | (uintptr_t)d) & 15) == 0;
    const bool whole =
        ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(nc * sizeof(O))) & (4 * sizeof(O) - 1)) == 0;
    timing_before(st, "k_q8_scores");
    if (aligned)
        hipLaunchKernelGGL((k_q8_scores<O, BM, BN, WM, WN, true>), grid, block, 0, st, x, xs, nq, d,
                           t, ts, nc, y, whole);
    else
        hipLaunchKernelGGL((k_q8_scores<O, BM, BN, WM, WN, false>), grid, block, 0, st, x, xs, nq,
                           d, t, ts, nc, y, whole);
    timing_after(st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_q8_scores(const int8_t *x, const float *xs, int64_t nq, int32_t d,
                            const int8_t *table, const float *ts, int64_t nc, int out_dtype,
                            void *y, hipStream_t st, int n_cu) {
    (void)n_cu;
    auto go = [&](auto o) {
        using O = decltype(o);
        return q8_scores<O, 128, 128, 2, 2>(x, xs, nq, d, table, ts, nc, (O *)y, st);
    };
    switch (out_dtype) {
    case kF32: return go(float());
    case kF16: return go(_Float16());
    default: return go(__bf16());
    }
}

}  // namespace vs
