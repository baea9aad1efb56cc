// q8.hip -- scores over a table held in 8 bits.
//
//   y[q][i] = xs[q] ts[i] sum_k xc[q][k] tc[i][k]
// The sum is a whole number below 2^31 (d <= 131,071 codes of -128 .. 127), taken
// exactly; it is rounded to fp32 once, multiplied by both scales there, and the
// result rounded to the output's type.
#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

constexpr int kTile = 64, kDepth = 16;

template <typename O>
__global__ __launch_bounds__(256) void k_q8_scores(const int8_t *__restrict__ x,
                                                   const float *__restrict__ xs, int64_t nq,
                                                   int32_t d, const int8_t *__restrict__ t,
                                                   const float *__restrict__ ts, int64_t nc,
                                                   O *__restrict__ y, int64_t tiles) {
    __shared__ int8_t As[kDepth][kTile + 4], Bs[kDepth][kTile + 4];
    const int64_t ctiles = (nc + kTile - 1) / kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t q0 = tile / ctiles * kTile, i0 = tile % ctiles * kTile;
        int acc[4][4] = {};
        for (int64_t k0 = 0; k0 < d; k0 += kDepth) {
            __syncthreads();
            for (int e = threadIdx.x; e < kTile * kDepth; e += 256) {
                const int64_t k = k0 + e % kDepth, q = q0 + e / kDepth, i = i0 + e / kDepth;
                As[e % kDepth][e / kDepth] = q < nq && k < d ? x[q * d + k] : int8_t(0);
                Bs[e % kDepth][e / kDepth] = i < nc && k < d ? t[i * d + k] : int8_t(0);
            }
            __syncthreads();
            for (int k = 0; k < kDepth; ++k)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[r][c] += (int)As[k][ty + 16 * r] * (int)Bs[k][tx + 16 * c];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int64_t q = q0 + ty + 16 * r, i = i0 + tx + 16 * c;
                if (q < nq && i < nc)
                    y[q * nc + i] = narrow<O>((float)acc[r][c] * xs[q] * ts[i]);
            }
    }
}

}  // namespace

hipError_t launch_q8_scores(const int8_t *x, const float *xs, int64_t nq, int32_t d,
                            const int8_t *table, const float *ts, int64_t nc, int out_dtype,
                            void *y, hipStream_t st, int n_cu) {
    (void)n_cu;
    const int64_t tiles = ((nq + kTile - 1) / kTile) * ((nc + kTile - 1) / kTile);
    const int64_t most = 1 << 24;
    const dim3 grid((unsigned)(tiles < most ? tiles : most));
    timing_before(st, "k_q8_scores");
    switch (out_dtype) {
    case kF32:
        hipLaunchKernelGGL((k_q8_scores<float>), grid, dim3(256), 0, st, x, xs, nq, d, table, ts,
                           nc, (float *)y, tiles);
        break;
    case kF16:
        hipLaunchKernelGGL((k_q8_scores<_Float16>), grid, dim3(256), 0, st, x, xs, nq, d, table,
                           ts, nc, (_Float16 *)y, tiles);
        break;
    default:
        hipLaunchKernelGGL((k_q8_scores<__bf16>), grid, dim3(256), 0, st, x, xs, nq, d, table, ts,
                           nc, (__bf16 *)y, tiles);
    }
    timing_after(st);
    return hipGetLastError();
}

}  // namespace vs
