// units.hip -- products of rows in unit order with each unit's matrix, and the
// gradients of both.
//
//   products   Y[p][j]  = sum_k X[p][k] W[g][j][k]    offsets[g] <= p < offsets[g + 1]
//   rows       dX[p][k] = sum_j dY[p][j] W[g][j][k]
//   matrices   dW[g][j][k] = sum over g's rows p of dY[p][j] X[p][k]
// Rows of no unit (offsets[n_groups] .. m - 1) give zeros.
//
// The rows' tiles are found on the device: unit g owns the tiles T(g) ..
// T(g + 1) - 1 with T(g) = offsets[g] / B + g for tiles of B rows, which is
// never fewer than its rows need, so that the grid follows from m and the number
// of units alone (a unit's spare tile ends at once).  T rises, and a wave finds
// its tile's unit by looking at 64 of them at a time.  The rows of no unit count
// as one unit more.
#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ int64_t offset_of(const int32_t *__restrict__ offsets, int64_t g,
                                             int64_t G, int64_t m) {
    if (g > G) return m;
    const int64_t o = offsets[g];
    return o < 0 ? 0 : o > m ? m : o;
}

struct RowTile {
    int64_t unit, lo, hi;  // rows lo .. hi - 1 of the unit (G: no unit)
};

// The rows of tile `slot`; the whole wave takes part.
__device__ __forceinline__ RowTile row_tile(const int32_t *__restrict__ offsets, int64_t G,
                                            int64_t m, int rows, int64_t slot) {
    const int lane = threadIdx.x & 63;
    // unit in [lo, hi): T(lo) <= slot, and T(hi) > slot or hi = G + 1
    int64_t lo = 0, hi = G + 1;
    while (hi - lo > 1) {
        const int64_t width = (hi - lo + 63) / 64;
        const int64_t g = lo + lane * width;
        const bool below = g < hi && offset_of(offsets, g, G, m) / rows + g <= slot;
        const unsigned long long set = __ballot(below) | 1;
        const int last = 63 - __clzll(set);
        lo += last * width;
        hi = lo + width < hi ? lo + width : hi;
    }
    RowTile t;
    t.unit = lo;
    const int64_t o = offset_of(offsets, lo, G, m), e = offset_of(offsets, lo + 1, G, m);
    const int64_t first = o / rows + lo;
    t.lo = o + (slot - first) * rows;
    t.hi = t.lo + rows < e ? t.lo + rows : e;
    return t;
}

// One 64 x 64 tile of C = A B^T: A(i, k), B(j, k) and the place of C by functions.
template <typename FA, typename FB, typename FC>
__device__ __forceinline__ void tile_product(int64_t K, FA fa, FB fb, FC fc) {
    __shared__ float As[kDepth][kTile + 1], Bs[kDepth][kTile + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kDepth) {
        __syncthreads();
        for (int e = threadIdx.x; e < kTile * kDepth; e += 256) {
            As[e % kDepth][e / kDepth] = fa(e / kDepth, k0 + e % kDepth);
            Bs[e % kDepth][e / kDepth] = fb(e / kDepth, k0 + e % kDepth);
        }
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[r][c] = __builtin_fmaf(As[k][ty + 16 * r], Bs[k][tx + 16 * c], acc[r][c]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) fc(ty + 16 * r, tx + 16 * c, acc[r][c]);
}

// out[p][j] = sum_k A[p][k] B(g)(j, k): B = W[g][j][k], or W[g][k][j] (ACROSS)
template <typename T, bool ACROSS>
__global__ __launch_bounds__(256) void k_unit_rows(const T *__restrict__ A, int64_t m, int32_t K,
                                                   const T *__restrict__ W,
                                                   const int32_t *__restrict__ offsets, int64_t G,
                                                   int32_t out_cols, T *__restrict__ out,
                                                   int64_t tiles) {
    const int64_t ctiles = (out_cols + kTile - 1) / kTile;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const RowTile rt = row_tile(offsets, G, m, kTile, tile / ctiles);
        if (rt.lo >= rt.hi) continue;
        const int64_t j0 = tile % ctiles * kTile;
        const T *w = W + (rt.unit < G ? rt.unit : 0) * (int64_t)K * out_cols;
        tile_product(
            rt.unit < G ? K : 0,
            [&](int r, int64_t k) {
                return rt.lo + r < rt.hi && k < K ? widen(A[(rt.lo + r) * K + k]) : 0.0f;
            },
            [&](int c, int64_t k) {
                const int64_t j = j0 + c;
                if (j >= out_cols || k >= K) return 0.0f;
                return widen(ACROSS ? w[k * out_cols + j] : w[j * K + k]);
            },
            [&](int r, int c, float v) {
                if (rt.lo + r < rt.hi && j0 + c < out_cols)
                    out[(rt.lo + r) * out_cols + j0 + c] = narrow<T>(v);
            });
    }
}

template <typename T, typename O>
__global__ __launch_bounds__(256) void k_unit_mats(const T *__restrict__ dY,
                                                   const T *__restrict__ X, int64_t m, int32_t d,
                                                   const int32_t *__restrict__ offsets, int64_t G,
                                                   int32_t cols, O *__restrict__ dW,
                                                   int64_t tiles) {
    const int64_t jt = (cols + kTile - 1) / kTile, kt = (d + kTile - 1) / kTile;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t g = tile / (jt * kt);
        const int64_t j0 = tile / kt % jt * kTile, k0 = tile % kt * kTile;
        const int64_t lo = offset_of(offsets, g, G, m), hi = offset_of(offsets, g + 1, G, m);
        tile_product(
            hi - lo,
            [&](int r, int64_t p) {
                return j0 + r < cols && lo + p < hi ? widen(dY[(lo + p) * cols + j0 + r]) : 0.0f;
            },
            [&](int c, int64_t p) {
                return k0 + c < d && lo + p < hi ? widen(X[(lo + p) * d + k0 + c]) : 0.0f;
            },
            [&](int r, int c, float v) {
                if (j0 + r < cols && k0 + c < d)
                    dW[(g * cols + j0 + r) * d + k0 + c] = narrow<O>(v);
            });
    }
}

template <typename F>
hipError_t by_type(int dtype, F f) {
    switch (dtype) {
    case kF32: return f(float());
    case kF16: return f(_Float16());
    default: return f(__bf16());
    }
}

inline unsigned grid_for(int64_t tiles) {
    const int64_t most = 1 << 24;
    return (unsigned)(tiles < most ? tiles : most);
}

}  // namespace

hipError_t launch_unit_rows(const void *A, int64_t m, int32_t K, int dtype, const void *W,
                            const int32_t *offsets, int64_t G, int32_t out_cols, bool across,
                            void *out, hipStream_t st, int n_cu) {
    (void)n_cu;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t tiles = (m / kTile + G + 1) * ((out_cols + kTile - 1) / kTile);
        timing_before(st, "k_unit_rows");
        if (across)
            hipLaunchKernelGGL((k_unit_rows<T, true>), dim3(grid_for(tiles)), dim3(256), 0, st,
                               (const T *)A, m, K, (const T *)W, offsets, G, out_cols, (T *)out,
                               tiles);
        else
            hipLaunchKernelGGL((k_unit_rows<T, false>), dim3(grid_for(tiles)), dim3(256), 0, st,
                               (const T *)A, m, K, (const T *)W, offsets, G, out_cols, (T *)out,
                               tiles);
        timing_after(st);
        return hipGetLastError();
    });
}

hipError_t launch_unit_mats(const void *dY, const void *X, int64_t m, int32_t d, int dtype,
                            const int32_t *offsets, int64_t G, int32_t cols, int grad_dtype,
                            void *dW, hipStream_t st, int n_cu) {
    (void)n_cu;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return by_type(grad_dtype, [&](auto o) {
            using O = decltype(o);
            const int64_t tiles =
                G * ((cols + kTile - 1) / kTile) * ((d + kTile - 1) / kTile);
            timing_before(st, "k_unit_mats");
            hipLaunchKernelGGL((k_unit_mats<T, O>), dim3(grid_for(tiles)), dim3(256), 0, st,
                               (const T *)dY, (const T *)X, m, d, offsets, G, cols, (O *)dW,
                               tiles);
            timing_after(st);
            return hipGetLastError();
        });
    });
}

}  // namespace vs
