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
#include <type_traits>

#include "tile.h"
#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

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

// four neighbouring results of a row of `cols`, from column c
template <typename O, typename Acc>
__device__ __forceinline__ void store4(O *row, int64_t c, int64_t cols, const Acc &v, bool whole) {
    if (whole && c + 4 <= cols) {
        Vec<O, 4> o;
#pragma unroll
        for (int t = 0; t < 4; ++t) o.v[t] = narrow<O>(v[t]);
        *reinterpret_cast<Vec<O, 4> *>(row + c) = o;
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (c + t < cols) row[c + t] = narrow<O>(v[t]);
    }
}

// out[p][j] = sum_k A[p][k] B(g)(j, k): B = W[g][j][k], or W[g][k][j] (ACROSS).
// `whole`: rows of out start where four neighbours can be stored at once.
template <typename T, int BM, int BN, int WM, int WN, bool ACROSS, bool ALIGNED>
__global__ __launch_bounds__(WM *WN * 64, BM * BN > 128 * 128 ? 1 : 2) void k_unit_rows(
    const T *__restrict__ A, int64_t m, int32_t K, const T *__restrict__ W,
    const int32_t *__restrict__ offsets, int64_t G, int32_t cols, T *__restrict__ out,
    int64_t slots, bool whole) {
    using C = tile::Core<T, BM, BN, WM, WN, false, ACROSS, ALIGNED>;
    __shared__ __attribute__((aligned(1024))) char bufs[2 * C::kBytes];
    const int64_t ctiles = (cols + BN - 1) / BN, total = slots * ctiles;
    for (int64_t id = blockIdx.x; id < (total + 7) / 8 * 8; id += gridDim.x) {
        const int64_t at = tile::xcd_order(id, total);
        if (at >= total) continue;
        const tile::Place pl = tile::place(at, slots, ctiles);
        const RowTile rt = row_tile(offsets, G, m, BM, pl.row);
        if (rt.lo >= rt.hi) continue;
        const int64_t j0 = pl.col * BN;
        const int64_t jn = cols - j0 < BN ? cols - j0 : BN;
        const bool none = rt.unit >= G;
        const T *w = W + (none ? 0 : rt.unit) * (int64_t)K * cols;
        C core;
        core.run({A + rt.lo * K, K, (int)(rt.hi - rt.lo)},
                 {ACROSS ? w + j0 : w + j0 * K, ACROSS ? cols : K, (int)jn}, none ? 0 : K, bufs);
        core.each([&](int i, int j, const tile::f32x4 &v) {
            if (rt.lo + i < rt.hi) store4(out + (rt.lo + i) * cols, j0 + j, cols, v, whole);
        });
    }
}

// dW[g][j][k] = sum over g's rows p of dY[p][j] X[p][k]: both sides across
template <typename T, typename O, int BM, int BN, int WM, int WN, bool ALIGNED>
__global__ __launch_bounds__(WM *WN * 64, BM * BN > 128 * 128 ? 1 : 2) void k_unit_mats(
    const T *__restrict__ dY, const T *__restrict__ X, int64_t m, int32_t d,
    const int32_t *__restrict__ offsets, int64_t G, int32_t cols, O *__restrict__ dW, bool whole) {
    using C = tile::Core<T, BM, BN, WM, WN, true, true, ALIGNED>;
    __shared__ __attribute__((aligned(1024))) char bufs[2 * C::kBytes];
    const int64_t jt = (cols + BM - 1) / BM, kt = (d + BN - 1) / BN, total = G * jt * kt;
    for (int64_t id = blockIdx.x; id < (total + 7) / 8 * 8; id += gridDim.x) {
        const int64_t at = tile::xcd_order(id, total);
        if (at >= total) continue;
        const int64_t g = at / (jt * kt);
        const tile::Place pl = tile::place(at - g * jt * kt, jt, kt);
        const int64_t j0 = pl.row * BM, k0 = pl.col * BN;
        const int64_t lo = offset_of(offsets, g, G, m), hi = offset_of(offsets, g + 1, G, m);
        const int64_t jn = cols - j0 < BM ? cols - j0 : BM, kn = d - k0 < BN ? d - k0 : BN;
        C core;
        core.run({dY + lo * cols + j0, cols, (int)jn}, {X + lo * d + k0, d, (int)kn}, hi - lo, bufs);
        core.each([&](int i, int k, const tile::f32x4 &v) {
            if (i < jn) store4(dW + (g * cols + j0 + i) * d, k0 + k, d, v, whole);
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

inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
// rows of `cols` elements of a matrix at p start on multiples of `bytes`
inline bool on(uintptr_t p, int64_t cols, int esize, uintptr_t bytes) {
    return ((p | (uintptr_t)(cols * esize)) & (bytes - 1)) == 0;
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t unit_rows(const void *A, int64_t m, int32_t K, const void *W, const int32_t *offsets,
                     int64_t G, int32_t cols, bool across, void *out, hipStream_t st) {
    const int64_t slots = m / BM + G + 1;
    const dim3 grid(tile::grid_of(slots * ((cols + BN - 1) / BN))), block(WM * WN * 64);
    const int es = (int)sizeof(T);
    const bool aligned = on(addr(A), K, es, 16) && on(addr(W), across ? cols : K, es, 16);
    const bool whole = on(addr(out), cols, es, 4 * es);
    auto go = [&](auto ac, auto al) {
        hipLaunchKernelGGL((k_unit_rows<T, BM, BN, WM, WN, decltype(ac)::value, decltype(al)::value>),
                           grid, block, 0, st, (const T *)A, m, K, (const T *)W, offsets, G, cols,
                           (T *)out, slots, whole);
    };
    timing_before(st, "k_unit_rows");
    if (across && aligned) go(std::true_type(), std::true_type());
    else if (across) go(std::true_type(), std::false_type());
    else if (aligned) go(std::false_type(), std::true_type());
    else go(std::false_type(), std::false_type());
    timing_after(st);
    return hipGetLastError();
}

template <typename T, typename O, int BM, int BN, int WM, int WN>
hipError_t unit_mats(const void *dY, const void *X, int64_t m, int32_t d, const int32_t *offsets,
                     int64_t G, int32_t cols, void *dW, hipStream_t st) {
    const int64_t total = G * ((cols + BM - 1) / BM) * ((d + BN - 1) / BN);
    const dim3 grid(tile::grid_of(total)), block(WM * WN * 64);
    const int es = (int)sizeof(T);
    const bool aligned = on(addr(dY), cols, es, 16) && on(addr(X), d, es, 16);
    const bool whole = on(addr(dW), d, (int)sizeof(O), 4 * sizeof(O));
    timing_before(st, "k_unit_mats");
    if (aligned)
        hipLaunchKernelGGL((k_unit_mats<T, O, BM, BN, WM, WN, true>), grid, block, 0, st,
                           (const T *)dY, (const T *)X, m, d, offsets, G, cols, (O *)dW, whole);
    else
        hipLaunchKernelGGL((k_unit_mats<T, O, BM, BN, WM, WN, false>), grid, block, 0, st,
                           (const T *)dY, (const T *)X, m, d, offsets, G, cols, (O *)dW, whole);
    timing_after(st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_unit_rows(const void *A, int64_t m, int32_t K, int dtype, const void *W,
                            const int32_t *offsets, int64_t G, int32_t cols, bool across, void *out,
                            hipStream_t st, int n_cu) {
    (void)n_cu;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return unit_rows<T, 128, 128, 2, 2>(A, m, K, W, offsets, G, cols, across, out, st);
    });
}

hipError_t launch_unit_mats(const void *dY, const void *X, int64_t m, int32_t d, int dtype,
                            const int32_t *offsets, int64_t G, int32_t cols, int grad_dtype,
                            void *dW, hipStream_t st, int n_cu) {
    (void)n_cu;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto o) {
            using O = decltype(o);
            return unit_mats<T, O, 128, 128, 2, 2>(dY, X, m, d, offsets, G, cols, dW, st);
        };
        return grad_dtype == dtype ? go(T()) : go(float());
    });
}

}  // namespace vs
