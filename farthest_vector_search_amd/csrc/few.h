// few.h -- products of few rows (a query, the rows of a decoding step) with a matrix
// that is read once, for units.hip and q8.hip.
//
// Bound by reading the matrix, so there are no tiles in LDS: a wave takes NB blocks of
// 16 of its rows and loads them straight into the matrix instruction's layout, 16 bytes
// a lane at any address, 256 bytes of k at a time (8 KiB of the matrix with NB = 2); the
// few rows' own, 16 MB at most, come from the caches the same way.  Where there are too
// few blocks to fill the GPU, the waves of a workgroup share a block along k, and the
// first of them adds their sums in order.
#pragma once

#include "tile.h"

namespace vs {
namespace few {

using tile::f32x4;
using tile::i32x4;
using tile::u32x4;

constexpr int kWaves = 8;
constexpr int kHalf = 64;  // bytes of k a matrix instruction takes

// Elements k .. k + N - 1 of a row of `depth`, zeros behind its end
template <typename T>
__device__ __forceinline__ u32x4 last_bytes(const T *row, int64_t k, int64_t depth) {
    constexpr int N = 16 / (int)sizeof(T);
    typedef unsigned __int128 Bits;
    Bits bits = 0;
    const int64_t n = depth - k;
    if (n >= N) {
        __builtin_memcpy(&bits, row + k, 16);
    } else if (n > 0 && depth >= N) {  // the row's last 16 bytes, shifted into place
        __builtin_memcpy(&bits, row + depth - N, 16);
        bits >>= (int)(N - n) * (int)sizeof(T) * 8;
    } else if (n > 0) {
        typedef typename std::conditional<
            sizeof(T) == 1, uint8_t,
            typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type>::type Whole;
#pragma unroll 1
        for (int t = 0; t < n; ++t)
            bits |= (Bits) reinterpret_cast<const Whole *>(row)[k + t] << (t * (int)sizeof(T) * 8);
    }
    return __builtin_bit_cast(u32x4, bits);
}

// out[m][n] = sum_k M(m, k) N(n, k) for rows of 16 MB at most and the wave's 16 NB
// of `nrows`; `share` of the workgroup's waves split k.  put(m, n, sums of rows n .. n
// + 3) is called for rows that are there.
template <typename T, int MB, int NB, typename F>
__device__ __forceinline__ void products(const T *M, int mrows, const T *N, int64_t n0,
                                         int64_t nrows, int64_t depth, int share, F put) {
    typedef typename tile::Sum<T>::type Acc;
    constexpr int kPer = kHalf / (int)sizeof(T);  // k's of a half
    constexpr int kLane = 16 / (int)sizeof(T);    // of them a lane's
    __shared__ Acc sums[kWaves][MB * NB][64];
    const int lane = threadIdx.x & 63, i = lane & 15, j = lane >> 4;
    const int wave = tile::uniform((int)(threadIdx.x >> 6));
    const int part = wave % share;  // of k
    n0 += (int64_t)(wave / share) * NB * 16;
    const T *mrow[MB], *nrow[NB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int r = b * 16 + i;
        mrow[b] = M + (int64_t)(r < mrows ? r : mrows - 1) * depth;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t r = n0 + b * 16 + i;
        nrow[b] = N + (r < nrows ? r : nrows - 1) * depth;
    }
    Acc acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[a][b] = Acc{0, 0, 0, 0};
    const int64_t halves = (depth + kPer - 1) / kPer, whole = depth / kPer;
    const int64_t h0 = halves * part / share, h1 = halves * (part + 1) / share;
    const int64_t end = h1 < whole ? h1 : whole;  // of the whole halves
    auto step = [&](int64_t h, auto count) {
        constexpr int U = decltype(count)::value;
        u32x4 m[U][MB], n[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = (h + u) * kPer + j * kLane;
#pragma unroll
            for (int b = 0; b < NB; ++b) __builtin_memcpy(&n[u][b], nrow[b] + k, 16);
#pragma unroll
            for (int b = 0; b < MB; ++b) __builtin_memcpy(&m[u][b], mrow[b] + k, 16);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[a][b] = tile::mac(acc[a][b], n[u][b], m[u][a], T());
    };
    int64_t h = h0;
    for (; h + 4 <= end; h += 4) step(h, std::integral_constant<int, 4>());
    for (; h < end; ++h) step(h, std::integral_constant<int, 1>());
    if (h < h1) {  // the last half, cut short
        const int64_t k = h * kPer + j * kLane;
        u32x4 n[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) n[b] = last_bytes(nrow[b], k, depth);
#pragma unroll
        for (int a = 0; a < MB; ++a) {
            const u32x4 m = last_bytes(mrow[a], k, depth);
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = tile::mac(acc[a][b], n[b], m, T());
        }
    }
    if (share > 1) {
        if (part > 0)
#pragma unroll
            for (int q = 0; q < MB * NB; ++q) sums[wave][q][lane] = acc[q / NB][q % NB];
        __syncthreads();
        if (part > 0) return;
        for (int p = 1; p < share; ++p)
#pragma unroll
            for (int q = 0; q < MB * NB; ++q) acc[q / NB][q % NB] += sums[wave + p][q][lane];
    }
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int m = a * 16 + i;
            const int64_t n = n0 + b * 16 + j * 4;
            if (m < mrows && n < nrows) put(m, n, acc[a][b]);
        }
}

// four neighbours of a row of `cols`, from column c
template <typename O>
__device__ __forceinline__ void store4(O *row, int64_t c, int64_t cols, const f32x4 &v) {
    O o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = narrow<O>(v[t]);
    if (c + 4 <= cols) {
        __builtin_memcpy(row + c, o, sizeof(o));
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (c + t < cols) row[c + t] = o[t];
    }
}

// How `blocks` blocks of 16 rows of `bytes` each, taken `times` times, are dealt out: nb
// of them a wave, `share` waves a block, so that there are 16 waves a CU if they can be
// had; a wave's part of k is not cut below 128 bytes.  Half and twice the waves, 16 of
// 65,536 rows of 4,096 bytes for 1 query: 86 and 53 us, so 51; 128 rows to 16 units of
// 2,048 x 2,048 bf16 48 and 32, so 30.
struct Deal {
    int nb, share;
    int64_t groups;  // workgroups
};
inline Deal deal(int64_t blocks, int64_t times, int64_t bytes, int n_cu) {
    Deal d{2, 1, 0};
    auto waves = [&] { return times * ((blocks + d.nb - 1) / d.nb) * d.share; };
    while (waves() < (int64_t)n_cu * 16) {
        if (d.share < kWaves && bytes >= 256 * d.share) d.share *= 2;
        else if (d.nb == 2) d.nb = 1;
        else break;
    }
    const int64_t per = (int64_t)(kWaves / d.share) * d.nb;
    d.groups = (blocks + per - 1) / per;
    return d;
}

}  // namespace few
}  // namespace vs
