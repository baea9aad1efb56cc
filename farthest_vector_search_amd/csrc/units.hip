// units.hip -- products of rows in unit order with each unit's matrix, and the
// gradients of both.
//
//   products   Y[p][j]  = sum_k X[p][k] W[g][j][k]    offsets[g] <= p < offsets[g + 1]
//   rows       dX[p][k] = sum_j dY[p][j] W[g][j][k]
//   matrices   dW[g][j][k] = sum over g's rows p of dY[p][j] X[p][k]
// Rows of no unit (before offsets[0], or from offsets[n_groups] on) give zeros.
//
// The rows' tiles are found on the device.  The rows form runs: those before the
// first unit, each unit's, those behind the last.  Run u owns the tiles T(u) ..
// T(u + 1) - 1 with T(u) = begin(u) / B + u for tiles of B rows, which is never fewer
// than its rows need, so that the grid follows from m and the number of units alone
// (a run's spare tile ends at once).  T rises, and a wave finds its tile's run by
// looking at 64 of them at a time.  Up to some hundred runs are counted through
// instead (counted_tile).
#include <type_traits>

#include "few.h"
#include "tile.h"
#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

// a place read from the offsets, held inside the rows
__device__ __forceinline__ int64_t place_of(const int32_t *__restrict__ offsets, int64_t g,
                                            int64_t m) {
    const int64_t o = offsets[g];
    return o < 0 ? 0 : o > m ? m : o;
}

// where run u of the rows begins: run 0 those before the first unit, run g + 1 unit g,
// run G + 1 those behind the last unit
__device__ __forceinline__ int64_t run_begin(const int32_t *__restrict__ offsets, int64_t u,
                                             int64_t G, int64_t m) {
    return u == 0 ? 0 : u > G + 1 ? m : place_of(offsets, u - 1, m);
}

struct RowTile {
    int64_t unit, lo, hi;  // rows lo .. hi - 1 of the unit
    bool none;             // they belong to none (unit is 0)
};

// The rows of tile `slot`; the whole wave takes part.
__device__ __forceinline__ RowTile row_tile(const int32_t *__restrict__ offsets, int64_t G,
                                            int64_t m, int rows, int64_t slot) {
    const int lane = threadIdx.x & 63;
    // run in [lo, hi): T(lo) <= slot, and T(hi) > slot or hi = G + 2
    int64_t lo = 0, hi = G + 2;
    while (hi - lo > 1) {
        const int64_t width = (hi - lo + 63) / 64;
        const int64_t u = lo + lane * width;
        const bool below = u < hi && run_begin(offsets, u, G, m) / rows + u <= slot;
        const unsigned long long set = __ballot(below) | 1;
        const int last = 63 - __clzll(set);
        lo += last * width;
        hi = lo + width < hi ? lo + width : hi;
    }
    const int64_t o = run_begin(offsets, lo, G, m), e = run_begin(offsets, lo + 1, G, m);
    RowTile t;
    t.none = lo == 0 || lo > G;
    t.unit = t.none ? 0 : lo - 1;
    t.lo = o + (slot - (o / rows + lo)) * rows;
    t.hi = t.lo + rows < e ? t.lo + rows : e;
    return t;
}
// tiles of `rows` rows that cover m rows of G units
inline int64_t slots_of(int64_t m, int64_t G, int rows) { return m / rows + G + 2; }

// inclusive sums over the wave's lanes: within rows of 16, then across them
__device__ __forceinline__ int scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from 1 lane below
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // 4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row 0's to 1, 2's to 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // the lower half's
    return v;
}

// The same for up to kCounted units, in an order that keeps the XCDs even: the tiles of
// the units are counted and dealt out in 8 equal stretches, one an XCD, and after them
// those of no unit, which cost little, the same way.  By slots, empty ones fall to some
// XCDs more than to others (bf16, us by slots and counted: 8,192 rows to one unit of
// 8,192 x 8,192 913 and 790; 10,240 to 64 of 1,024 x 1,024 58 and 50; 32 to 64 of 2,048 x
// 1,024 24.9 and 21.2).  Counting takes every lane more loads the more units there are:
// 65,536 rows to 300 of 2,048 x 2,048 707 and 707; 60,000 to 300 of 512 x 512 71 and 74,
// to 1,000 137 and 165; 2,500 to 2,500 of 512 x 256 94 and 199.  Whole tiles first and
// units' last tiles behind them was slower (65,536 rows to 128 of 2,048 x 2,048: 609, so
// 669), since W is then read twice.
constexpr int64_t kCounted = 256;
__device__ __forceinline__ bool counted_tile(const int32_t *__restrict__ offsets, int64_t G,
                                             int64_t m, int rows, int64_t ctiles, int64_t id,
                                             RowTile &t, int64_t &col) {
    const int lane = threadIdx.x & 63;
    const int per = (int)((G + 63) / 64);  // a lane's units
    auto count = [&](int64_t g) {
        if (g >= G) return 0;
        const int64_t n = place_of(offsets, g + 1, m) - place_of(offsets, g, m);
        return n > 0 ? (int)(((uint32_t)n + rows - 1) / rows) : 0;
    };
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += count((int64_t)lane * per + i);
    int sum = scan(mine);
    const int64_t begin = place_of(offsets, 0, m), end = place_of(offsets, G, m);
    const int before_units = (int)((begin + rows - 1) / rows);
    const int64_t all = __builtin_amdgcn_readlane(sum, 63);
    const int64_t others = before_units + (m - end + rows - 1) / rows;
    const int64_t turn = id >> 3, xcd = id & 7;
    const int64_t first = (all * ctiles + 7) >> 3, then = (others * ctiles + 7) >> 3;
    t.none = turn >= first;
    const int64_t at = t.none ? xcd * then + turn - first : xcd * first + turn;
    if (t.none ? turn - first >= then || at >= others * ctiles : at >= all * ctiles) return false;
    const tile::Place pl = tile::place(at, t.none ? others : all, ctiles);
    const int row = tile::uniform((int)pl.row);
    col = pl.col;
    int64_t e;
    if (t.none) {
        const bool front = row < before_units;
        t.unit = 0;
        t.lo = front ? (int64_t)row * rows : end + (int64_t)(row - before_units) * rows;
        e = front ? begin : m;
    } else {
        int holder = __ffsll((unsigned long long)__ballot(sum > row)) - 1;
        int before = __builtin_amdgcn_readlane(sum - mine, holder);
        t.unit = (int64_t)holder * per;
        if (per > 1) {  // which of the lane's units
            mine = lane < per ? count(t.unit + lane) : 0;
            sum = before + scan(mine);
            holder = __ffsll((unsigned long long)__ballot(sum > row)) - 1;
            before = __builtin_amdgcn_readlane(sum - mine, holder);
            t.unit += holder;
        }
        if (holder < 0 || row < before) return false;  // places that fall, and sums past 31 bits
        t.lo = place_of(offsets, t.unit, m) + (int64_t)(row - before) * rows;
        e = place_of(offsets, t.unit + 1, m);
    }
    t.hi = t.lo + rows < e ? t.lo + rows : e;
    return true;
}

// out[p][j] = sum_k A[p][k] B(g)(j, k): B = W[g][j][k], or W[g][k][j] (ACROSS).  Bound
// by the matrix cores where units have many rows (8,192 rows to one unit of 8,192 x 8,192
// bf16: 810 us, 781 at best, 1,408 TFLOP/s; across 796 and 750 us, 1,466 TFLOP/s), with
// 65,536 rows to 128 of 2,048 x 2,048 at random 600 us (916 TFLOP/s: units' last tiles); fp32
// 971 us for 16,384 to 16 of 2,048 x 2,048 (142 TFLOP/s).  By reading W where they have few: 1,024
// rows to 64 of 1,024 x 1,024 28 us (4.9 TB/s).
template <typename T, int BM, int BN, int WM, int WN, bool ACROSS, int PIECE>
__global__ __launch_bounds__(WM *WN * 64, 2) void k_unit_rows(
    const T *__restrict__ A, int64_t m, int32_t K, const T *__restrict__ W,
    const int32_t *__restrict__ offsets, int64_t G, int32_t cols, T *__restrict__ out,
    int64_t slots) {
    using C = tile::Core<T, BM, BN, WM, WN, false, ACROSS, PIECE>;
    __shared__ __attribute__((aligned(1024))) char bufs[2 * C::kBytes];
    const int64_t ctiles = (cols + BN - 1) / BN;
    auto job = [&](int64_t id, tile::Job<T, T> &j) {
        RowTile rt;
        int64_t col;
        if (G <= kCounted) {
            if (!counted_tile(offsets, G, m, BM, ctiles, id, rt, col)) return false;
        } else {
            int64_t at;
            if (!tile::xcd_tile(id, slots * ctiles, at)) return false;
            const tile::Place pl = tile::place(at, slots, ctiles);
            rt = row_tile(offsets, G, m, BM, pl.row);
            col = pl.col;
        }
        if (rt.lo >= rt.hi) return false;
        const int64_t j0 = col * BN;
        const T *w = W + rt.unit * (int64_t)K * cols;
        const int jn = (int)(cols - j0 < BN ? cols - j0 : BN);
        j.depth = rt.none ? 0 : K;
        j.m = {A + rt.lo * K, K, (int)(rt.hi - rt.lo)};
        j.n = {ACROSS ? w + j0 : w + j0 * K, ACROSS ? cols : K, jn};
        j.out = out + rt.lo * cols + j0;
        j.ld = cols;
        return true;
    };
    // A unit's last tile is half empty on average: with tiles of 256 rows it is taken as
    // one of 64 or 128 where that is enough.  65,536 rows to 128 units of 2,048 x 2,048 at
    // random: 609 us, with 128 alone 617, without 641.  (Tiles of 128 as 64: no gain.)
    if constexpr (BM == 256)
        tile::run_tiles<T, T, C, tile::Core<T, 64, BN, 1, 8, false, ACROSS, PIECE>,
                        tile::Core<T, 128, BN, 2, 4, false, ACROSS, PIECE>>(slots * ctiles + 16, bufs, job);
    else
        tile::run_tiles<T, T, C>(slots * ctiles + 16, bufs, job);
}

// The same along k for units of few rows: 16 rows a tile, `groups` workgroups for each.
// Bound by reading W: 16 rows to 8 units of 2,048 x 2,048 bf16 16.6 us (4.0 TB/s), to 4 of
// 8,192 x 8,192 121 us (4.4 TB/s).
template <typename T, int NB>
__global__ __launch_bounds__(few::kWaves * 64) void k_unit_rows_few(
    const T *__restrict__ A, int64_t m, int32_t K, const T *__restrict__ W,
    const int32_t *__restrict__ offsets, int64_t G, int32_t cols, T *__restrict__ out,
    int64_t slots, int64_t groups, int share) {
    const int per = few::kWaves / share * NB * 16;
    for (int64_t id = blockIdx.x; id < slots * groups; id += gridDim.x) {
        const RowTile rt = row_tile(offsets, G, m, 16, id / groups);
        if (rt.lo >= rt.hi) continue;
        const int64_t j0 = id % groups * per;
        const T *w = W + rt.unit * (int64_t)K * cols;
        __syncthreads();  // the last turn's sums have been read
        few::products<T, 1, NB>(A + rt.lo * K, (int)(rt.hi - rt.lo), w, j0, cols, rt.none ? 0 : K,
                                share, [&](int i, int64_t j, const tile::f32x4 &v) {
                                    few::store4(out + (rt.lo + i) * cols, j, cols, v);
                                });
    }
}

// dW[g][j][k] = sum over g's rows p of dY[p][j] X[p][k]: both sides across.  With
// `parts` > 1 each unit's rows are cut into so many equal runs, whose sums stand one
// array of matrices behind the other.  Bound by the matrix cores where units have many
// rows (8,192 of one, 8,192 x 8,192 bf16: 819 us, 777 at best, 1,415 TFLOP/s), by writing
// dW where they have few (64 rows to 64 of 1,024 x 1,024: 35 us, 3.8 TB/s).
template <typename T, typename O, int BM, int BN, int WM, int WN, int PIECE>
__global__ __launch_bounds__(WM *WN * 64, 2) void k_unit_mats(
    const T *__restrict__ dY, const T *__restrict__ X, int64_t m, int32_t d,
    const int32_t *__restrict__ offsets, int64_t G, int32_t cols, O *__restrict__ dW, int parts) {
    using C = tile::Core<T, BM, BN, WM, WN, true, true, PIECE>;
    __shared__ __attribute__((aligned(1024))) char bufs[2 * C::kBytes];
    const int64_t jt = (cols + BM - 1) / BM, kt = (d + BN - 1) / BN, total = G * parts * jt * kt;
    tile::run_tiles<T, O, C>(
        total, bufs,
        [&](int64_t id, tile::Job<T, O> &j) {
            int64_t at;
            if (!tile::xcd_tile(id, total, at)) return false;
            const int64_t run = at / (jt * kt), g = run / parts, part = run - g * parts;
            const tile::Place pl = tile::place(at - run * jt * kt, jt, kt);
            const int64_t j0 = pl.row * BM, k0 = pl.col * BN;
            const int64_t first = place_of(offsets, g, m), end = place_of(offsets, g + 1, m);
            const int64_t rows = end > first ? end - first : 0;
            const int64_t lo = first + rows * part / parts, hi = first + rows * (part + 1) / parts;
            j.depth = hi - lo;
            j.m = {dY + lo * cols + j0, cols, (int)(cols - j0 < BM ? cols - j0 : BM)};
            j.n = {X + lo * d + k0, d, (int)(d - k0 < BN ? d - k0 : BN)};
            j.out = dW + ((part * G + g) * cols + j0) * d + k0;
            j.ld = d;
            return true;
        });
}

// the sums of a unit's runs of rows, in their order
template <typename O>
__global__ __launch_bounds__(256) void k_unit_join(const float *__restrict__ sums, int parts,
                                                   int64_t n, O *__restrict__ dW) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        float s = sums[i];
        for (int p = 1; p < parts; ++p) s += sums[p * n + i];
        dW[i] = narrow<O>(s);
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

inline int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }
// a width that tiles of 256 pad by more than a fifth beyond those of 128
inline bool wasteful(int64_t n) { return tiles_of(n, 256) * 256 * 5 > tiles_of(n, 128) * 128 * 6; }

// the bytes that rows at p and q move in, by the boundaries they lie on: 16, 4 or (0) any
inline int piece_of(uintptr_t p, int64_t pcols, uintptr_t q, int64_t qcols, int esize) {
    auto both = [&](uintptr_t b) { return on(p, pcols, esize, b) && on(q, qcols, esize, b); };
    return both(16) ? 16 : both(4) ? 4 : 0;
}

// f(piece as a constant); tiles of 256 are for pieces of 16, and fp32 has none of 0
template <typename T, int BM, typename F>
void by_piece(int piece, F f) {
    if constexpr (BM < 256) {
        if (piece == 4) f(std::integral_constant<int, 4>());
        if constexpr (sizeof(T) < 4)
            if (piece == 0) f(std::integral_constant<int, 0>());
    }
    if (piece == 16) f(std::integral_constant<int, 16>());
}

// `piece`: of the rows of A, and of W as the product takes them
template <typename T, int BM, int BN, int WM, int WN>
hipError_t unit_rows(const void *A, int64_t m, int32_t K, const void *W, const int32_t *offsets,
                     int64_t G, int32_t cols, bool across, int piece, void *out,
                     hipStream_t st) {
    const int64_t slots = slots_of(m, G, BM);
    // 16 more: each of the 8 stretches of either kind is rounded up
    const dim3 grid(tile::grid_of(slots * tiles_of(cols, BN) + 16)), block(WM * WN * 64);
    auto go = [&](auto ac, auto pc) {
        static const tile::FormName name("k_unit_rows", BM, BN, decltype(pc)::value,
                                         decltype(ac)::value ? ",across" : "");
        timing_before(st, name.text);
        hipLaunchKernelGGL((k_unit_rows<T, BM, BN, WM, WN, decltype(ac)::value, decltype(pc)::value>),
                           grid, block, 0, st, (const T *)A, m, K, (const T *)W, offsets, G, cols,
                           (T *)out, slots);
        timing_after(st);
    };
    auto way = [&](auto pc) {
        if (across) go(std::true_type(), pc);
        else go(std::false_type(), pc);
    };
    by_piece<T, BM>(piece, way);
    return hipGetLastError();
}

template <typename T>
hipError_t unit_rows_few(const void *A, int64_t m, int32_t K, const void *W, const int32_t *offsets,
                         int64_t G, int32_t cols, const few::Deal &d, void *out, hipStream_t st) {
    const int64_t slots = slots_of(m, G, 16), total = slots * d.groups, most = tile::kMostGroups;
    const dim3 grid((unsigned)(total < most ? total : most)), block(few::kWaves * 64);
    timing_before(st, "k_unit_rows_few");
    if (d.nb == 2)
        hipLaunchKernelGGL((k_unit_rows_few<T, 2>), grid, block, 0, st, (const T *)A, m, K,
                           (const T *)W, offsets, G, cols, (T *)out, slots, d.groups, d.share);
    else
        hipLaunchKernelGGL((k_unit_rows_few<T, 1>), grid, block, 0, st, (const T *)A, m, K,
                           (const T *)W, offsets, G, cols, (T *)out, slots, d.groups, d.share);
    timing_after(st);
    return hipGetLastError();
}

template <typename T, typename O, int BM, int BN, int WM, int WN>
hipError_t unit_mats(const void *dY, const void *X, int64_t m, int32_t d, const int32_t *offsets,
                     int64_t G, int32_t cols, int piece, void *dW, int parts, hipStream_t st) {
    const dim3 grid(tile::grid_of(G * parts * tiles_of(cols, BM) * tiles_of(d, BN)));
    const dim3 block(WM * WN * 64);
    auto go = [&](auto pc) {
        static const tile::FormName name("k_unit_mats", BM, BN, decltype(pc)::value);
        timing_before(st, name.text);
        hipLaunchKernelGGL((k_unit_mats<T, O, BM, BN, WM, WN, decltype(pc)::value>), grid, block, 0,
                           st, (const T *)dY, (const T *)X, m, d, offsets, G, cols, (O *)dW, parts);
        timing_after(st);
    };
    by_piece<T, BM>(piece, go);
    return hipGetLastError();
}

}  // namespace

// Which tile, from the rows a unit has on average (r) and the number of tiles; in
// brackets us of the tile taken and of its neighbour, bf16 unless said.
//   few.h      r <= 16, and
//              - tiles of 64 x 64 are two for a CU at most (16 rows to 8 units of 2,048 x
//                2,048: 16.6, 64 x 64 28.7; to 16 of them 128 rows 31, 36, 256 47, 36; to
//                64 of them 128 rows 112, 113, 256 147, 131; at odd addresses 64 to 16 of
//                1,027 x 1,025 24, 25), or fp32 has r <= 8, since its tiles' matrix
//                instructions are mostly padding (256 to 64 of 1,024 x 1,024: 53, 64 x 64
//                75; 512 67, 75; 1,024 103, 74);
//              - and its empty workgroups cost less than the tiles' steps along k.  It
//                launches `groups` of them for every unit, at 3.1 us for a thousand that
//                find no rows; a step, 128 bytes of k, takes a tile 0.5 us in 16 bits and 1
//                in fp32 (1 row to 64 of 2,048 x 1,024: 27, 64 x 64 8; 1 to 64 of 1,024 x
//                4,096: 16.5 and 32, f32 19 and 72)
//   256 x 256  r >= 128 and a tile for every CU (64 units of 1,024 x 1,024, r = 150: 39,
//              128 x 128 48; 256 of 2,048 x 2,048: 546 and 668, r = 200 573 and 696; r = 96:
//              454 and 438, of 1,024 x 1,024 145 and 141); 16-byte addresses only (through
//              registers, 20,000 rows to 60 of 1,027 x 1,027: 141, 128 x 128 117)
//   128 x 128  r >= 96 and two for every CU (256 of 2,048 x 2,048, r = 96: 438, 64 x 128
//              512; r = 48: 426 and 424)
//   64 x 128   fewer rows (of the same, r = 48: 424, 64 x 64 490); 64 x 64
//              at other addresses (2,501 rows to 60 of 257 x 515 f16: 14, 64 x 128 19)
//              and where tiles are few
// fp32 has 64 x 64 only: bound by its matrix instructions, larger ones gain nothing
// (16,384 rows to 16 of 2,048 x 2,048: 1,015, 128 x 128 1,043).
hipError_t launch_unit_rows(const void *A, int64_t m, int32_t K, int dtype, const void *W,
                            const int32_t *offsets, int64_t G, int32_t cols, bool across, void *out,
                            hipStream_t st, int n_cu) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int ES = (int)sizeof(T);
        const int piece = piece_of(addr(A), K, addr(W), across ? cols : K, ES);
        const bool aligned = piece == 16;
        const int64_t units = G < m ? G : m;  // that have rows, at most
        const int64_t r = m / units;
        auto tiles = [&](int bm, int bn) { return (m / bm + units / 2) * tiles_of(cols, bn); };
        if (!across && r <= 16) {
            const few::Deal deal = few::deal(tiles_of(cols, 16), units, (int64_t)K * ES, n_cu);
            const int64_t empty = slots_of(m, G, 16) * deal.groups;
            if (empty * 4 <= (int64_t)K * ES * (ES == 4 ? 10 : 5) &&
                ((ES == 4 && r <= 8) || units * tiles_of(cols, 64) <= 2 * (int64_t)n_cu))
                return unit_rows_few<T>(A, m, K, W, offsets, G, cols, deal, out, st);
        }
        if constexpr (ES == 2) {
            if (aligned && r >= 128 && tiles(256, 256) >= n_cu && !wasteful(cols))
                return unit_rows<T, 256, 256, 2, 4>(A, m, K, W, offsets, G, cols, across, piece,
                                                    out, st);
            if (r >= 96 && tiles(128, 128) >= 2 * (int64_t)n_cu)
                return unit_rows<T, 128, 128, 2, 2>(A, m, K, W, offsets, G, cols, across, piece,
                                                    out, st);
            if (aligned && units * tiles_of(cols, 128) >= n_cu)
                return unit_rows<T, 64, 128, 2, 2>(A, m, K, W, offsets, G, cols, across, piece,
                                                   out, st);
        }
        return unit_rows<T, 64, 64, 2, 2>(A, m, K, W, offsets, G, cols, across, piece, out, st);
    });
}

// Runs that a unit's rows are cut into for the matrices' gradient, 32 at most: enough for
// two tiles for every CU, of 128 x 128 if there are 64 of those and they pad little, else
// of 64 x 64 (fp32 has those alone, but is no slower with the runs that the large ones
// ask for: 65,536 rows to one unit of 1,024 x 1,024, 8 runs 1,018 us, 2 1,092), and so
// many rows on average that a run saves more than its sums cost to store and join (us in
// one run and in runs):
//   16 bits  1,024 rows (1 unit of 64 x 64, 2,048 rows: 13, 2 runs 11; 4,096: 21, 4 runs
//            11), and four runs where matrices hold more than 2^18 elements together and
//            rows move in pieces of 16 (16 units of 256 x 256, 1,024 rows each: 9.6, 8 runs
//            24; 2,048: 16, 2 runs 22; 4,096: 34, 4 runs 26; 4 of 515 x 263, 2,048 rows
//            through registers: 33, 2 runs 26)
//   fp32     128 rows and four runs up to 2^18 elements (4 units of 64 x 64, 512 rows each:
//            15.1, 4 runs 10.1; 256 rows 10.2, 2 runs 9.7), 1,024 rows beyond (16 of 256 x
//            256, 1,024 rows: 27, 2 runs 30; 4,096: 87, 4 runs 77)
static int64_t mats_tiles(int64_t G, int32_t cols, int32_t d, int b) {
    return G * tiles_of(cols, b) * tiles_of(d, b);
}
// tiles of 128 x 128 pad a matrix by a fifth more than those of 64 x 64 at most
static bool mats_filled(int64_t G, int32_t cols, int32_t d) {
    return mats_tiles(G, cols, d, 128) * 4 * 5 <= mats_tiles(G, cols, d, 64) * 6;
}
static bool mats_large(int64_t G, int32_t cols, int32_t d) {
    return mats_tiles(G, cols, d, 128) >= 64 && mats_filled(G, cols, d);
}
static int mats_parts(int64_t m, int64_t G, int32_t cols, int32_t d, int esize, int piece) {
    const int64_t tiles = mats_tiles(G, cols, d, mats_large(G, cols, d) ? 128 : 64);
    const int64_t want = (512 + tiles - 1) / tiles;
    if (want < 2) return 1;  // also: matrices whose elements 64 bits do not count
    const bool small = G * (int64_t)cols * d <= (1 << 18);
    const int64_t rows = small && esize == 4 ? 128 : 1024;
    const int64_t least = esize == 4 ? (small ? 4 : 2) : (small || piece != 16 ? 2 : 4);
    const int64_t most = m / G / rows, parts = want < most ? want : most;
    return (int)(most < least || parts < 1 ? 1 : parts > 32 ? 32 : parts);
}

// for rows of any type and boundary
size_t unit_mats_workspace(int64_t m, int64_t G, int32_t cols, int32_t d) {
    int parts = mats_parts(m, G, cols, d, 4, 16);
    for (const int piece : {16, 0}) {
        const int p = mats_parts(m, G, cols, d, 2, piece);
        if (p > parts) parts = p;
    }
    return parts > 1 ? (size_t)parts * (size_t)G * (size_t)cols * (size_t)d * 4 : 0;
}

// The same for the matrices' gradient, by the number of tiles: 256 x 256 if there are
// two for every CU (4,096 rows of 64 units of 1,024 x 1,024, 1,024 tiles: 37, as 128
// x 128; 65,536 of 128 of 2,048 x 2,048: 665, 128 x 128 784), 128 x 128 if there is
// one and it pads little (20,000 rows to 60 of 1,027 x 1,027 f16: 151, 64 x 64 200; 9,000
// to 100 of 260 x 130: 16.5, so 64 x 64 11.9; of 384 x 384: 15.4, 64 x 64 18.8).  Where
// tiles are few and units have many rows, the rows are cut into runs, which a second
// kernel joins (65,536 rows to 4 units of 64 x 64: 15, in one run 73; of 512 x 512: 47
// and 119).
hipError_t launch_unit_mats(const void *dY, const void *X, int64_t m, int32_t d, int dtype,
                            const int32_t *offsets, int64_t G, int32_t cols, int grad_dtype,
                            void *dW, void *ws, hipStream_t st, int n_cu) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int ES = (int)sizeof(T);
        const int piece = piece_of(addr(dY), cols, addr(X), d, ES);
        const int parts = mats_parts(m, G, cols, d, ES, piece);
        auto tiles = [&](int b) { return mats_tiles(G, cols, d, b); };
        auto go = [&](auto o) {
            using O = decltype(o);
            if (parts > 1) {
                auto sums = [&] {
                    if constexpr (ES == 2)
                        if (mats_large(G, cols, d))
                            return unit_mats<T, float, 128, 128, 2, 2>(dY, X, m, d, offsets, G, cols,
                                                                       piece, ws, parts, st);
                    return unit_mats<T, float, 64, 64, 2, 2>(dY, X, m, d, offsets, G, cols, piece,
                                                             ws, parts, st);
                };
                const hipError_t e = sums();
                if (e != hipSuccess) return e;
                const int64_t n = G * (int64_t)cols * d, want = (n + 255) / 256;
                const int64_t most = (int64_t)n_cu * 32;
                hipLaunchKernelGGL((k_unit_join<O>), dim3((unsigned)(want < most ? want : most)),
                                   dim3(256), 0, st, (const float *)ws, parts, n, (O *)dW);
                return hipGetLastError();
            }
            if constexpr (ES == 2) {
                if (piece == 16 && tiles(256) >= 2 * (int64_t)n_cu && !wasteful(cols) && !wasteful(d))
                    return unit_mats<T, O, 256, 256, 2, 4>(dY, X, m, d, offsets, G, cols, piece,
                                                           dW, 1, st);
                if (tiles(128) >= n_cu && mats_filled(G, cols, d))
                    return unit_mats<T, O, 128, 128, 2, 2>(dY, X, m, d, offsets, G, cols, piece,
                                                           dW, 1, st);
            }
            return unit_mats<T, O, 64, 64, 2, 2>(dY, X, m, d, offsets, G, cols, piece, dW, 1, st);
        };
        return grad_dtype == dtype ? go(T()) : go(float());
    });
}

}  // namespace vs
