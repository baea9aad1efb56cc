// rows.hip -- rows of a table by index, rows sent to their units and brought
// back with weights, and the gradients of both.
//
//   lookup            Y[i] = scale T[ids[i]]           (zeros: ids outside the table)
//   lookup backward   dT[g] = scale sum dY[order[p]], p = offsets[g] .. offsets[g+1]-1
//   route             Xs[slot[i k + j]] = X[i]
//   combine           Y[i] = sum_j w[i k + j] Ys[slot[i k + j]]
//   combine backward  dYs[slot[e]] = w[e] dY[e / k],  dw[e] = dY[e / k] . Ys[slot[e]]
//   route backward    combine with every weight 1
// All are bound by memory: a group of lanes takes a row, each lane one vector
// of it at a time.  Sums are fp32 in a fixed order and rounded once.  Indices
// come from device memory, so each is checked against its array before use.
#include <type_traits>

#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

// Lanes per row: the smallest power of two that covers a row's vectors, at
// most a wave.  A workgroup of 256 threads takes 256 / lanes rows at a time.
struct RowGrid {
    int lanes, log2_lanes;
    unsigned grid;
};
RowGrid row_grid(int64_t rows, int64_t vecs, int n_cu) {
    RowGrid g{1, 0, 1};
    while (g.lanes < 64 && g.lanes < vecs) g.lanes <<= 1, ++g.log2_lanes;
    const int64_t want = (rows * g.lanes + 255) / 256;
    const int64_t most = (int64_t)n_cu * 64;
    g.grid = (unsigned)(want < 1 ? 1 : want < most ? want : most);
    return g;
}

// 65,536 rows of 256 f32 out of 262,144: 22 us, 6.1 TB/s.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_row_lookup(const T *__restrict__ table, int64_t G,
                                                    int32_t d, const int32_t *__restrict__ ids,
                                                    int64_t n, float scale, T *__restrict__ Y,
                                                    int lsh) {
    using V = Vec<T, N>;
    const int lane = threadIdx.x & ((1 << lsh) - 1);
    const int64_t step = (int64_t)gridDim.x * (256 >> lsh);
    const int vecs = d / N;
    for (int64_t i = (int64_t)blockIdx.x * (256 >> lsh) + (threadIdx.x >> lsh); i < n; i += step) {
        const int64_t id = ids[i];
        const bool ok = id >= 0 && id < G;
        const V *src = reinterpret_cast<const V *>(table + (ok ? id : 0) * d);
        V *dst = reinterpret_cast<V *>(Y + i * d);
        for (int c = lane; c < vecs; c += 1 << lsh) {
            V v;
            if (ok) v = src[c];
#pragma unroll
            for (int t = 0; t < N; ++t) v.v[t] = ok ? narrow<T>(scale * widen(v.v[t])) : T(0.0f);
            store_once(dst + c, v);
        }
    }
}

// ---- lookup backward -------------------------------------------------------
//
// The sorted order cuts into one run of rows per unit, summed by the lanes of
// one unit.  Units differ widely in length (padding, common tokens), so one
// with more than `run` rows is cut at multiples of `run` places: each piece's
// sum goes to the workspace in fp32 and a second kernel adds a unit's pieces,
// always in the same order.  A long unit covers the first or the last place
// of every stretch of `run` places it touches, so a stretch holds at most two
// pieces: part 0 of the unit at its first place, part 1 of the one at its
// last if that unit starts inside the stretch.
//
// run is 64, and 16 for few rows, where a long unit's rows would come one
// behind the other with the GPU idle.  Both kernels, us, 16 / 64 (even ids; in
// brackets frequencies about 1 / rank): 1,023 x 257 f16 into 1,000 units 6.5 /
// 6.5 (9.4 / 12.1); 2,048 x 256 f32 into 100 units 12.3 / 7.2 (10.0 / 11.8);
// 4,096 x 768 bf16 into 64 units 13.5 / 23.8 (16.1 / 22.9); 16,384 x 256 f32
// into 256 units 13.6 / 21.1 (15.7 / 18.4), so 16 would pay for some rows more;
// 131,072 x 768 bf16 into 65,536 units 85 / 75 (97 / 84).
inline int run_of(int64_t n) { return n <= 4096 ? 16 : 64; }
constexpr int kAhead = 8;        // rows in flight per lane
constexpr int kJoinWaves = 8;

struct Span {
    int64_t lo, hi;
};
__device__ __forceinline__ Span unit_span(const int32_t *__restrict__ offsets, int64_t g,
                                          int64_t n) {
    Span s{offsets[g], offsets[g + 1]};
    s.lo = s.lo < 0 ? 0 : s.lo;
    s.hi = s.hi > n ? n : s.hi;
    return s;
}

// unit of the entry at place p, or -1
__device__ __forceinline__ int64_t unit_at(const int32_t *__restrict__ ids,
                                           const int32_t *__restrict__ order, int64_t p, int64_t n,
                                           int64_t G) {
    const int64_t i = order[p];
    if (i < 0 || i >= n) return -1;
    const int64_t g = ids[i];
    return g < G ? g : -1;
}

// C rows at places p .. p + C - 1, all loads issued before the first use (an
// index that does not fit loads row 0 and adds nothing)
template <typename T, int N, int C>
__device__ __forceinline__ void add_rows(const T *__restrict__ dY, int64_t n, int32_t d,
                                         const int32_t *__restrict__ order, int64_t p, int c,
                                         float (&acc)[N]) {
    using V = Vec<T, N>;
    V v[C];
    bool ok[C];
#pragma unroll
    for (int a = 0; a < C; ++a) {
        const int64_t i = order[p + a];
        ok[a] = i >= 0 && i < n;
        v[a] = reinterpret_cast<const V *>(dY + (ok[a] ? i : 0) * d)[c];
    }
#pragma unroll
    for (int a = 0; a < C; ++a)
#pragma unroll
        for (int t = 0; t < N; ++t) acc[t] += ok[a] ? widen(v[a].v[t]) : 0.0f;
}

template <typename T, int N>
__device__ __forceinline__ void sum_rows(const T *__restrict__ dY, int64_t n, int32_t d,
                                         const int32_t *__restrict__ order, Span s, int c,
                                         float (&acc)[N]) {
    int64_t p = s.lo;
    for (; p + kAhead <= s.hi; p += kAhead) add_rows<T, N, kAhead>(dY, n, d, order, p, c, acc);
    static_assert(kAhead == 8, "the rest is at most 4 + 2 + 1 rows");
    const int64_t left = s.hi - p;  // negative for a span that holds nothing
    if (left >= 4) {
        add_rows<T, N, 4>(dY, n, d, order, p, c, acc);
        p += 4;
    }
    if (p + 2 <= s.hi) {
        add_rows<T, N, 2>(dY, n, d, order, p, c, acc);
        p += 2;
    }
    if (p < s.hi) add_rows<T, N, 1>(dY, n, d, order, p, c, acc);
}

template <typename O, int N>
__device__ __forceinline__ void store_row(O *__restrict__ dT, int64_t g, int32_t d, int c,
                                          float scale, const float (&acc)[N]) {
    Vec<O, N> o;
#pragma unroll
    for (int t = 0; t < N; ++t) o.v[t] = narrow<O>(scale * acc[t]);
    store_once(reinterpret_cast<Vec<O, N> *>(dT + g * d) + c, o);
}

// Workgroups 0 .. piece_blocks - 1 sum the pieces of long units, the others a
// short unit per group of lanes.  Neighbouring groups take the blocks of
// columns of one row, so that a row is read in one go.  Bound by memory:
// 65,536 x 256 f32 rows into 16,384 units in 15.5 us (5.4 TB/s); 131,072 x 768
// bf16 rows into 65,536 units, a few of which hold half of them, in 73 us (short
// random rows, 4.1 TB/s) and 10 us for the join.  Rows of odd width in 16 bits
// go 2 bytes a lane: 65,536 x 767 bf16 into 16,384 units 79 us, x 768 30 us.
// Several units per group or several vectors per lane came out slower (101 and
// 87 to 90 us for 83).
template <typename T, typename O, int N>
__global__ __launch_bounds__(256) void k_row_lookup_bwd(
    const T *__restrict__ dY, int64_t n, int32_t d, const int32_t *__restrict__ ids,
    const int32_t *__restrict__ order, const int32_t *__restrict__ offsets, int64_t G, float scale,
    O *__restrict__ dT, float *__restrict__ part, int run, unsigned piece_blocks, int lsh,
    unsigned cols) {
    const int lane = threadIdx.x & ((1 << lsh) - 1);
    const int per = 256 >> lsh;
    const int vecs = d / N;
    if (blockIdx.x < piece_blocks) {
        int64_t kept = offsets[G];
        kept = kept > n ? n : kept;
        const int64_t step = (int64_t)piece_blocks * per;
        for (int64_t item = (int64_t)blockIdx.x * per + (threadIdx.x >> lsh);; item += step) {
            const int64_t s = item / cols;
            if (s * run >= kept) break;
            const int c = ((int)(item - s * cols) << lsh) + lane;
            if (c >= vecs) continue;
            const int64_t p0 = s * run, p1 = p0 + run < kept ? p0 + run : kept;
            const int64_t g0 = unit_at(ids, order, p0, n, G);
            const int64_t g1 = unit_at(ids, order, p1 - 1, n, G);
            for (int b = 0; b < 2; ++b) {
                const int64_t g = b ? g1 : g0;
                if (g < 0 || (b && g1 == g0)) continue;
                Span u = unit_span(offsets, g, n);
                if (u.hi - u.lo <= run) continue;
                u.lo = u.lo > p0 ? u.lo : p0;
                u.hi = u.hi < p1 ? u.hi : p1;
                float acc[N] = {};
                sum_rows<T, N>(dY, n, d, order, u, c, acc);
                Vec<float, N> o;
#pragma unroll
                for (int t = 0; t < N; ++t) o.v[t] = acc[t];
                reinterpret_cast<Vec<float, N> *>(part + (2 * s + b) * d)[c] = o;
            }
        }
        return;
    }
    const int64_t step = (int64_t)(gridDim.x - piece_blocks) * per;
    for (int64_t item = (int64_t)(blockIdx.x - piece_blocks) * per + (threadIdx.x >> lsh);;
         item += step) {
        const int64_t g = item / cols;
        if (g >= G) break;
        const int c = ((int)(item - g * cols) << lsh) + lane;
        if (c >= vecs) continue;
        const Span u = unit_span(offsets, g, n);
        if (u.hi - u.lo > run) continue;
        float acc[N] = {};
        sum_rows<T, N>(dY, n, d, order, u, c, acc);
        store_row<O, N>(dT, g, d, c, u.hi > u.lo ? scale : 0.0f, acc);
    }
}

// A workgroup looks at kJoinWaves stretches, a wave each, for long units that
// start there (most hold none); for each it found, its waves take the unit's
// pieces in turn, and the waves' sums are added in their order.  It takes 3.8 us
// where it finds nothing (65,536 rows), and as long as its longest unit needs,
// since one workgroup a block of columns adds that unit's pieces: 131,072 x 256
// f32 rows in two units 13.6 us after 28, 1,048,576 in one 228 us after 202.
template <typename O, int N>
__global__ __launch_bounds__(kJoinWaves * 64) void k_row_lookup_join(
    int64_t n, int32_t d, const int32_t *__restrict__ ids, const int32_t *__restrict__ order,
    const int32_t *__restrict__ offsets, int64_t G, float scale, const float *__restrict__ part,
    int run, O *__restrict__ dT) {
    using V = Vec<float, N>;
    __shared__ V sums[kJoinWaves][64];
    __shared__ int32_t unit[kJoinWaves];  // -1: no long unit starts in the stretch
    __shared__ Span span[kJoinWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c = (int)blockIdx.y * 64 + lane;
    const bool in = c < d / N;
    int64_t kept = offsets[G];
    kept = kept > n ? n : kept;
    for (int64_t s0 = (int64_t)blockIdx.x * kJoinWaves; s0 * run < kept;
         s0 += (int64_t)gridDim.x * kJoinWaves) {
        if (lane == 0) {
            const int64_t p0 = (s0 + w) * run, p1 = p0 + run < kept ? p0 + run : kept;
            int64_t g = p0 < kept ? unit_at(ids, order, p1 - 1, n, G) : -1;
            if (g >= 0) {
                const Span u = unit_span(offsets, g, n);
                if (u.hi - u.lo <= run || u.lo < p0 || u.lo >= p1) g = -1;
                span[w] = u;
            }
            unit[w] = (int32_t)g;
        }
        __syncthreads();
        for (int f = 0; f < kJoinWaves; ++f) {
            const int64_t g = unit[f];
            if (g < 0) continue;  // uniform over the workgroup
            const int64_t s = s0 + f;
            const Span u = span[f];
            const int64_t last = (u.hi - 1) / run;
            V sum;
#pragma unroll
            for (int t = 0; t < N; ++t) sum.v[t] = 0.0f;
            if (in)
#pragma unroll 8
                for (int64_t q = s + w; q <= last; q += kJoinWaves) {
                    const int64_t slot = 2 * q + (q == s && u.lo > s * run ? 1 : 0);
                    const V v = reinterpret_cast<const V *>(part + slot * d)[c];
#pragma unroll
                    for (int t = 0; t < N; ++t) sum.v[t] += v.v[t];
                }
            sums[w][lane] = sum;
            __syncthreads();
            if (w == 0 && in) {
                float acc[N];
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    acc[t] = sums[0][lane].v[t];
                    for (int v = 1; v < kJoinWaves; ++v) acc[t] += sums[v][lane].v[t];
                }
                store_row<O, N>(dT, g, d, c, scale, acc);
            }
            __syncthreads();
        }
        __syncthreads();  // `unit` is written again in the next turn
    }
}

// rows kept .. m-1 of a unit-ordered matrix (those of no unit) set to zero
template <typename T, int N>
__device__ __forceinline__ void zero_tail(T *__restrict__ Xs, int64_t kept, int64_t m, int32_t d,
                                          int lane, int lsh, int64_t row, int64_t step) {
    if (kept < 0) kept = 0;
    for (int64_t p = kept + row; p < m; p += step)
        for (int c = lane; c < d / N; c += 1 << lsh) {
            Vec<T, N> z;
#pragma unroll
            for (int t = 0; t < N; ++t) z.v[t] = T(0.0f);
            reinterpret_cast<Vec<T, N> *>(Xs + p * d)[c] = z;
        }
}

// UV vectors of a row are loaded before they are stored k times over, past the
// caches (65,536 x 2,048 bf16 rows of 16,384, calls back to back, so that X
// stays in the last-level cache: 87 us one at a time through them, 53 us four
// past them; 64 us behind other kernels, 5.2 TB/s).
template <typename T, int N, int UV>
__global__ __launch_bounds__(256) void k_route_rows(const T *__restrict__ X, int64_t n, int32_t d,
                                                    const int32_t *__restrict__ slot,
                                                    const int32_t *__restrict__ kept, int32_t k,
                                                    T *__restrict__ Xs, int lsh) {
    using V = Vec<T, N>;
    const int lane = threadIdx.x & ((1 << lsh) - 1);
    const int64_t step = (int64_t)gridDim.x * (256 >> lsh);
    const int64_t row = (int64_t)blockIdx.x * (256 >> lsh) + (threadIdx.x >> lsh);
    const int64_t m = n * k;
    const int vecs = d / N;
    const int width = 1 << lsh;
    for (int64_t i = row; i < n; i += step) {
        const V *src = reinterpret_cast<const V *>(X + i * d);
        for (int c = lane; c < vecs; c += UV * width) {
            V v[UV];
#pragma unroll
            for (int u = 0; u < UV; ++u) v[u] = src[c + u * width < vecs ? c + u * width : c];
            for (int j = 0; j < k; ++j) {
                const int64_t p = slot[i * k + j];
                if (p < 0 || p >= m) continue;
                V *dst = reinterpret_cast<V *>(Xs + p * d);
#pragma unroll
                for (int u = 0; u < UV; ++u)
                    if (c + u * width < vecs) store_once(dst + c + u * width, v[u]);
            }
        }
    }
    zero_tail<T, N>(Xs, *kept, m, d, lane, lsh, row, step);
}

// A chunk of a row's entries: places (-1: dropped) and weights, loaded at once.
template <int KC>
struct Entries {
    int64_t p[KC];
    float w[KC];
    __device__ __forceinline__ void load(const int32_t *__restrict__ slot,
                                         const float *__restrict__ weights, int64_t e0, int left,
                                         int64_t m) {
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            const int64_t q = j < left ? slot[e0 + j] : -1;
            p[j] = q >= 0 && q < m ? q : -1;
            w[j] = weights && j < left ? weights[e0 + j] : 1.0f;
        }
    }
    // the row to load: row 0, whose values are not used, for a dropped entry
    __device__ __forceinline__ int64_t at(int j) const { return p[j] >= 0 ? p[j] : 0; }
};

// Two vectors of the row and KC of its entries are in flight per lane (65,536 x
// 2,048 bf16 rows two to one, past the caches: 70 us, 5.7 TB/s; one at a time
// through them 110 us).
template <typename T, int N, int KC>
__global__ __launch_bounds__(256) void k_combine_rows(const T *__restrict__ Ys, int64_t n,
                                                      int32_t d, const int32_t *__restrict__ slot,
                                                      const float *__restrict__ weights, int32_t k,
                                                      T *__restrict__ Y, int lsh) {
    using V = Vec<T, N>;
    const int lane = threadIdx.x & ((1 << lsh) - 1);
    const int64_t step = (int64_t)gridDim.x * (256 >> lsh);
    const int64_t m = n * k;
    const int vecs = d / N, width = 1 << lsh;
    for (int64_t i = (int64_t)blockIdx.x * (256 >> lsh) + (threadIdx.x >> lsh); i < n; i += step) {
        Entries<KC> en;
        en.load(slot, weights, i * k, k, m);
        for (int c = lane; c < vecs; c += 2 * width) {
            const int c1 = c + width < vecs ? c + width : c;  // the last one alone: twice
            float acc[2][N] = {};
            for (int j0 = 0; j0 < k; j0 += KC) {
                if (k > KC) en.load(slot, weights, i * k + j0, k - j0, m);
                V v[2][KC];
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    const V *src = reinterpret_cast<const V *>(Ys + en.at(j) * d);
                    v[0][j] = load_once(src + c);
                    v[1][j] = load_once(src + c1);
                }
#pragma unroll
                for (int j = 0; j < KC; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < N; ++t) {
                            const float s = __builtin_fmaf(en.w[j], widen(v[h][j].v[t]), acc[h][t]);
                            acc[h][t] = en.p[j] >= 0 ? s : acc[h][t];
                        }
            }
            V o[2];
#pragma unroll
            for (int t = 0; t < N; ++t) {
                o[0].v[t] = narrow<T>(acc[0][t]);
                o[1].v[t] = narrow<T>(acc[1][t]);
            }
            V *dst = reinterpret_cast<V *>(Y + i * d);
            store_once(dst + c, o[0]);
            if (c1 != c) store_once(dst + c1, o[1]);
        }
    }
}

// dY is read once for its KC entries; two vectors of each are in flight and all
// stores come behind the loads, which would else wait for them (65,536 x 2,048
// bf16 rows four to one, calls back to back: 118 us, one vector at a time
// through the caches 139 us; behind other kernels 127 us, 4.8 TB/s).
template <typename T, int N, int KC>
__global__ __launch_bounds__(256) void k_combine_rows_bwd(
    const T *__restrict__ dY, const T *__restrict__ Ys, int64_t n, int32_t d,
    const int32_t *__restrict__ slot, const float *__restrict__ weights,
    const int32_t *__restrict__ kept, int32_t k, T *__restrict__ dYs, float *__restrict__ dw,
    int lsh) {
    using V = Vec<T, N>;
    const int lane = threadIdx.x & ((1 << lsh) - 1);
    const int64_t step = (int64_t)gridDim.x * (256 >> lsh);
    const int64_t row = (int64_t)blockIdx.x * (256 >> lsh) + (threadIdx.x >> lsh);
    const int64_t m = n * k;
    const int vecs = d / N, width = 1 << lsh;
    for (int64_t i = row; i < n; i += step) {
        for (int j0 = 0; j0 < k; j0 += KC) {
            Entries<KC> en;
            en.load(slot, weights, i * k + j0, k - j0, m);
            float dot[KC] = {};
            for (int c = lane; c < vecs; c += 2 * width) {
                V a[2], b[KC][2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int cu = c + u * width < vecs ? c + u * width : c;
                    a[u] = reinterpret_cast<const V *>(dY + i * d)[cu];
#pragma unroll
                    for (int j = 0; j < KC; ++j)
                        b[j][u] = load_once(reinterpret_cast<const V *>(Ys + en.at(j) * d) + cu);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (c + u * width >= vecs) break;
#pragma unroll
                    for (int j = 0; j < KC; ++j) {
                        if (en.p[j] < 0) continue;
                        V o;
#pragma unroll
                        for (int t = 0; t < N; ++t) {
                            dot[j] = __builtin_fmaf(widen(a[u].v[t]), widen(b[j][u].v[t]), dot[j]);
                            o.v[t] = narrow<T>(en.w[j] * widen(a[u].v[t]));
                        }
                        store_once(reinterpret_cast<V *>(dYs + en.p[j] * d) + c + u * width, o);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < KC; ++j)
                for (int s = 1; s < 1 << lsh; s <<= 1) dot[j] += __shfl_xor(dot[j], s);
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < KC; ++j)
                    if (j0 + j < k) dw[i * k + j0 + j] = dot[j];
        }
    }
    zero_tail<T, N>(dYs, *kept, m, d, lane, lsh, row, step);
}

// f(element type, elements per access) for a row type; N covers 16 bytes and
// the smaller powers of two
template <typename T, typename F>
hipError_t with_vec(int n, F f) {
    switch (n) {
    case 8:
        if constexpr (sizeof(T) == 2) return f(T(), std::integral_constant<int, 8>());
        return hipErrorInvalidValue;
    case 4: return f(T(), std::integral_constant<int, 4>());
    case 2: return f(T(), std::integral_constant<int, 2>());
    default: return f(T(), std::integral_constant<int, 1>());
    }
}
template <typename F>
hipError_t with_type(int dtype, int n, F f) {
    switch (dtype) {
    case kF32: return with_vec<float>(n, f);
    case kF16: return with_vec<_Float16>(n, f);
    default: return with_vec<__bf16>(n, f);
    }
}

// f(vectors a lane takes at a time) for rows of `vecs` vectors and 64 lanes: as
// many as the row has for it, four at most.  It matters for long rows (1 / 2 / 4
// at a time, us: 16,384 x 4 rows of 256 vectors 64 / 58 / 52, 16,384 x 2 of 192
// 24.3 / 24.2 / 23.6); 65,536 x 2 rows of 64 and 32,768 x 2 of 128 take 31 us
// with any.
template <typename F>
hipError_t with_vectors(int vecs, F f) {
    if (vecs <= 64) return f(std::integral_constant<int, 1>());
    if (vecs <= 128) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 4>());
}

// f(entries taken at a time) for rows of k entries
template <typename F>
hipError_t with_entries(int32_t k, F f) {
    if (k == 1) return f(std::integral_constant<int, 1>());
    if (k == 2) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 4>());
}

inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

hipError_t launch_row_lookup(const void *table, int64_t G, int32_t d, int dtype,
                             const int32_t *ids, int64_t n, float scale, void *Y, hipStream_t st,
                             int n_cu) {
    const int nv = vec_elems(d, dtype_bytes(dtype), addr(table) | addr(Y));
    const RowGrid g = row_grid(n, d / nv, n_cu);
    return with_type(dtype, nv, [&](auto t, auto nc) {
        using T = decltype(t);
        timing_before(st, "k_row_lookup");
        hipLaunchKernelGGL((k_row_lookup<T, decltype(nc)::value>), dim3(g.grid), dim3(256), 0, st,
                           (const T *)table, G, d, ids, n, scale, (T *)Y, g.log2_lanes);
        timing_after(st);
        return hipGetLastError();
    });
}

// Two fp32 rows per stretch of run_of(n) places; none where no unit can be long.
size_t row_lookup_bwd_workspace(int64_t n, int32_t d) {
    const int run = run_of(n);
    if (n <= run) return 0;
    const size_t stretches = (size_t)((n + run - 1) / run);
    return stretches * 2 * (size_t)d * 4;
}

static int idle_lanes(int vecs, int lsh) {
    const int lanes = 1 << lsh;
    return (vecs + lanes - 1) / lanes * lanes - vecs;
}

template <typename T, typename O, int N>
static hipError_t lookup_bwd(const void *dY, int64_t n, int32_t d, const int32_t *ids,
                             const int32_t *order, const int32_t *offsets, int64_t G, float scale,
                             void *dT, float *part, hipStream_t st, int n_cu) {
    const int vecs = d / N;
    // lanes per row: a wave, or half or a quarter of one where that leaves
    // fewer lanes without a vector in the last block of columns
    int lsh = 0;
    while (lsh < 6 && (1 << lsh) < vecs) ++lsh;
    for (int less = lsh - 1; vecs > 64 && less >= 4; --less)
        if (idle_lanes(vecs, less) < idle_lanes(vecs, lsh)) lsh = less;
    const int per = 256 >> lsh;
    const unsigned cols = (unsigned)((vecs + (1 << lsh) - 1) >> lsh);
    const int run = run_of(n);
    const int64_t stretches = (n + run - 1) / run, most = (int64_t)n_cu * 32;
    const int64_t pb = (stretches * cols + per - 1) / per;
    const int64_t ub = (G * cols + per - 1) / per;
    const unsigned pieces = (unsigned)(pb < most ? pb : most);
    const unsigned units = (unsigned)(ub < most ? ub : most);
    timing_before(st, "k_row_lookup_bwd");
    hipLaunchKernelGGL((k_row_lookup_bwd<T, O, N>), dim3(pieces + units), dim3(256), 0, st,
                       (const T *)dY, n, d, ids, order, offsets, G, scale, (O *)dT, part, run, pieces,
                       lsh, cols);
    timing_after(st);
    if (n > run) {  // else no unit is long
        const unsigned jc = (unsigned)((vecs + 63) / 64);
        const int64_t looks = (stretches + kJoinWaves - 1) / kJoinWaves;
        hipLaunchKernelGGL((k_row_lookup_join<O, N>),
                           dim3((unsigned)(looks < most ? looks : most), jc),
                           dim3(kJoinWaves * 64), 0, st, n, d, ids, order, offsets, G, scale, part,
                           run, (O *)dT);
    }
    return hipGetLastError();
}

hipError_t launch_row_lookup_bwd(const void *dY, int64_t n, int32_t d, int dtype,
                                 const int32_t *ids, const int32_t *order, const int32_t *offsets,
                                 int64_t G, float scale, int grad_dtype, void *dT, void *ws,
                                 hipStream_t st, int n_cu) {
    // one vector length for both sides: the shorter of what each allows
    int nv = vec_elems(d, dtype_bytes(dtype), addr(dY));
    const int no = vec_elems(d, dtype_bytes(grad_dtype), addr(dT));
    if (no < nv) nv = no;
    return with_type(dtype, nv, [&](auto t, auto nc) {
        using T = decltype(t);
        constexpr int N = decltype(nc)::value;
        if (grad_dtype == dtype)
            return lookup_bwd<T, T, N>(dY, n, d, ids, order, offsets, G, scale, dT, (float *)ws,
                                       st, n_cu);
        // N is 4 at most for fp32 rows
        if constexpr (N <= 4)
            return lookup_bwd<T, float, N>(dY, n, d, ids, order, offsets, G, scale, dT,
                                           (float *)ws, st, n_cu);
        return hipErrorInvalidValue;
    });
}

hipError_t launch_route_rows(const void *X, int64_t n, int32_t d, int dtype, const int32_t *slot,
                             const int32_t *kept, int32_t k, void *Xs, hipStream_t st, int n_cu) {
    const int nv = vec_elems(d, dtype_bytes(dtype), addr(X) | addr(Xs));
    const RowGrid g = row_grid(n, d / nv, n_cu);
    return with_type(dtype, nv, [&](auto t, auto nc) {
        using T = decltype(t);
        constexpr int N = decltype(nc)::value;
        return with_vectors(d / nv, [&](auto uv) {
            timing_before(st, "k_route_rows");
            hipLaunchKernelGGL((k_route_rows<T, N, decltype(uv)::value>), dim3(g.grid), dim3(256),
                               0, st, (const T *)X, n, d, slot, kept, k, (T *)Xs, g.log2_lanes);
            timing_after(st);
            return hipGetLastError();
        });
    });
}

hipError_t launch_combine_rows(const void *Ys, int64_t n, int32_t d, int dtype,
                               const int32_t *slot, const float *weights, int32_t k, void *Y,
                               hipStream_t st, int n_cu) {
    const int nv = vec_elems(d, dtype_bytes(dtype), addr(Ys) | addr(Y));
    const RowGrid g = row_grid(n, d / nv, n_cu);
    return with_type(dtype, nv, [&](auto t, auto nc) {
        using T = decltype(t);
        constexpr int N = decltype(nc)::value;
        return with_entries(k, [&](auto kc) {
            timing_before(st, "k_combine_rows");
            hipLaunchKernelGGL((k_combine_rows<T, N, decltype(kc)::value>), dim3(g.grid),
                               dim3(256), 0, st, (const T *)Ys, n, d, slot, weights, k, (T *)Y,
                               g.log2_lanes);
            timing_after(st);
            return hipGetLastError();
        });
    });
}

hipError_t launch_combine_rows_bwd(const void *dY, const void *Ys, int64_t n, int32_t d, int dtype,
                                   const int32_t *slot, const float *weights, const int32_t *kept,
                                   int32_t k, void *dYs, float *dw, hipStream_t st, int n_cu) {
    const int nv = vec_elems(d, dtype_bytes(dtype), addr(dY) | addr(Ys) | addr(dYs));
    const RowGrid g = row_grid(n, d / nv, n_cu);
    return with_type(dtype, nv, [&](auto t, auto nc) {
        using T = decltype(t);
        constexpr int N = decltype(nc)::value;
        return with_entries(k, [&](auto kc) {
            timing_before(st, "k_combine_rows_bwd");
            hipLaunchKernelGGL((k_combine_rows_bwd<T, N, decltype(kc)::value>), dim3(g.grid),
                               dim3(256), 0, st, (const T *)dY, (const T *)Ys, n, d, slot,
                               weights, kept, k, (T *)dYs, dw, g.log2_lanes);
            timing_after(st);
            return hipGetLastError();
        });
    });
}

}  // namespace vs
