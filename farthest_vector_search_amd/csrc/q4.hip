// q4.hip -- a candidate table in 4-bit codes and the scores of queries over it.
//
// Row i of the table stands for v[i, k] = s[i, k / group] (c[i, k] - 8), codes
// c in 0 .. 15, one 16-bit scale per group of 32, 64 or 128 columns.  Scores
// are the dot products y[q, i] = sum_k x[q, k] v[i, k], one group at a time:
//   y = sum_g s_g (sum_{k in g} (16 + c_k) x_k - 24 sum_{k in g} x_k).
// 16 + c is a 16-bit float made by putting the four code bits behind its
// leading one, so a pair of codes costs one shift and one and-or; the matrix
// instruction multiplies it exactly, and a second one with the constant -24
// supplies the other sum.  Both start from zero in every group, in fp32.
//
// The matrix instruction is v_mfma_f32_16x16x32: 16 table rows x 16 columns of
// queries.  f16 queries use its f16 form.  bf16 queries use the bf16 form;
// f32 queries too, as three bf16 columns that add up to the query exactly
// (8 + 8 + 8 bits), five queries to a tile of 16 columns.
//
// Layout of the table: blocks of 16 rows x 128 columns, a row block's one
// behind the other.  A block is 1 KiB of codes in the order of the lanes: lane
// l (row l % 16, part l / 16) holds 16 bytes, and its 32-bit word t holds
// columns 32 t + 8 (l / 16) .. + 7 of the block, what the lane feeds to the
// t-th instruction.  Columns 2 j and 2 j + 1 of the eight sit at bits 4 j and
// 16 + 4 j.  Its scales follow in four runs (rows 4 r .. 4 r + 3) of
// [group][row], in the same stretch of memory (an array of their own cost
// 2 us of 47 at 65,536 x 4,096, group 128).
#include <type_traits>

#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

constexpr int kBlockRows = 16, kBlockCols = 128;

inline int64_t row_blocks(int64_t nc) { return (nc + kBlockRows - 1) / kBlockRows; }
inline int64_t col_blocks(int64_t d) { return (d + kBlockCols - 1) / kBlockCols; }

// ---- quantize: codes and scales of a plain table ---------------------------
//
// One lane per two columns (a byte of codes); the lanes of a group share its
// largest magnitude.  s = max / 7 rounded to the scale type and held inside
// its finite range; c = rint(v / s) held in -8 .. 7, ties to even, plus 8.  No
// code stands for a NaN, so a group that holds one gets a NaN for its scale
// (and codes of 8): its row's scores are NaN, as the row's products are.
// Two columns and two divisions a lane: 65,536 x 4,096 bf16 (group 128) 541 us,
// 1.3 TB/s; it runs once per table.
__device__ __forceinline__ float larger(float a, float b) {  // a NaN if either is one
    return a >= b || a != a ? a : b;
}

template <typename T, typename S>
__global__ __launch_bounds__(256) void k_q4_quantize(const T *__restrict__ table, int64_t nc,
                                                     int32_t d, int group,
                                                     uint8_t *__restrict__ codes,
                                                     S *__restrict__ scales) {
    const int lanes = group / 2;
    const int64_t groups = (d + group - 1) / group;
    const int64_t bytes = ((int64_t)d + 1) / 2;
    const int64_t total = nc * groups;
    const int sub = threadIdx.x & (lanes - 1);
    const int per = 256 / lanes;
    const float top = sizeof(S) == 2 && std::is_same<S, _Float16>::value ? 65504.0f : 3.3895314e38f;
    for (int64_t e = (int64_t)blockIdx.x * per + threadIdx.x / lanes; e < total;
         e += (int64_t)gridDim.x * per) {
        const int64_t row = e / groups, g = e - row * groups;
        const int64_t k = g * group + 2 * sub;
        const T *src = table + row * d;
        const float v0 = k < d ? widen(src[k]) : 0.0f;
        const float v1 = k + 1 < d ? widen(src[k + 1]) : 0.0f;
        float m = larger(fabsf(v0), fabsf(v1));
        for (int s = 1; s < lanes; s <<= 1) m = larger(m, __shfl_xor(m, s));
        const S sc = narrow<S>(m / 7.0f > top ? top : m / 7.0f);
        const float s = widen(sc);
        int c0 = 8, c1 = 8;
        if (s > 0.0f) {
            c0 = 8 + (int)fminf(fmaxf(rintf(v0 / s), -8.0f), 7.0f);
            c1 = 8 + (int)fminf(fmaxf(rintf(v1 / s), -8.0f), 7.0f);
        }
        if (k < d) codes[row * bytes + k / 2] = (uint8_t)(c0 | c1 << 4);
        if (sub == 0) scales[row * groups + g] = sc;
    }
}

// ---- layout: plain codes and scales into blocks ------------------------------
//
// words: every row of codes starts on a 4-byte boundary.  A word a thread:
// 65,536 x 4,096 (group 128) 120 us, 2.3 TB/s; it runs once per table.

constexpr int block_bytes(int per) { return 1024 + kBlockRows * 2 * per; }  // per: groups a block

__global__ __launch_bounds__(256) void k_q4_layout(const uint8_t *__restrict__ codes,
                                                   const uint16_t *__restrict__ scales, int64_t nc,
                                                   int32_t d, int group, int64_t nrb, int64_t ncb,
                                                   uint8_t *__restrict__ out, int words) {
    const int64_t bytes = ((int64_t)d + 1) / 2;
    const int per = kBlockCols / group;
    const int64_t groups = (d + group - 1) / group;
    // a workgroup per block: 256 words of codes, 16 x per scales
    for (int64_t blk = blockIdx.x; blk < nrb * ncb; blk += gridDim.x) {
        const int64_t rb = blk / ncb, cb = blk - rb * ncb;
        uint8_t *to = out + blk * block_bytes(per);
        const int lane = (int)threadIdx.x >> 2, t = (int)threadIdx.x & 3;
        const int64_t row = rb * kBlockRows + (lane & 15);
        const int64_t k0 = cb * kBlockCols + 32 * t + 8 * (lane >> 4);
        uint32_t plain = 0x88888888u;  // columns k0 .. k0 + 7, four bits each; 8 stands for 0
        if (row < nc && k0 < d) {
            const uint8_t *from = codes + row * bytes + k0 / 2;
            if (words && k0 + 8 <= d) {
                plain = *reinterpret_cast<const uint32_t *>(from);
            } else {
                plain = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    plain |= (k0 + e < d ? (uint32_t)(from[e / 2] >> (4 * (e & 1))) & 15 : 8u)
                             << (4 * e);
            }
        }
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w |= ((plain >> (4 * e)) & 15) << (4 * (e >> 1) + 16 * (e & 1));
        reinterpret_cast<uint32_t *>(to)[threadIdx.x] = w;
        if ((int)threadIdx.x < per * kBlockRows) {
            const int in = threadIdx.x;
            const int run = in / (4 * per), g = in / 4 % per, r = in % 4;
            const int64_t srow = rb * kBlockRows + 4 * run + r, gg = cb * per + g;
            reinterpret_cast<uint16_t *>(to + 1024)[in] =
                srow < nc && gg < groups ? scales[srow * groups + gg] : (uint16_t)0;
        }
    }
}

// ---- scores -------------------------------------------------------------------

// How queries of type X enter the matrix instruction.
template <typename X>
struct Form {  // f32 and bf16: bf16 columns
    using A = bf16x8;
    static constexpr int pieces = std::is_same<X, float>::value ? 3 : 1;
    // 16 + c: 0x4180 | c << 3; -24 is 0xc1c0
    static constexpr int place = 3;
    static constexpr uint32_t lead = 0x41804180u, mask = 0x00780078u, minus24 = 0xc1c0c1c0u;
    static __device__ __forceinline__ f32x4 mul(A a, A b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Form<_Float16> {
    using A = f16x8;
    static constexpr int pieces = 1;
    // 16 + c: 0x4c00 | c << 6; -24 is 0xce00
    static constexpr int place = 6;
    static constexpr uint32_t lead = 0x4c004c00u, mask = 0x03c003c0u, minus24 = 0xce00ce00u;
    static __device__ __forceinline__ f32x4 mul(A a, A b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

union Frag {
    uint32_t u[4];
    bf16x8 b;
    f16x8 h;
};
template <typename A>
__device__ __forceinline__ A frag_as(const Frag &f) {
    if constexpr (std::is_same<A, f16x8>::value) return f.h;
    else return f.b;
}

// The eight codes of a word as 16 + c.
template <typename F>
__device__ __forceinline__ Frag expand(uint32_t w) {
    Frag f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int up = F::place - 4 * j;
        f.u[j] = ((up >= 0 ? w << up : w >> -up) & F::mask) | F::lead;
    }
    return f;
}

// Piece p of an f32 value: x = piece 0 + piece 1 + piece 2, each the leading
// 8 bits of what is left.  A value that is not finite is its own piece 0.
__device__ __forceinline__ uint32_t bf16_piece(float x, int p) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7f800000u) == 0x7f800000u) {
        if (p > 0) return 0;
        return (u >> 16) | ((u & 0x007fffffu) ? 0x40u : 0u);  // a NaN stays one
    }
    float r = x;
    for (int i = 0; i < p; ++i) r -= __uint_as_float(__float_as_uint(r) & 0xffff0000u);
    return __float_as_uint(r) >> 16;
}

// Columns k .. k + 7 of a query (its row; d columns) as one lane's operand,
// zeros past the query: raw() loads them, frag() makes the operand.  wide:
// queries start on 16-byte boundaries and d % 8 == 0, so all eight are there
// or none.
template <typename X>
struct QueryPart {
    Vec<X, 8> v;
    int left;  // columns there, 8 at most (<= 0: none)
    __device__ __forceinline__ void raw(const X *__restrict__ row, int32_t d, int32_t k,
                                        bool wide) {
        left = d - k < 8 ? d - k : 8;
        const X *from = row + (left > 0 ? k : 0);  // without any, unused values
        if (wide) {
            using W = Vec<X, 16 / sizeof(X)>;
            W *to = reinterpret_cast<W *>(&v);
#pragma unroll
            for (int j = 0; j < (int)(8 / (16 / sizeof(X))); ++j)
                to[j] = reinterpret_cast<const W *>(from)[j];
        } else {
            const int last = left > 0 ? left - 1 : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] = from[e < last ? e : last];
        }
    }
    __device__ __forceinline__ Frag frag(int piece, bool wide) const {
        Frag f;
        if constexpr (std::is_same<X, float>::value) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f.u[j] = bf16_piece(v.v[2 * j], piece) | bf16_piece(v.v[2 * j + 1], piece) << 16;
        } else {
            __builtin_memcpy(&f, &v, 16);
        }
        if (wide) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f.u[j] = left > 0 ? f.u[j] : 0;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= left) f.u[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
        }
        return f;
    }
};

// One block's codes and scales as a lane holds them.
template <typename S, int PER>
struct Block {
    uint4 a;
    Vec<S, 4 * PER> s;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ table, int64_t blk,
                                         int lane) {
        const uint8_t *from = table + blk * block_bytes(PER);
        a = reinterpret_cast<const uint4 *>(from)[lane];
        s = reinterpret_cast<const Vec<S, 4 * PER> *>(from + 1024)[lane >> 4];
    }
};

// Where the staged operand of 8 query columns (chunk: their number / 8), tile
// ct and column c lies: [step = chunk / 4][ct][part = chunk % 4][c], with c
// turned by the chunk.  A wave's read of a step takes 1 KiB in a row; the
// staging writes of one column, a chunk per lane, spread over all banks.
template <int NT>
__device__ __forceinline__ int frag_place(int chunk, int ct, int c) {
    return (((chunk >> 2) * NT + ct) * 4 + (chunk & 3)) * 16 + (c ^ (chunk & 15));
}

// Many rows: a workgroup of 16 waves takes a run of row blocks, whose blocks
// lie one behind the other, and cuts that stream into 16 equal segments, so
// waves differ by less than a row block whatever the table's shape.  The
// queries are staged once, in operand order, in LDS; each wave then streams
// its segment with kBlocksAhead blocks in flight and no barrier.  A row block
// cut by a segment's border is finished by the wave that began it, from the
// parts (heads) the next waves leave in LDS, added in their order.  Bound by
// the stream: 65,536 x 4,096 (group 128) for 16 f16 queries 33 us, 4.4 TB/s;
// 262,144 x 256 (group 32) for one bf16 query 11.3 us (10.1 us a pass among
// others, 3.9 TB/s), of which about 4 us are the launch, the staging and the
// first blocks.  Tables of some thousand rows leave CUs idle, since a workgroup
// takes whole row blocks (8,359 x 767, five f32 queries: 7.2 us).  16 f32 queries
// fill 48 columns: 65,536 x 4,096 is read four times, 136 us.  8 waves and twice the
// workgroups took 48 us of 33 (the queries staged twice), 3 or 4 blocks ahead
// gained nothing.
constexpr int kStreamWaves = 16;
constexpr int kBlocksAhead = 2;

template <typename X, typename S, int GROUP, int NT>
__global__ __launch_bounds__(kStreamWaves * 64) void k_q4_scores_stream(
    const X *__restrict__ x, int64_t nq, int64_t nc, int32_t d, int64_t nrb, int32_t ncb,
    const uint8_t *__restrict__ table, float *__restrict__ y,
    int32_t rows_per, int wide, int quads) {
    using F = Form<X>;
    using A = typename F::A;
    constexpr int QT = 16 / F::pieces;
    constexpr int PER = kBlockCols / GROUP;
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    Frag *frags = reinterpret_cast<Frag *>(lds);  // 4 ncb NT 64, see frag_place
    f32x4 *heads = reinterpret_cast<f32x4 *>(frags + (size_t)ncb * 4 * NT * 64);  // [wave][NT][64]

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, part = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.x * rows_per;
    const int64_t r1 = r0 + rows_per < nrb ? r0 + rows_per : nrb;
    const int32_t total = (int32_t)(r1 - r0) * ncb;
    const int32_t seg = (total + kStreamWaves - 1) / kStreamWaves;
    const int32_t b0 = seg * w < total ? seg * w : total;
    const int32_t b1 = b0 + seg < total ? b0 + seg : total;
    const int64_t base = r0 * ncb;
    const int64_t q0 = (int64_t)blockIdx.y * NT * QT;

    // Staging, a query's 64 x 8 columns to a wave at a time: neighbouring lanes
    // read neighbouring columns (the same column of 16 queries could lie in
    // one L2 channel).  The first are asked for before the first blocks: loads
    // return in order, so behind a block they would wait for it.  Columns of
    // no query keep what LDS held: their sums go nowhere.
    constexpr int kParts = std::is_same<X, float>::value ? 4 : 8;
    const int chunks = ncb * (kBlockCols / 8), runs = (chunks + 63) >> 6;
    const int queries = (int)(nq - q0 < NT * QT ? nq - q0 : NT * QT);
    QueryPart<X> qp[kParts];
    // (query, run of 64 parts) of this wave's next part; all uniform
    const int step_q = kStreamWaves / runs, step_run = kStreamWaves - step_q * runs;
    int ask_q = w / runs, ask_run = w - ask_q * runs, stage_q = ask_q, stage_run = ask_run;
    auto go_on = [&](int &q, int &run) {
        q += step_q;
        run += step_run;
        if (run >= runs) {
            run -= runs;
            ++q;
        }
    };
    auto ask = [&]() {
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            if (ask_q >= queries) break;
            qp[h].raw(x + (q0 + ask_q) * d, d, 8 * (64 * ask_run + lane), wide != 0);
            go_on(ask_q, ask_run);
        }
    };
    auto stage = [&]() {
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            if (stage_q >= queries) break;
            const int chunk = 64 * stage_run + lane;
            if (chunk < chunks) {
                const int ct = stage_q / QT;
#pragma unroll
                for (int p = 0; p < F::pieces; ++p)
                    frags[frag_place<NT>(chunk, ct, stage_q - ct * QT + p * QT)] =
                        qp[h].frag(p, wide != 0);
            }
            go_on(stage_q, stage_run);
        }
    };
    ask();
    Block<S, PER> buf[kBlocksAhead];
    if (b0 < b1)
#pragma unroll
        for (int u = 0; u < kBlocksAhead; ++u)
            buf[u].load(table, base + (b0 + u < b1 ? b0 + u : b1 - 1), lane);
    stage();
    while (stage_q < queries) {
        ask();
        stage();
    }
    __syncthreads();

    Frag m24;
#pragma unroll
    for (int j = 0; j < 4; ++j) m24.u[j] = F::minus24;
    f32x4 acc[NT];
#pragma unroll
    for (int ct = 0; ct < NT; ++ct) acc[ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // scores of 16 rows: a query's pieces added smallest first
    auto store = [&](int64_t rb) {
#pragma unroll
        for (int ct = 0; ct < NT; ++ct) {
            f32x4 v = acc[ct];
            if constexpr (F::pieces == 3) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float mid = __shfl(acc[ct][r], lane + QT), lo = __shfl(acc[ct][r], lane + 2 * QT);
                    v[r] += mid + lo;
                }
            }
            const int64_t q = q0 + ct * QT + col, row = rb * kBlockRows + 4 * part;
            if (col < QT && q < nq) {
                float *to = y + q * nc + row;
                if (quads) {  // nc % 4 == 0: all four rows are there, or none
                    if (row < nc) __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(to));
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (row + r < nc) to[r] = v[r];
                }
            }
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int ct = 0; ct < NT; ++ct) acc[ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    auto leave_head = [&]() {
#pragma unroll
        for (int ct = 0; ct < NT; ++ct) heads[(w * NT + ct) * 64 + lane] = acc[ct];
    };

    int32_t rb = b0 / ncb, cb = b0 - rb * ncb;  // row block inside the run
    bool head = cb != 0;
    auto work = [&](const Block<S, PER> &now) __attribute__((always_inline)) {
        const uint32_t a[4] = {now.a.x, now.a.y, now.a.z, now.a.w};
#pragma unroll
        for (int g = 0; g < PER; ++g) {
            f32x4 c[NT];
#pragma unroll
            for (int ct = 0; ct < NT; ++ct) c[ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < GROUP / 32; ++s) {
                const int t = g * (GROUP / 32) + s;
                const Frag e = expand<F>(a[t]);
#pragma unroll
                for (int ct = 0; ct < NT; ++ct) {
                    const Frag q = frags[frag_place<NT>(16 * cb + 4 * t + part, ct, col)];
                    c[ct] = F::mul(frag_as<A>(m24), frag_as<A>(q), c[ct]);
                    c[ct] = F::mul(frag_as<A>(e), frag_as<A>(q), c[ct]);
                }
            }
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[ct][r] = __builtin_fmaf(widen(now.s.v[4 * g + r]), c[ct][r], acc[ct][r]);
        }
        if (++cb == ncb) {
            if (head) leave_head();
            else store(r0 + rb);
            head = false;
            clear();
            cb = 0;
            ++rb;
        }
    };
    // Every step asks for a block, past the end for the last one again: after a
    // load that may not be there, each wait would be a wait for all.
    for (int32_t b = b0; b < b1; b += kBlocksAhead) {
#pragma unroll
        for (int u = 0; u < kBlocksAhead; ++u) {
            if (b + u >= b1) break;
            const Block<S, PER> now = buf[u];
            const int32_t next = b + u + kBlocksAhead;
            buf[u].load(table, base + (next < b1 ? next : b1 - 1), lane);
            work(now);
        }
    }
    const bool open = b0 < b1 && cb != 0;  // the segment ends inside a row block
    if (open && head) leave_head();
    __syncthreads();
    if (open && !head) {
        const int32_t end = (rb + 1) * ncb;
        for (int v = w + 1; v < kStreamWaves && seg * v < end; ++v)
#pragma unroll
            for (int ct = 0; ct < NT; ++ct) acc[ct] += heads[(v * NT + ct) * 64 + lane];
        store(r0 + rb);
    }
}

// Wide queries whose operands do not fit in LDS: a workgroup per row block and
// tile of columns, its waves taking the row block's blocks in turn and the
// queries straight from memory.  Bound by those reads, four times the codes':
// 4,096 x 14,336 (group 128) for one bf16 query 15.3 us, 2.0 TB/s, for 16 18.2 us;
// 28,672 x 8,192 for one 48 us, 2.5 TB/s, for 16 70 us.
constexpr int kWideWaves = 16;

template <typename X, typename S, int GROUP>
__global__ __launch_bounds__(kWideWaves * 64) void k_q4_scores_wide(
    const X *__restrict__ x, int64_t nq, int64_t nc, int32_t d, int64_t nrb, int64_t ncb,
    const uint8_t *__restrict__ table, float *__restrict__ y,
    int wide) {
    using F = Form<X>;
    using A = typename F::A;
    constexpr int QT = 16 / F::pieces;     // queries per tile of columns
    constexpr int PER = kBlockCols / GROUP;  // groups per block
    __shared__ float red[kWideWaves][16][17];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int col = lane & 15, part = lane >> 4;
    const int64_t tiles = (nq + QT - 1) / QT;
    const int piece = col / QT;
    Frag m24;
#pragma unroll
    for (int j = 0; j < 4; ++j) m24.u[j] = F::minus24;

    for (int64_t ct = blockIdx.y; ct < tiles; ct += gridDim.y)
        for (int64_t rb = blockIdx.x; rb < nrb; rb += gridDim.x) {
            const int64_t q = col < QT * F::pieces ? ct * QT + col % QT : nq;
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int64_t cb = w; cb < ncb; cb += kWideWaves) {
                const int64_t blk = rb * ncb + cb;
                Block<S, PER> now;
                now.load(table, blk, lane);
                const uint32_t a[4] = {now.a.x, now.a.y, now.a.z, now.a.w};
#pragma unroll
                for (int g = 0; g < PER; ++g) {
                    f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < GROUP / 32; ++s) {
                        const int t = g * (GROUP / 32) + s;
                        QueryPart<X> qp;
                        qp.raw(x + (q < nq ? q : 0) * d, q < nq ? d : 0,
                               (int32_t)cb * kBlockCols + 32 * t + 8 * part, wide != 0);
                        const Frag b = qp.frag(piece, wide != 0);
                        c = F::mul(frag_as<A>(m24), frag_as<A>(b), c);
                        c = F::mul(frag_as<A>(expand<F>(a[t])), frag_as<A>(b), c);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[r] = __builtin_fmaf(widen(now.s.v[4 * g + r]), c[r], acc[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) red[w][col][4 * part + r] = acc[r];
            __syncthreads();
            for (int o = threadIdx.x; o < QT * 16; o += kWideWaves * 64) {
                const int r = o & 15, qq = o >> 4;
                float sum = 0.0f;
                for (int p = F::pieces - 1; p >= 0; --p)
                    for (int v = 0; v < kWideWaves; ++v) sum += red[v][qq + p * QT][r];
                const int64_t row = rb * kBlockRows + r, query = ct * QT + qq;
                if (row < nc && query < nq) y[query * nc + row] = sum;
            }
            __syncthreads();
        }
}

constexpr size_t kLds = 160 * 1024;

// LDS of the streaming kernel with nt tiles of columns
size_t stream_lds(int64_t ncb, int nt) {
    return ((size_t)ncb * 4 + kStreamWaves) * (size_t)nt * 1024;
}

template <typename X, typename S, int GROUP, int NT>
void launch_stream(const X *x, int64_t nq, int32_t d, const uint8_t *table, int64_t nc,
                   float *y, int wide, hipStream_t st, int n_cu) {
    const int64_t nrb = row_blocks(nc), ncb = col_blocks(d);
    constexpr int QT = 16 / Form<X>::pieces;
    // a run of row blocks per CU, of fewer than 2^30 blocks
    int64_t per = (nrb + n_cu - 1) / n_cu;
    const int64_t most = (int64_t(1) << 30) / ncb;
    if (per > most) per = most;
    const int64_t cols = (nq + (int64_t)NT * QT - 1) / ((int64_t)NT * QT);
    for (int64_t c = 0; c < cols; c += 65535) {  // the grid's limit in y
        const int quads = nc % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
        const int64_t cn = cols - c < 65535 ? cols - c : 65535, q = c * NT * QT;
        hipLaunchKernelGGL((k_q4_scores_stream<X, S, GROUP, NT>),
                           dim3((unsigned)((nrb + per - 1) / per), (unsigned)cn),
                           dim3(kStreamWaves * 64), stream_lds(ncb, NT), st, x + q * d, nq - q, nc,
                           d, nrb, (int32_t)ncb, table, y + q * nc, (int32_t)per, wide,
                           quads);
    }
}

template <typename X, typename S, int GROUP>
hipError_t scores_group(const X *x, int64_t nq, int32_t d, const uint8_t *table, int64_t nc, float *y,
                        hipStream_t st, int n_cu) {
    const int64_t nrb = row_blocks(nc), ncb = col_blocks(d);
    const int wide = d % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
    constexpr int QT = 16 / Form<X>::pieces;
    const int64_t tiles = (nq + QT - 1) / QT;
    timing_before(st, "k_q4_scores");
    // the table is read once per launch row of column tiles: as many tiles as
    // the queries need and LDS holds (1 / 2 / 4 tiles, us: 65,536 x 768 for 32
    // bf16 queries 16.7 / 12.3, for 64 29 / 22 / 17; 8,192 x 512 for 48 f16
    // queries 8.7 / 7.5 / 6.1; 65,536 x 2,048 for 32 bf16 queries 31 / 23)
    if (tiles > 2 && stream_lds(ncb, 4) <= kLds)
        launch_stream<X, S, GROUP, 4>(x, nq, d, table, nc, y, wide, st, n_cu);
    else if (tiles > 1 && stream_lds(ncb, 2) <= kLds)
        launch_stream<X, S, GROUP, 2>(x, nq, d, table, nc, y, wide, st, n_cu);
    else if (stream_lds(ncb, 1) <= kLds)
        launch_stream<X, S, GROUP, 1>(x, nq, d, table, nc, y, wide, st, n_cu);
    else {
        const dim3 grid((unsigned)(nrb < (1 << 20) ? nrb : 1 << 20),
                        (unsigned)(tiles < 64 ? tiles : 64));
        hipLaunchKernelGGL((k_q4_scores_wide<X, S, GROUP>), grid, dim3(kWideWaves * 64), 0, st, x,
                           nq, nc, d, nrb, ncb, table, y, wide);
    }
    timing_after(st);
    return hipGetLastError();
}

template <typename X, typename S>
hipError_t scores_type(const X *x, int64_t nq, int32_t d, const uint8_t *table, int64_t nc, int group,
                       float *y, hipStream_t st, int n_cu) {
    switch (group) {
    case 32: return scores_group<X, S, 32>(x, nq, d, table, nc, y, st, n_cu);
    case 64: return scores_group<X, S, 64>(x, nq, d, table, nc, y, st, n_cu);
    default: return scores_group<X, S, 128>(x, nq, d, table, nc, y, st, n_cu);
    }
}

template <typename X>
hipError_t scores_scale(const void *x, int64_t nq, int32_t d, const void *table, int64_t nc,
                        int group, int scale_dtype, float *y, hipStream_t st, int n_cu) {
    if (scale_dtype == kF16)
        return scores_type<X, _Float16>((const X *)x, nq, d, (const uint8_t *)table, nc, group, y,
                                            st, n_cu);
    return scores_type<X, __bf16>((const X *)x, nq, d, (const uint8_t *)table, nc, group, y,
                                            st, n_cu);
}

template <typename T>
hipError_t quantize_scale(const void *table, int64_t nc, int32_t d, int group, int scale_dtype,
                          uint8_t *codes, void *scales, unsigned grid, hipStream_t st) {
    if (scale_dtype == kF16)
        hipLaunchKernelGGL((k_q4_quantize<T, _Float16>), dim3(grid), dim3(256), 0, st,
                           (const T *)table, nc, d, group, codes, (_Float16 *)scales);
    else
        hipLaunchKernelGGL((k_q4_quantize<T, __bf16>), dim3(grid), dim3(256), 0, st,
                           (const T *)table, nc, d, group, codes, (__bf16 *)scales);
    return hipGetLastError();
}

}  // namespace

size_t q4_bytes(int64_t nc, int32_t d, int group) {
    return (size_t)row_blocks(nc) * (size_t)col_blocks(d) *
           (size_t)block_bytes(kBlockCols / group);
}

hipError_t launch_q4_quantize(const void *table, int64_t nc, int32_t d, int dtype, int group,
                              int scale_dtype, uint8_t *codes, void *scales, hipStream_t st,
                              int n_cu) {
    const int64_t want = (nc * ((d + group - 1) / group) * (group / 2) + 255) / 256;
    const int64_t most = (int64_t)n_cu * 64;
    const unsigned grid = (unsigned)(want < most ? want : most);
    switch (dtype) {
    case kF32: return quantize_scale<float>(table, nc, d, group, scale_dtype, codes, scales, grid, st);
    case kF16: return quantize_scale<_Float16>(table, nc, d, group, scale_dtype, codes, scales, grid, st);
    default: return quantize_scale<__bf16>(table, nc, d, group, scale_dtype, codes, scales, grid, st);
    }
}

hipError_t launch_q4_layout(const uint8_t *codes, const void *scales, int64_t nc, int32_t d,
                            int group, void *out, hipStream_t st, int n_cu) {
    const int64_t nrb = row_blocks(nc), ncb = col_blocks(d);
    const int64_t most = (int64_t)n_cu * 64, want = nrb * ncb;
    hipLaunchKernelGGL(k_q4_layout, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st,
                       codes, (const uint16_t *)scales, nc, d, group, nrb, ncb, (uint8_t *)out,
                       (int)(((d + 1) / 2) % 4 == 0 && (reinterpret_cast<uintptr_t>(codes) & 3) == 0));
    return hipGetLastError();
}

hipError_t launch_q4_scores(const void *x, int64_t nq, int32_t d, int dtype, const void *table,
                            int64_t nc, int group, int scale_dtype, float *y, hipStream_t st,
                            int n_cu) {
    switch (dtype) {
    case kF32: return scores_scale<float>(x, nq, d, table, nc, group, scale_dtype, y, st, n_cu);
    case kF16: return scores_scale<_Float16>(x, nq, d, table, nc, group, scale_dtype, y, st, n_cu);
    default: return scores_scale<__bf16>(x, nq, d, table, nc, group, scale_dtype, y, st, n_cu);
    }
}

}  // namespace vs
