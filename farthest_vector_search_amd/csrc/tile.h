// tile.h -- products of tiles on the matrix cores, for units.hip and q8.hip:
//
//   acc[m][n] = sum_k M(m, k) N(n, k)
//
// for a tile of BM x BN by a workgroup of WM x WN waves.  A side's matrix lies
// along k in memory (rows of k: "along") or across it (a row for each k, the side's
// own index inside: "across").  Element types: fp32, fp16, bf16 (sums in fp32) and
// int8 (along only, sums in int32).
//
// A step is 128 bytes of k (32, 64 or 128 elements), in two halves of 64.  Both
// sides' pieces of a step are brought into LDS (two buffers, one barrier a step)
// while others are multiplied.  LDS holds a side as
//   along   128 bytes for each of its rows; the eight 16-byte chunks of row r stand
//           at chunk ^ (r & 7), so that 8 lanes reading one chunk of 8 rows meet 8
//           different bank groups
//   across  a row for each k; chunks of row k stand at chunk ^ 2 (k & 3) for 16-bit
//           elements, chunk ^ (k & 4) for fp32, for the same reason
// The matrix instruction takes 16 bytes of k a lane.  From an "along" side that is
// one 16-byte read; from an "across" side of 16-bit elements two transposing reads
// (4 rows of 16 elements each, delivered by column), of fp32 four single reads.  The
// four fp32 instructions of a 16-byte piece take element i of every lane, so their k
// run i, 4 + i, 8 + i, 12 + i: the same on both sides, and the sum's order is free.
//
// N is the instruction's first operand, so that a lane's four results are
// neighbours in n: lane l holds (m = l % 16, n = 4 (l / 16) + 0 .. 3) of a block.
//
// What lies behind the end of k inside a step is brought in as zeros on both sides
// (a NaN of a neighbour must not meet a zero); rows behind a side's end are brought
// in as copies of rows that are there, and their results not stored.
#pragma once

#include <type_traits>
#include <utility>

#include "vs_internal.h"
#include "vs_types.h"

namespace vs {
namespace tile {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr int kStep = 128;  // bytes of k a step

// f(0), f(1), .. f(N - 1) with constants: the compiler gives up unrolling loops as
// large as these, and arrays indexed by a variable would leave the registers
template <typename F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F &&f) {
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void count_to(F &&f) {
    each_of(std::make_integer_sequence<int, N>(), f);
}

// 16 bytes of zeros that loads behind the end of k are pointed at
__device__ const u32x4 g_zeros = {0, 0, 0, 0};

template <typename T>
struct Sum {
    typedef f32x4 type;
};
template <>
struct Sum<int8_t> {
    typedef i32x4 type;
};

__device__ __forceinline__ f32x4 mac(f32x4 c, u32x4 n, u32x4 m, float) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(n[i]), __uint_as_float(m[i]), c, 0,
                                                 0, 0);
    return c;
}
__device__ __forceinline__ f32x4 mac(f32x4 c, u32x4 n, u32x4 m, _Float16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, n),
                                                  __builtin_bit_cast(f16x8, m), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mac(f32x4 c, u32x4 n, u32x4 m, __bf16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, n),
                                                   __builtin_bit_cast(bf16x8, m), c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mac(i32x4 c, u32x4 n, u32x4 m, int8_t) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, n),
                                                 __builtin_bit_cast(i32x4, m), c, 0, 0, 0);
}

// One side of a product: `base` is element (first row, k = 0), `rows` of its rows
// are there (1 at least), `ld` elements lie between rows (along) or between k's
// (across).
template <typename T>
struct Side {
    const T *base;
    int64_t ld;
    int rows;
};

// One 16-byte piece a lane from memory into LDS: lane l's lands at lds + 16 l.  In
// assembly because the compiler, which cannot tell the two buffers apart, would wait
// for it before every LDS read; who uses it waits itself (wait_vmcnt) before the
// barrier behind which the piece is read.
// m0, which names the place in LDS, is put back for the compiler.
__device__ __forceinline__ void fetch(const void *base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "v"(off), "s"(base), "s"(lds));
}
__device__ __forceinline__ void fetch_from(const void *p, uint32_t lds) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "v"(p), "s"(lds));
}

// a value that is the same in all lanes, in scalar registers
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
__device__ __forceinline__ const char *uniform(const char *p) {
    return reinterpret_cast<const char *>(uniform((int64_t)(uintptr_t)p));
}

// R rows of a side, moved by W waves.  ALIGNED: 16-byte loads straight into LDS; all
// addresses, ld and (along) the number of k's are multiples of 16 bytes.  Else
// through registers, 16 bytes a load at any address, and by elements where 16 bytes
// would leave a row.
template <typename T, int R, int W, bool ACROSS, bool ALIGNED>
struct Mover {
    static constexpr int ES = (int)sizeof(T);
    static constexpr int N = 16 / ES;               // elements a chunk
    static constexpr int K = kStep / ES;            // k's a step
    static constexpr int kChunks = R * ES / 16;     // chunks of a k's row (across)
    static constexpr int kLoads = R / 8 / W;        // loads a wave
    static_assert(R % (8 * W) == 0, "every wave moves the same number of pieces");
    const T *base;
    int64_t ld;
    uint32_t off[kLoads];  // bytes from a step's first k to the lane's chunk
    int part[kLoads];      // the chunk's first k inside the step (along), its k (across)
    int left[kLoads];      // across, unaligned: elements from the chunk's first to the row's end
    u32x4 held[ALIGNED ? 1 : kLoads];

    __device__ __forceinline__ void set(const Side<T> &s, int wave, int lane) {
        base = s.base;
        ld = s.ld;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int piece = wave * kLoads + i;  // 64 chunks, 1 KiB of LDS
            if constexpr (!ACROSS) {
                const int r = piece * 8 + lane / 8;
                const int c = (lane & 7) ^ (lane / 8);
                const int row = r < s.rows ? r : s.rows - 1;
                off[i] = (uint32_t)row * (uint32_t)(s.ld * ES) + c * 16;
                part[i] = c * N;
            } else {
                const int k = (piece * 64 + lane) / kChunks, at = (piece * 64 + lane) % kChunks;
                const int c = at ^ (ES == 2 ? (k & 3) << 1 : k & 4);
                const bool in = c * N < s.rows;
                off[i] = (uint32_t)k * (uint32_t)(s.ld * ES) + (in ? c * 16 : 0);
                part[i] = k;
                left[i] = in ? s.rows - c * N : s.rows;
            }
        }
    }

    // where a step's first k lies
    __device__ __forceinline__ const char *from(int64_t k0) const {
        return reinterpret_cast<const char *>(base + (ACROSS ? k0 * ld : k0));
    }

    // ALIGNED: load i of the step at `step`; lds: where the side's buffer begins
    __device__ __forceinline__ void load(int i, const char *step, uint32_t lds, int wave) const {
        fetch(step, off[i], lds + (wave * kLoads + i) * 1024);
    }
    // the same for a step of which only `have` k's are there
    __device__ __forceinline__ void load_part(int i, const char *step, uint32_t lds, int wave,
                                              int have) const {
        const char *p = step + off[i];
        if (part[i] >= have) p = reinterpret_cast<const char *>(&g_zeros);
        fetch_from(p, lds + (wave * kLoads + i) * 1024);
    }

    // Not ALIGNED: the step at k0, of which `have` k's are there, into registers ...
    __device__ __forceinline__ void read(int64_t k0, int64_t have) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const T *p = reinterpret_cast<const T *>(from(k0) + off[i]);
            int n = N;  // elements that may be read
            if constexpr (!ACROSS) {
                if (have - part[i] < N) n = (int)(have - part[i]);
            } else {
                if (left[i] < N) n = left[i];
                if (part[i] >= have) n = 0;
            }
            if (n >= N) {
                __builtin_memcpy(&held[i], p, 16);
            } else {
                T e[N];
#pragma unroll
                for (int t = 0; t < N; ++t) e[t] = t < n ? p[t] : T(0);
                __builtin_memcpy(&held[i], e, 16);
            }
        }
    }
    // ... and from there into LDS.
    __device__ __forceinline__ void write(char *lds, int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<u32x4 *>(lds + (wave * kLoads + i) * 1024 + lane * 16) = held[i];
    }
};

// Block b (16 rows) of half h (64 bytes of k) of a side in LDS, as the matrix
// instruction takes it.
template <typename T, int R, bool ACROSS>
__device__ __forceinline__ u32x4 fragment(const char *lds, int b, int h, int lane) {
    const int i = lane & 15, j = lane >> 4;
    if constexpr (!ACROSS) {
        return *reinterpret_cast<const u32x4 *>(lds + (b * 16 + i) * kStep +
                                                (((h * 4 + j) ^ (lane & 7)) << 4));
    } else if constexpr (sizeof(T) == 2) {
        typedef __attribute__((address_space(3))) s16x4 *P;
        const char *p = lds + (h * 32 + 8 * j + i / 4) * (R * 2) +
                        (((b * 2 + (i & 3) / 2) ^ ((i / 4) << 1)) << 4) + (i & 1) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * R * 2));
        typedef __attribute__((ext_vector_type(8))) short s16x8;
        return __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        u32x4 v;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int k = h * 16 + 4 * j + t;
            v[t] = *reinterpret_cast<const uint32_t *>(lds + k * (R * 4) + (((b * 4 + i / 4) ^ (k & 4)) << 4) +
                                                       (i & 3) * 4);
        }
        return v;
    }
}

template <typename T, int BM, int BN, int WM, int WN, bool M_ACROSS, bool N_ACROSS, bool ALIGNED>
struct Core {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MB = BM / WM / 16, NB = BN / WN / 16;  // blocks of a wave
    static constexpr int kSide = BM * kStep;                    // where the N side begins
    static constexpr int kBytes = (BM + BN) * kStep;            // of a buffer
    static constexpr int K = kStep / (int)sizeof(T);
    typedef typename Sum<T>::type Acc;
    typedef Mover<T, BM, kWaves, M_ACROSS, ALIGNED> MMover;
    typedef Mover<T, BN, kWaves, N_ACROSS, ALIGNED> NMover;
    struct Frags {
        u32x4 m[MB], n[NB];
    };
    Acc acc[MB][NB];
    int lane, wave, wm, wn;

    // fragment r of a half, in the order in which the products take them
    __device__ __forceinline__ void take(Frags &f, int r, const char *lds, int h) const {
        // n 0, m 0, n 1 .., m 1 ..
        if (r == 1) f.m[0] = fragment<T, BM, M_ACROSS>(lds, wm * MB, h, lane);
        else if (r <= NB) {
            const int b = r ? r - 1 : 0;
            f.n[b] = fragment<T, BN, N_ACROSS>(lds + kSide, wn * NB + b, h, lane);
        } else {
            f.m[r - NB] = fragment<T, BM, M_ACROSS>(lds, wm * MB + r - NB, h, lane);
        }
    }

    // One half's products, from `f`; in between, where asked, the fragments of half
    // `h` at `next` into `g` (in the first three quarters, since a barrier or the
    // next half waits for them), and the loads of the step at mstep / nstep into the
    // buffer at `to`.  The order is fixed as written: one wave has a SIMD to itself
    // (or two have it), and what it waits for has to be asked for in time.
    template <bool READ, bool LOAD>
    __device__ __forceinline__ void half(const Frags &f, Frags &g, const char *next, int h,
                                         const MMover &mm, const NMover &nm, const char *mstep,
                                         const char *nstep, uint32_t to) {
        constexpr int kAll = MB * NB, kFrags = MB + NB;
        constexpr int kLoads = MMover::kLoads + NMover::kLoads;
        count_to<kAll>([&](auto qc) {
            constexpr int q = decltype(qc)::value;
            if constexpr (READ) {
                constexpr int lo = least(kFrags, (q * kFrags * 4 + kAll * 3 - 1) / (kAll * 3));
                constexpr int hi = least(kFrags, ((q + 1) * kFrags * 4 + kAll * 3 - 1) / (kAll * 3));
                count_to<hi - lo>([&](auto r) { take(g, lo + decltype(r)::value, next, h); });
            }
            if constexpr (LOAD) {
                constexpr int lo = (q * kLoads + kAll - 1) / kAll;
                constexpr int hi = ((q + 1) * kLoads + kAll - 1) / kAll;
                count_to<hi - lo>([&](auto ic) {
                    constexpr int i = lo + decltype(ic)::value;
                    if constexpr (i < MMover::kLoads) mm.load(i, mstep, to, wave);
                    else nm.load(i - MMover::kLoads, nstep, to + kSide, wave);
                });
            }
            acc[q / NB][q % NB] = mac(acc[q / NB][q % NB], f.n[q % NB], f.m[q / NB], T());
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    static constexpr int least(int a, int b) { return a < b ? a : b; }

    // The sums over k = 0 .. depth - 1; all threads of the workgroup take part.
    // bufs: two buffers of kBytes.  A caller that writes into them, or calls again,
    // has a barrier in between (run begins with one).
    __device__ __forceinline__ void run(const Side<T> &ms, const Side<T> &ns, int64_t depth,
                                        char *bufs) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wm = wave / WN;
        wn = wave % WN;
        count_to<MB * NB>([&](auto q) { acc[q / NB][q % NB] = Acc{0, 0, 0, 0}; });
        if (depth <= 0) return;
        MMover mm;
        NMover nm;
        mm.set(ms, wave, lane);
        nm.set(ns, wave, lane);
        depth = uniform(depth);
        const int64_t steps = (depth + K - 1) / K;
        if constexpr (ALIGNED) {
            // The first step is the one that may be short, so that all others are whole.
            const int first = (int)(depth - (steps - 1) * K);
            const uint32_t lds = (uint32_t)(uintptr_t)(
                __attribute__((address_space(3))) char *)bufs;
            lds_barrier();
            count_to<MMover::kLoads>(
                [&](auto i) { mm.load_part(i, mm.from(0), lds, wave, first); });
            count_to<NMover::kLoads>(
                [&](auto i) { nm.load_part(i, nm.from(0), lds + kSide, wave, first); });
            const char *mstep = uniform(mm.from(first)), *nstep = uniform(nm.from(first));  // step 1's
            const int64_t madd = uniform(mm.from(K) - mm.from(0));
            const int64_t nadd = uniform(nm.from(K) - nm.from(0));
            wait_vmcnt_n<0>();
            lds_barrier();
            if (steps > 1) {
                count_to<MMover::kLoads>([&](auto i) { mm.load(i, mstep, lds + kBytes, wave); });
                count_to<NMover::kLoads>(
                    [&](auto i) { nm.load(i, nstep, lds + kBytes + kSide, wave); });
                mstep += madd;
                nstep += nadd;
            }
            Frags f, g;
            count_to<MB + NB>([&](auto r) { take(f, r, bufs, 0); });
            // Step t is in the buffer at `now`, its first half in f.  Behind the barrier
            // this wave's reads of step t are done, everyone's are, and step t + 1 is
            // there; the last two steps load nothing, the last reads what nobody uses.
            int now = 0;
            int64_t t = 0;
            auto turn = [&](auto load) {
                const char *cur = bufs + now, *nxt = bufs + (kBytes - now);
                half<true, false>(f, g, cur, 1, mm, nm, mstep, nstep, 0);
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                lds_barrier();
                half<true, decltype(load)::value>(g, f, nxt, 0, mm, nm, mstep, nstep, lds + now);
                mstep += madd;
                nstep += nadd;
                now = kBytes - now;
            };
            for (; t < steps - 2; ++t) turn(std::true_type());
            for (; t < steps; ++t) turn(std::false_type());
        } else {
            __syncthreads();
            mm.read(0, depth);
            nm.read(0, depth);
            for (int64_t t = 0; t < steps; ++t) {
                char *buf = bufs + (t & 1) * kBytes;
                // step t - 2's reads of this buffer ended before the last barrier
                mm.write(buf, wave, lane);
                nm.write(buf + kSide, wave, lane);
                __syncthreads();
                if (t + 1 < steps) {
                    mm.read((t + 1) * K, depth - (t + 1) * K);
                    nm.read((t + 1) * K, depth - (t + 1) * K);
                }
                count_to<2>([&](auto h) {
                    Frags f;
                    count_to<MB + NB>([&](auto r) { take(f, r, buf, h); });
                    count_to<MB * NB>([&](auto q) {
                        acc[q / NB][q % NB] = mac(acc[q / NB][q % NB], f.n[q % NB], f.m[q / NB], T());
                    });
                });
            }
        }
    }

    // f(m, n, four neighbours along n) for every block of the wave
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        count_to<MB * NB>([&](auto q) {
            f((wm * MB + q / NB) * 16 + (lane & 15), (wn * NB + q % NB) * 16 + (lane >> 4) * 4,
              acc[q / NB][q % NB]);
        });
    }
};

// Tiles are numbered so that those of one XCD (workgroups are dealt out to the 8 in
// turn) follow each other, and run through `cols` column tiles in groups of 8, all
// row tiles for each group: the 32 tiles an XCD works on at a time share their sides.
struct Place {
    int64_t row, col;
};
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
    return (id & 7) * ((total + 7) >> 3) + (id >> 3);
}
__device__ __forceinline__ Place place(int64_t tile, int64_t rows, int64_t cols) {
    const int64_t group = tile / (rows * 8), in = tile - group * rows * 8;
    const int64_t left = cols - group * 8, width = left < 8 ? left : 8;
    return Place{in / width, group * 8 + in % width};
}
inline unsigned grid_of(int64_t total) {
    const int64_t want = (total + 7) / 8 * 8, most = 1 << 24;
    return (unsigned)(want < most ? want : most);
}

}  // namespace tile
}  // namespace vs
