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
//           at chunk ^ (r / 2 & 7), so that 16 lanes reading one chunk of 16 rows meet 16
//           different groups of banks (two rows fill the 64 banks)
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

#include <stdio.h>

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

// A piece of 16 or 4 bytes a lane from memory into LDS: lane l's lands at lds + l pieces.
// In assembly because the compiler, which cannot tell the two buffers apart, would wait
// for it before every LDS read; who uses it waits itself (wait_vmcnt) before the
// barrier behind which the piece is read.  m0, which names the place in LDS, is put
// back for the compiler; the s_nop is what the load has to stay behind a vector
// instruction's write of its scalar address (five states), which the compiler does
// not see here.
template <int PIECE>
__device__ __forceinline__ void fetch(const void *base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    if constexpr (PIECE == 16)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 4\n\t"
                     "global_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                     : "=&s"(m0)
                     : "v"(off), "s"(base), "s"(lds));
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 4\n\t"
                     "global_load_lds_dword %1, %2\n\ts_mov_b32 m0, %0"
                     : "=&s"(m0)
                     : "v"(off), "s"(base), "s"(lds));
}
template <int PIECE>
__device__ __forceinline__ void fetch_from(const void *p, uint32_t lds) {
    uint32_t m0;
    if constexpr (PIECE == 16)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 4\n\t"
                     "global_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                     : "=&s"(m0)
                     : "v"(p), "s"(lds));
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 4\n\t"
                     "global_load_lds_dword %1, off\n\ts_mov_b32 m0, %0"
                     : "=&s"(m0)
                     : "v"(p), "s"(lds));
}

// a value that is the same in all lanes, in scalar registers
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
template <typename P>
__device__ __forceinline__ P *uniform(P *p) {
    return reinterpret_cast<P *>(uniform((int64_t)(uintptr_t)p));
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// R rows of a side, moved by W waves.  PIECE of 16 or 4: loads of so many bytes straight
// into LDS; all addresses, ld and (along) the number of k's are multiples of them.
// PIECE of 0: through registers, 16 bytes a load at any address.  us in pieces of 4 and
// through registers: 16,384 rows to 16 units of 2,049 x 2,049 fp32 1,160 and 1,334;
// 20,000 to 60 of 1,026 x 1,026 bf16 121 and 133; 1,000 codes' rows of 1,004 over 20,000
// 41 and 45.  In pieces of 16: 1,024 x 1,024 67, 1,008 codes 38.
template <typename T, int R, int W, bool ACROSS, int PIECE>
struct Mover {
    static constexpr int ES = (int)sizeof(T);
    static constexpr int N = 16 / ES;               // elements a chunk
    static constexpr int K = kStep / ES;            // k's a step
    static constexpr int kChunks = R * ES / 16;     // chunks of a k's row (across)
    static constexpr int kBytes = PIECE ? PIECE : 16;  // a lane's of a load
    static constexpr int kLoads = R * kStep / (64 * kBytes * W);  // loads a wave
    static constexpr int kIn = 16 / kBytes;         // loads' parts of a chunk
    static_assert(R % (8 * W) == 0, "every wave moves the same number of pieces");
    typedef unsigned __int128 Bits;
    typedef typename std::conditional<
        ES == 1, uint8_t, typename std::conditional<ES == 2, uint16_t, uint32_t>::type>::type Whole;
    const T *base;
    int64_t ld;
    uint32_t off[kLoads];  // bytes from a step's first k to the lane's
    int part[kLoads];      // the lane's first k inside the step (along), its k (across)
    int left[kLoads];      // across, unaligned: elements from the chunk's first to the row's end
    u32x4 held[PIECE ? 1 : kLoads];
    int held_have;  // k's of the step in `held`
    bool tiny;
    bool whole;     // along: all of the step's chunks are there

    __device__ __forceinline__ void set(const Side<T> &s, int wave, int lane) {
        base = s.base;
        ld = s.ld;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int piece = (wave * kLoads + i) * 64 + lane;  // its place in LDS
            const int chunk = piece / kIn, e = piece % kIn * (kBytes / ES);  // element of it
            if constexpr (!ACROSS) {
                const int r = chunk / 8;
                const int c = (chunk & 7) ^ (r >> 1 & 7);
                const int row = r < s.rows ? r : s.rows - 1;
                off[i] = (uint32_t)row * (uint32_t)(s.ld * ES) + (c * N + e) * ES;
                part[i] = c * N + e;
            } else {
                const int k = chunk / kChunks, at = chunk % kChunks;
                const int c = (at ^ (ES == 2 ? (k & 3) << 1 : k & 4)) * N + e;
                const bool in = c < s.rows;
                off[i] = (uint32_t)k * (uint32_t)(s.ld * ES) + (in ? c * ES : 0);
                part[i] = k;
                left[i] = in ? s.rows - c : s.rows;
            }
        }
    }

    // where a step's first k lies
    __device__ __forceinline__ const char *from(int64_t k0) const {
        return reinterpret_cast<const char *>(base + (ACROSS ? k0 * ld : k0));
    }

    // PIECE: load i of the step at `step`; lds: where the side's buffer begins
    __device__ __forceinline__ void load(int i, const char *step, uint32_t lds, int wave) const {
        fetch<PIECE>(step, off[i], lds + (wave * kLoads + i) * 64 * kBytes);
    }
    // the same for a step of which only `have` k's are there
    __device__ __forceinline__ void load_part(int i, const char *step, uint32_t lds, int wave,
                                              int have) const {
        const char *p = step + off[i];
        if (part[i] >= have) p = reinterpret_cast<const char *>(&g_zeros);
        fetch_from<PIECE>(p, lds + (wave * kLoads + i) * 64 * kBytes);
    }

    // No PIECE: the step at k0, of which `have` k's are there, into registers ...
    // Of a chunk that ends behind its row, the row's last 16 bytes are loaded, and
    // shifted into place when they are written, so that all loads are whole and none
    // waits for another.  Rows of fewer than 16 bytes go by elements.
    __device__ __forceinline__ int there(int i) const {  // of a chunk's elements
        if constexpr (!ACROSS) return held_have - part[i];
        return part[i] < held_have ? left[i] : 0;
    }
    __device__ __forceinline__ void read(int64_t k0, int64_t have, int64_t row) {
        held_have = have < K ? (int)have : K;
        tiny = row < N;
        // Most steps are whole and need none of what follows: 20,000 rows to 60 units of
        // 1,027 x 1,027 bf16 139 us for 150.  (Across, the same gained nothing.)
        whole = !ACROSS && have >= K;
        if (whole) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) __builtin_memcpy(&held[i], from(k0) + off[i], 16);
            return;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const T *p = reinterpret_cast<const T *>(from(k0) + off[i]);
            const int n = there(i);
            if (tiny) {
                Bits bits = 0;
#pragma unroll 1
                for (int t = 0; t < n && t < N; ++t)
                    bits |= (Bits)reinterpret_cast<const Whole *>(p)[t] << (t * ES * 8);
                held[i] = __builtin_bit_cast(u32x4, bits);
                continue;
            }
            if constexpr (!ACROSS) {
                if (n <= 0) p = base;
                else if (n < N) p -= N - n;
            } else {
                if (n <= 0) p -= (int64_t)part[i] * ld;  // the same chunk of k0, which is there
                if (left[i] < N) p -= N - left[i];
            }
            __builtin_memcpy(&held[i], p, 16);
        }
    }
    // ... and from there into LDS.
    __device__ __forceinline__ void write(char *lds, int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            u32x4 v = held[i];
            const int n = there(i);
            if (!whole && !tiny && n < N) {
                Bits bits = __builtin_bit_cast(Bits, v);
                bits = n <= 0 ? 0 : bits >> ((N - n) * ES * 8);
                v = __builtin_bit_cast(u32x4, bits);
            }
            *reinterpret_cast<u32x4 *>(lds + (wave * kLoads + i) * 1024 + lane * 16) = v;
        }
    }
};

// Block b (16 rows) of half h (64 bytes of k) of a side in LDS, as the matrix
// instruction takes it.
template <typename T, int R, bool ACROSS>
__device__ __forceinline__ u32x4 fragment(const char *lds, int b, int h, int lane) {
    const int i = lane & 15, j = lane >> 4;
    if constexpr (!ACROSS) {
        return *reinterpret_cast<const u32x4 *>(lds + (b * 16 + i) * kStep +
                                                (((h * 4 + j) ^ (i >> 1)) << 4));
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

template <typename T, int BM, int BN, int WM, int WN, bool M_ACROSS, bool N_ACROSS, int PIECE>
struct Core {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MB = BM / WM / 16, NB = BN / WN / 16;  // blocks of a wave
    static constexpr int kSide = BM * kStep;                    // where the N side begins
    static constexpr int kBytes = (BM + BN) * kStep;            // of a buffer
    static constexpr int K = kStep / (int)sizeof(T);
    static constexpr int kRows = BM;
    typedef typename Sum<T>::type Acc;
    typedef Mover<T, BM, kWaves, M_ACROSS, PIECE> MMover;
    typedef Mover<T, BN, kWaves, N_ACROSS, PIECE> NMover;
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
                                         const char *mstep, const char *nstep, uint32_t to) {
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

    MMover mm;
    NMover nm;
    int64_t depth;

    __device__ __forceinline__ Core() {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wm = wave / WN;
        wn = wave % WN;
    }

    // Begins a product over k = 0 .. k_count - 1: its first step is on its way into the
    // first of the two buffers at `bufs`, whose earlier contents no wave needs any
    // more.  The first step is the one that may be short, so that all others are whole.
    __device__ __forceinline__ void begin(const Side<T> &ms, const Side<T> &ns, int64_t k_count,
                                          char *bufs) {
        depth = uniform(k_count);
        if (depth <= 0) return;
        const int l = fresh(lane);
        mm.set(ms, wave, l);
        nm.set(ns, wave, l);
        if constexpr (PIECE > 0) {
            const int first = (int)((depth - 1) % K) + 1;
            count_to<MMover::kLoads>(
                [&](auto i) { mm.load_part(i, mm.from(0), lds_at(bufs), wave, first); });
            count_to<NMover::kLoads>(
                [&](auto i) { nm.load_part(i, nm.from(0), lds_at(bufs) + kSide, wave, first); });
        } else {
            read(0);
        }
    }
    __device__ __forceinline__ void read(int64_t k0) {
        mm.read(k0, depth - k0, M_ACROSS ? mm.ld : depth);
        nm.read(k0, depth - k0, N_ACROSS ? nm.ld : depth);
    }
    // the lane as a value of its own: what follows from it is computed again for every
    // tile instead of being held in registers that the sums need
    static __device__ __forceinline__ int fresh(int l) {
        asm volatile("" : "+v"(l));
        return l;
    }
    static __device__ __forceinline__ uint32_t lds_at(char *p) {
        return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)p;
    }

    // The sums, in acc.  All waves are through with both buffers behind a barrier.
    __device__ __forceinline__ void sum(char *bufs) {
        count_to<MB * NB>([&](auto q) { acc[q / NB][q % NB] = Acc{0, 0, 0, 0}; });
        if (depth <= 0) return;
        const int64_t steps = (depth + K - 1) / K;
        if constexpr (PIECE > 0) {
            const int first = (int)((depth - 1) % K) + 1;
            const uint32_t lds = lds_at(bufs);
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
                half<true, false>(f, g, cur, 1, mstep, nstep, 0);
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                lds_barrier();
                half<true, decltype(load)::value>(g, f, nxt, 0, mstep, nstep, lds + now);
                mstep += madd;
                nstep += nadd;
                now = kBytes - now;
            };
            for (; t < steps - 2; ++t) turn(std::true_type());
            for (; t < steps; ++t) turn(std::false_type());
        } else {
            for (int64_t t = 0; t < steps; ++t) {
                char *buf = bufs + (t & 1) * kBytes;
                // step t - 2's reads of this buffer ended before the last barrier
                mm.write(buf, wave, lane);
                nm.write(buf + kSide, wave, lane);
                __syncthreads();
                if (t + 1 < steps) read((t + 1) * K);
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

    // Results into rows of `out` (`ld` elements apart), rows 0 .. rows - 1 and
    // columns 0 .. cols - 1 of the tile.  convert(a, b, sums of block row a and block
    // column b) gives their floats.  A wave's blocks go through its part of the buffers,
    // which no wave reads any more: stored from the matrix instruction's layout, 32 bytes
    // of a row at a time, 8,192 x 8,192 bf16 results of 128 products each took 71 us,
    // whole lines at a time 51.
    template <typename O, typename F>
    __device__ __forceinline__ void put(char *bufs, O *out, int64_t ld, int rows, int cols,
                                        F convert) const {
        constexpr int kRow = NB * 16 * (int)sizeof(O);  // bytes of a row of the wave's part
        constexpr int kChunks = kRow / 16;
        constexpr int kPer = 16 / (int)sizeof(O);       // elements a chunk
        constexpr int kTurns = (BM * BN * (int)sizeof(O) + 2 * kBytes - 1) / (2 * kBytes);
        constexpr int kBlocks = MB / kTurns;            // blocks of rows a turn
        static_assert(MB % kTurns == 0 && (kChunks & (kChunks - 1)) == 0, "whole turns");
        char *mine = bufs + wave * (kBlocks * 16 * kRow);
        const int l = fresh(lane), i = l & 15, j = l >> 4;
        count_to<kTurns>([&](auto turn) {
            count_to<kBlocks * NB>([&](auto q) {
                constexpr int a = turn * kBlocks + q / NB, b = q % NB;
                Vec<O, 4> v;
                const f32x4 f = convert(a, b, acc[a][b]);
#pragma unroll
                for (int t = 0; t < 4; ++t) v.v[t] = narrow<O>(f[t]);
                const int byte = (b * 16 + j * 4) * (int)sizeof(O);
                const int chunk = (byte >> 4) ^ (i & (kChunks - 1));
                *reinterpret_cast<Vec<O, 4> *>(mine + (q / NB * 16 + i) * kRow + chunk * 16 +
                                               (byte & 15)) = v;
            });
#pragma unroll 4
            for (int e = l; e < kBlocks * 16 * kChunks; e += 64) {
                const int r = e / kChunks, c = e % kChunks;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(
                    mine + r * kRow + ((c ^ (r & 15 & (kChunks - 1))) << 4));
                const int m = (wm * MB + turn * kBlocks) * 16 + r;
                const int n = wn * NB * 16 + c * kPer;
                if (m >= rows || n >= cols) continue;
                O *to = out + m * ld + n;
                if (n + kPer <= cols) {
                    __builtin_memcpy(to, &v, 16);
                } else {
                    O o[kPer];
                    __builtin_memcpy(o, &v, 16);
#pragma unroll
                    for (int t = 0; t < kPer; ++t)
                        if (n + t < cols) to[t] = o[t];
                }
            }
        });
    }

    // int8: sums times their row's and their column's scale.  What a lane needs of the
    // scales is loaded at once, from rows that are there.
    template <typename O>
    __device__ __forceinline__ void put_scaled(char *bufs, O *out, int64_t ld, int rows, int cols,
                                               const float *mscale, const float *nscale) const {
        const int l = fresh(lane);
        float ms[MB];
        f32x4 ns[NB];
        count_to<MB>([&](auto a) {
            ms[a] = mscale[least_of((wm * MB + a) * 16 + (l & 15), rows - 1)];
        });
        count_to<NB>([&](auto b) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                ns[b][t] = nscale[least_of((wn * NB + b) * 16 + (l >> 4) * 4 + t, cols - 1)];
        });
        put(bufs, out, ld, rows, cols, [&](int a, int b, const Acc &v) {
            f32x4 f;
#pragma unroll
            for (int t = 0; t < 4; ++t) f[t] = (float)v[t] * ms[a] * ns[b][t];
            return f;
        });
    }
    static __device__ __forceinline__ int least_of(int a, int b) { return a < b ? a : b; }
};

// Tiles are numbered so that those of one XCD (workgroups are dealt out to the 8 in
// turn) follow each other, and run through `cols` column tiles in groups of 8, all
// row tiles for each group: the 32 tiles an XCD works on at a time share their sides.
struct Place {
    int64_t row, col;
};
// The tile of workgroup `id`; false where it has none.  Each of the 8 has a stretch
// of the tiles, and an id behind its XCD's stretch must not run into the next one.
__host__ __device__ inline bool xcd_tile(int64_t id, int64_t total, int64_t &at) {
    const int64_t stretch = (total + 7) >> 3, turn = id >> 3;
    at = (id & 7) * stretch + turn;
    return turn < stretch && at < total;
}
__host__ __device__ inline Place place(int64_t tile, int64_t rows, int64_t cols) {
    const int64_t group = tile / (rows * 8), in = tile - group * rows * 8;
    const int64_t left = cols - group * 8, width = left < 8 ? left : 8;
    return Place{in / width, group * 8 + in % width};
}
// One tile's work: out[m][n] of its sides' rows.
template <typename T, typename O>
struct Job {
    Side<T> m, n;
    int64_t depth;
    O *out;
    int64_t ld;
    const float *mscale, *nscale;  // int8: the rows' scales of either side
};

// A workgroup's tiles.  job(id, j) says what tile `id` of `total` is (numbered as
// workgroups are, see xcd_tile), or that there is nothing to do.  As a rule a workgroup
// has one tile: workgroups that stayed, took the next tile's first loads up before
// they stored this one's results, and so saved its start, were no faster (65,536 x
// 2,048 rows into 128 units of 2,048 columns, bf16, 557 us so, 589 us then), since
// all of them store at the same time and the loads behind wait for the stores.
// A tile of few rows is taken by the first of the lower cores `Low` that holds them.
template <typename T, typename O, typename C, typename... Low, typename FJ>
__device__ __forceinline__ void run_tiles(int64_t total, char *bufs, FJ job) {
    for (int64_t id = blockIdx.x; id < (total + 7) / 8 * 8; id += gridDim.x) {
        Job<T, O> j;
        if (!job(id, j)) continue;
        lds_barrier();  // the last tile's results have left the buffers
        auto work = [&](auto core) {
            core.begin(j.m, j.n, j.depth, bufs);
            core.sum(bufs);
            lds_barrier();  // no wave reads the buffers any more
            if constexpr (std::is_same<T, int8_t>::value) {
                core.put_scaled(bufs, j.out, j.ld, j.m.rows, j.n.rows, j.mscale, j.nscale);
            } else {
                core.put(bufs, j.out, j.ld, j.m.rows, j.n.rows,
                         [](int, int, const f32x4 &v) { return v; });
            }
            return true;
        };
        const int rows = uniform(j.m.rows);
        if ((... || (rows <= Low::kRows && work(Low())))) continue;
        work(C());
    }
}

// What the timing hook calls a kernel: its tile, the bytes that rows move in, and more
struct FormName {
    char text[48];
    FormName(const char *kernel, int bm, int bn, int piece, const char *more = "") {
        snprintf(text, sizeof(text), "%s<%dx%d,%d%s>", kernel, bm, bn, piece, more);
    }
};

// Workgroups for `total` tiles, a multiple of 8.  The most keeps the number of threads
// below 2^32, which a launch counts in 32 bits.
constexpr int64_t kMostGroups = 1 << 20;
inline unsigned grid_of(int64_t total) {
    const int64_t want = (total + 7) / 8 * 8, most = kMostGroups;
    return (unsigned)(want < most ? want : most);
}

}  // namespace tile
}  // namespace vs
