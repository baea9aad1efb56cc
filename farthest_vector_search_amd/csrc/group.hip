// group.hip -- entries grouped by unit: a stable sort of indices.
//
// ids[i] in [0, G) names entry i's unit; anything else means the entry is
// dropped.  Three results, all whole numbers and the same on every call:
//   order[p]    the entry at place p when entries are sorted by unit, equal
//               units in their own order; -1 behind the last kept entry
//   offsets[g]  the first place of unit g (G + 1 values; the last is the
//               number of kept entries)
//   slot[i]     the place of entry i, -1 if dropped (the inverse of order)
// A dropped entry is given the key G, so it sorts behind every kept one.
#include "vs_internal.h"

namespace vs {

namespace {

// ---- few entries: every place by counting ---------------------------------
//
// place(i) = #{j : (key_j, j) < (key_i, i)} and offsets[g] = #{j : key_j < g},
// one launch with nothing passed between workgroups.  A workgroup serves 64
// entries (or 64 units) with 16 waves, each wave counting over a 16th of the
// keys; the keys arrive through scalar loads, 16 at a time, so a pair costs
// one compare and one add with carry.
constexpr int kRankWaves = 16;

__device__ __forceinline__ uint32_t key_of(int32_t id, uint32_t G) {
    const uint32_t u = (uint32_t)id;
    return u < G ? u : G;
}

__global__ __launch_bounds__(kRankWaves * 64) void k_group_rank(
    const int32_t *__restrict__ ids, int32_t n, uint32_t G, int32_t entry_blocks,
    int32_t *__restrict__ order, int32_t *__restrict__ offsets, int32_t *__restrict__ slot) {
    __shared__ uint32_t part[kRankWaves][64];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool entries = (int32_t)blockIdx.x < entry_blocks;
    // i0: first entry of the block; past every j for the blocks of units,
    // whose counts take key_j < g for all j
    const int32_t i0 = entries ? (int32_t)blockIdx.x * 64 : 0;
    const int32_t i = i0 + lane;
    const int64_t g = entries ? 0 : ((int64_t)blockIdx.x - entry_blocks) * 64 + lane;
    const uint32_t key = entries ? (i < n ? key_of(ids[i], G) : G)
                                 : (uint32_t)(g < (int64_t)G ? g : (int64_t)G);

    // this wave's keys: a multiple of 16 per wave, so a group of 16 lies
    // wholly before, inside or behind the block's own 64 entries
    const int32_t per = ((n + kRankWaves - 1) / kRankWaves + 15) & ~15;
    const int64_t lo64 = (int64_t)per * w;
    const int32_t lo = lo64 < n ? (int32_t)lo64 : n;
    const int32_t hi = lo + per < n && lo + per > 0 ? lo + per : n;
    uint32_t cnt = 0;
    int32_t j = lo;
    for (; j + 16 <= hi; j += 16) {
        if (entries && j >= i0 && j < i0 + 64) {
#pragma unroll
            for (int t = 0; t < 16; ++t)
                cnt += key_of(ids[j + t], G) < key + (uint32_t)(j + t < i);
        } else {
            const uint32_t lim = key + (uint32_t)(entries && j < i0);
#pragma unroll
            for (int t = 0; t < 16; ++t) cnt += key_of(ids[j + t], G) < lim;
        }
    }
    for (; j < hi; ++j) cnt += key_of(ids[j], G) < key + (uint32_t)(entries && j < i);

    part[w][lane] = cnt;
    __syncthreads();
    if (w != 0) return;
    uint32_t place = 0;
#pragma unroll
    for (int t = 0; t < kRankWaves; ++t) place += part[t][lane];
    if (entries) {
        if (i < n) {
            order[place] = key < G ? i : -1;
            if (slot) slot[i] = key < G ? (int32_t)place : -1;
        }
    } else if (g <= (int64_t)G) {
        offsets[g] = (int32_t)place;
    }
}

// ---- many entries: radix passes, lowest digit first -------------------------
//
// Each pass sorts stably by one digit: digit counts per tile of entries, an
// exclusive scan of each digit over the tiles, then every entry is moved to
// digit start + tile start + its rank inside the tile.  Ranks come from wave
// votes (lanes that share a digit), so no order depends on an atomic.
constexpr int kTileWaves = 4;
constexpr int kTileRounds = 8;
constexpr int kTile = kTileWaves * 64 * kTileRounds;  // entries per workgroup
constexpr int kMaxBits = 10;

__global__ __launch_bounds__(256) void k_group_hist(const int32_t *__restrict__ ids,
                                                    const uint32_t *__restrict__ keys, int64_t n,
                                                    uint32_t G, int shift, int bits,
                                                    uint32_t *__restrict__ counts) {
    __shared__ uint32_t h[1 << kMaxBits];
    const int D = 1 << bits;
    for (int t = threadIdx.x; t < D; t += 256) h[t] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kTile;
#pragma unroll
    for (int r = 0; r < kTile / 256; ++r) {
        const int64_t i = base + r * 256 + threadIdx.x;
        if (i < n) {
            const uint32_t key = keys ? keys[i] : key_of(ids[i], G);
            atomicAdd(&h[(key >> shift) & (D - 1)], 1u);
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < D; t += 256) counts[(int64_t)blockIdx.x * D + t] = h[t];
}

// counts[b][digit] becomes the sum over tiles before b; total[digit] the sum
// over all.  A workgroup serves 64 digits with 16 waves, each a run of tiles.
__global__ __launch_bounds__(1024) void k_group_scan(uint32_t *__restrict__ counts, int64_t tiles,
                                                     int bits, uint32_t *__restrict__ total) {
    __shared__ uint32_t part[16][64];
    const int D = 1 << bits;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int digit = blockIdx.x * 64 + lane;
    const int64_t per = (tiles + 15) / 16;
    const int64_t lo = per * w < tiles ? per * w : tiles;
    const int64_t hi = lo + per < tiles ? lo + per : tiles;
    uint32_t sum = 0;
    if (digit < D)
        for (int64_t b = lo; b < hi; ++b) sum += counts[b * D + digit];
    part[w][lane] = sum;
    __syncthreads();
    if (digit >= D) return;
    uint32_t run = 0, all = 0;
    for (int t = 0; t < 16; ++t) {
        if (t < w) run += part[t][lane];
        all += part[t][lane];
    }
    for (int64_t b = lo; b < hi; ++b) {
        const uint32_t c = counts[b * D + digit];
        counts[b * D + digit] = run;
        run += c;
    }
    if (w == 0) total[digit] = all;
}

// last: writes order and slot (and the sorted keys) instead of (key, entry)
__global__ __launch_bounds__(256) void k_group_scatter(
    const int32_t *__restrict__ ids, const uint32_t *__restrict__ keys,
    const int32_t *__restrict__ entry, int64_t n, uint32_t G, int shift, int bits,
    const uint32_t *__restrict__ counts, const uint32_t *__restrict__ total,
    uint32_t *__restrict__ keys_out, int32_t *__restrict__ entry_out, int last,
    int32_t *__restrict__ slot) {
    __shared__ uint32_t at[kTileWaves][1 << kMaxBits];
    __shared__ uint32_t wsum[kTileWaves];
    const int D = 1 << bits;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int t = threadIdx.x; t < D; t += 256)
        for (int v = 0; v < kTileWaves; ++v) at[v][t] = 0;
    __syncthreads();

    // each wave owns a run of 64 x kTileRounds consecutive entries
    const int64_t base = (int64_t)blockIdx.x * kTile + (int64_t)w * 64 * kTileRounds;
    uint32_t key[kTileRounds];
    int32_t ent[kTileRounds];
#pragma unroll
    for (int r = 0; r < kTileRounds; ++r) {
        const int64_t i = base + r * 64 + lane;
        key[r] = 0;
        ent[r] = -1;
        if (i < n) {
            key[r] = keys ? keys[i] : key_of(ids[i], G);
            ent[r] = entry ? entry[i] : (int32_t)i;
            atomicAdd(&at[w][(key[r] >> shift) & (D - 1)], 1u);
        }
    }
    __syncthreads();

    // digit starts: exclusive scan of the totals, plus this tile's start and
    // the counts of the waves before
    uint32_t carry = 0;
    for (int t0 = 0; t0 < D; t0 += 256) {
        const int t = t0 + threadIdx.x;
        const uint32_t own = t < D ? total[t] : 0;
        uint32_t inc = own;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t up = __shfl_up(inc, s);
            if (lane >= s) inc += up;
        }
        if (lane == 63) wsum[w] = inc;
        __syncthreads();
        uint32_t before = carry, all = 0;
        for (int v = 0; v < kTileWaves; ++v) {
            if (v < w) before += wsum[v];
            all += wsum[v];
        }
        if (t < D) {
            uint32_t run = before + inc - own + counts[(int64_t)blockIdx.x * D + t];
            for (int v = 0; v < kTileWaves; ++v) {
                const uint32_t c = at[v][t];
                at[v][t] = run;
                run += c;
            }
        }
        carry += all;
        __syncthreads();
    }

#pragma unroll
    for (int r = 0; r < kTileRounds; ++r) {
        const bool live = ent[r] >= 0;
        const uint32_t digit = (key[r] >> shift) & (D - 1);
        uint64_t peers = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((digit >> b) & 1);
            peers &= ((digit >> b) & 1) ? set : ~set;
        }
        const int before = __popcll(peers & ((1ull << lane) - 1));
        uint32_t p = 0;
        if (live) p = at[w][digit] + before;
        // the reads above come before the write below, and that before the
        // next round's reads (one wave, its own row of `at`)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (live && before == 0) at[w][digit] += (uint32_t)__popcll(peers);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (!live) continue;
        keys_out[p] = key[r];
        if (last) {
            entry_out[p] = key[r] < G ? ent[r] : -1;
            if (slot) slot[ent[r]] = key[r] < G ? (int32_t)p : -1;
        } else {
            entry_out[p] = ent[r];
        }
    }
}

// offsets[g] = #{p : sorted key < g}, by bisection
__global__ __launch_bounds__(256) void k_group_offsets(const uint32_t *__restrict__ keys,
                                                       int64_t n, int64_t G,
                                                       int32_t *__restrict__ offsets) {
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g <= G;
         g += (int64_t)gridDim.x * 256) {
        int64_t lo = 0, hi = n;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (keys[mid] < (uint64_t)g) lo = mid + 1;
            else hi = mid;
        }
        offsets[g] = (int32_t)lo;
    }
}

// Counting every place takes n (n + G) compares in one launch; the radix
// passes take 7 launches and more for any n.
bool use_rank(int64_t n, int64_t G) {
    return n <= 32768 && G <= (1 << 24) && (double)n * (double)(n + G) <= 1.0e9;
}

int key_bits(int64_t G) {  // bits of the largest key, G
    int b = 1;
    while ((G >> b) != 0) ++b;
    return b;
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t group_workspace(int64_t n, int64_t G) {
    if (use_rank(n, G)) return 256;
    const size_t arr = up256((size_t)n * 4);
    const size_t tiles = (size_t)((n + kTile - 1) / kTile);
    return 4 * arr + up256(tiles * (4u << kMaxBits)) + (4u << kMaxBits);
}

hipError_t launch_group(const int32_t *ids, int64_t n, int64_t G, int32_t *order,
                        int32_t *offsets, int32_t *slot, void *ws, hipStream_t st) {
    if (use_rank(n, G)) {
        const int32_t eb = (int32_t)((n + 63) / 64);
        const unsigned grid = (unsigned)(eb + (G + 1 + 63) / 64);
        timing_before(st, "k_group_rank");
        hipLaunchKernelGGL(k_group_rank, dim3(grid), dim3(kRankWaves * 64), 0, st, ids, (int32_t)n,
                           (uint32_t)G, eb, order, offsets, slot);
        timing_after(st);
        return hipGetLastError();
    }
    const size_t arr = up256((size_t)n * 4);
    const int64_t tiles = (n + kTile - 1) / kTile;
    char *p = static_cast<char *>(ws);
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(p), reinterpret_cast<uint32_t *>(p + arr)};
    int32_t *ent[2] = {reinterpret_cast<int32_t *>(p + 2 * arr),
                       reinterpret_cast<int32_t *>(p + 3 * arr)};
    uint32_t *counts = reinterpret_cast<uint32_t *>(p + 4 * arr);
    uint32_t *total = reinterpret_cast<uint32_t *>(p + 4 * arr +
                                                   up256((size_t)tiles * (4u << kMaxBits)));
    const int tb = key_bits(G);
    const int passes = (tb + kMaxBits - 1) / kMaxBits;
    const int bits = (tb + passes - 1) / passes;
    const dim3 grid((unsigned)tiles), block(256);
    const uint32_t *kin = nullptr;
    const int32_t *ein = nullptr;
    for (int q = 0; n > 0 && q < passes; ++q) {
        const bool last = q == passes - 1;
        uint32_t *kout = keys[q & 1];
        int32_t *eout = last ? order : ent[q & 1];
        hipLaunchKernelGGL(k_group_hist, grid, block, 0, st, ids, kin, n, (uint32_t)G, q * bits,
                           bits, counts);
        hipLaunchKernelGGL(k_group_scan, dim3((unsigned)(((1 << bits) + 63) / 64)), dim3(1024), 0,
                           st, counts, tiles, bits, total);
        if (last) timing_before(st, "k_group_scatter");
        hipLaunchKernelGGL(k_group_scatter, grid, block, 0, st, ids, kin, ein, n, (uint32_t)G,
                           q * bits, bits, counts, total, kout, eout, (int)last, slot);
        if (last) timing_after(st);
        kin = kout;
        ein = eout;
    }
    const int64_t want = (G + 1 + 255) / 256;
    hipLaunchKernelGGL(k_group_offsets, dim3((unsigned)(want < 65536 ? want : 65536)), block, 0,
                       st, kin, n, G, offsets);
    return hipGetLastError();
}

}  // namespace vs
