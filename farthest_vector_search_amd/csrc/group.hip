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

__device__ __forceinline__ uint32_t key_of(int32_t id, uint32_t G) {
    const uint32_t u = (uint32_t)id;
    return u < G ? u : G;
}

// ---- few entries: every place by counting ---------------------------------
//
// place(i) = #{j : (key_j, j) < (key_i, i)} and offsets[g] = #{j : key_j < g},
// one launch with nothing passed between workgroups.  A workgroup serves 16
// entries (or 16 units) with 16 waves, each wave counting over a 16th of the
// keys: lanes hold 64 keys, an entry's key is uniform, so 64 pairs cost one
// vector compare and a scalar bit count of its mask.  With many units their
// offsets come from the sorted keys instead (keys_out, k_group_offsets).
constexpr int kRankWaves = 16;
constexpr int kRankEntries = 16;

__global__ __launch_bounds__(kRankWaves * 64) void k_group_rank(
    const int32_t *__restrict__ ids, int32_t n, uint32_t G, int32_t entry_blocks,
    int32_t *__restrict__ order, int32_t *__restrict__ offsets, int32_t *__restrict__ slot,
    uint32_t *__restrict__ keys_out) {
    __shared__ uint32_t part[kRankWaves][kRankEntries];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool entries = (int32_t)blockIdx.x < entry_blocks;
    const int e = lane & (kRankEntries - 1);
    const int32_t i0 = entries ? (int32_t)blockIdx.x * kRankEntries : 0;
    const int32_t i = i0 + e;
    const int64_t g = entries ? 0 : ((int64_t)blockIdx.x - entry_blocks) * kRankEntries + e;
    const uint32_t key = entries ? (i < n ? key_of(ids[i], G) : G)
                                 : (uint32_t)(g < (int64_t)G ? g : (int64_t)G);

    const int32_t per = ((n + kRankWaves - 1) / kRankWaves + 63) & ~63;
    const int32_t lo = per * w < n ? per * w : n;
    const int32_t hi = lo + per < n ? lo + per : n;
    uint32_t cnt[kRankEntries] = {};
    constexpr int kHeld = 4;
    for (int32_t j0 = lo; j0 < hi; j0 += 64 * kHeld) {
        uint32_t kv[kHeld];
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int32_t j = j0 + 64 * h + lane;
            kv[h] = j < hi ? key_of(ids[j], G) : 0xffffffffu;  // above every key
        }
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int32_t jv = j0 + 64 * h;
            if (jv >= hi) break;
            if (entries && jv < i0 + kRankEntries && jv + 64 > i0) {
                // the block's own entries are among these keys
#pragma unroll
                for (int t = 0; t < kRankEntries; ++t) {
                    const uint32_t lim = __builtin_amdgcn_readlane(key, t);
                    cnt[t] += __popcll(__ballot(kv[h] < lim + (uint32_t)(jv + lane < i0 + t)));
                }
            } else {
                const uint32_t up = entries && jv < i0 ? 1u : 0u;  // equal keys before i count
#pragma unroll
                for (int t = 0; t < kRankEntries; ++t)
                    cnt[t] += __popcll(__ballot(kv[h] < __builtin_amdgcn_readlane(key, t) + up));
            }
        }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int t = 0; t < kRankEntries; ++t) mine = lane == t ? cnt[t] : mine;
    if (lane < kRankEntries) part[w][lane] = mine;
    __syncthreads();
    if (threadIdx.x >= kRankEntries) return;
    uint32_t place = 0;
#pragma unroll
    for (int t = 0; t < kRankWaves; ++t) place += part[t][lane];
    if (entries) {
        if (i < n) {
            order[place] = key < G ? i : -1;
            if (slot) slot[i] = key < G ? (int32_t)place : -1;
            if (keys_out) keys_out[place] = key;
        }
    } else if (g <= (int64_t)G) {
        offsets[g] = (int32_t)place;
    }
}

// ---- many entries: radix passes, lowest digit first -------------------------
//
// Each pass sorts stably by one digit of up to kMaxBits bits: digit counts per
// tile of entries, then every entry is moved to digit start + count of its
// digit in the tiles before + its rank inside the tile.  Ranks come from wave
// votes (lanes that share a digit), so no order depends on an atomic.  Up to
// kFusedCounts counts in all, each tile of the move adds up those it needs by
// itself; beyond, a scan over the tiles runs in between.  The launches are short
// and wait for each other: 65,536 entries take 8.5 us for 128 units and 21 us
// for 16,384, 131,072 entries of 65,536 units 30 us, 1,000,000 of 128 units 44 us
// and of 262,144 units 127 us (the scan has a workgroup per 64 digits).
constexpr int kTileWaves = 8;
constexpr int kTileThreads = kTileWaves * 64;
constexpr int kTileRounds = 2;
constexpr int kTile = kTileThreads * kTileRounds;  // entries per workgroup
constexpr int kMaxBits = 10;
// By itself / with the scan (us): 131,072 entries in 128 digits 9.4 / 12.4, in
// 512 digits twice 30.7 / 31.3, in 1,024 digits 17.9 / 14.0; 262,144 entries in
// 256 digits 12.4 / 15.7, in 1,024 digits 28.8 / 18.6.
constexpr int64_t kFusedCounts = 65536;

__global__ __launch_bounds__(kTileThreads) void k_group_hist(const int32_t *__restrict__ ids,
                                                             const uint32_t *__restrict__ keys,
                                                             int64_t n, uint32_t G, int shift,
                                                             int bits,
                                                             uint32_t *__restrict__ counts) {
    __shared__ uint32_t h[1 << kMaxBits];
    const int D = 1 << bits;
    for (int t = threadIdx.x; t < D; t += kTileThreads) h[t] = 0;
    const int64_t base = (int64_t)blockIdx.x * kTile;
    uint32_t key[kTileRounds];
#pragma unroll
    for (int r = 0; r < kTileRounds; ++r) {
        const int64_t i = base + r * kTileThreads + threadIdx.x;
        if (i < n) key[r] = keys ? keys[i] : key_of(ids[i], G);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTileRounds; ++r)
        if (base + r * kTileThreads + threadIdx.x < n)
            atomicAdd(&h[(key[r] >> shift) & (D - 1)], 1u);
    __syncthreads();
    for (int t = threadIdx.x; t < D; t += kTileThreads)
        counts[(int64_t)blockIdx.x * D + t] = h[t];
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

// scanned: counts and total as k_group_scan leaves them; else the tiles' plain
// counts.  last: writes order and slot instead of entries.  starts (last pass)
// receives the D digit starts and n, from tile 0.
__global__ __launch_bounds__(kTileThreads) void k_group_scatter(
    const int32_t *__restrict__ ids, const uint32_t *__restrict__ keys,
    const int32_t *__restrict__ entry, int64_t n, uint32_t G, int shift, int bits,
    const uint32_t *__restrict__ counts, const uint32_t *__restrict__ total, int scanned,
    int tiles, uint32_t *__restrict__ keys_out, int32_t *__restrict__ entry_out, int last,
    int32_t *__restrict__ slot, int32_t *__restrict__ starts, int64_t n_starts) {
    __shared__ uint32_t at[kTileWaves][1 << kMaxBits];
    __shared__ uint32_t sum_all[1 << kMaxBits], sum_before[1 << kMaxBits];
    __shared__ uint32_t wsum[kTileWaves];
    const int D = 1 << bits;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

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
        }
    }
    for (int t = threadIdx.x; t < D; t += kTileThreads) {
#pragma unroll
        for (int v = 0; v < kTileWaves; ++v) at[v][t] = 0;
        sum_all[t] = scanned ? total[t] : 0;
        sum_before[t] = scanned ? counts[(int64_t)blockIdx.x * D + t] : 0;
    }
    __syncthreads();
    if (!scanned) {
        // threads beyond the digits share the tiles out among them
        const int digit = threadIdx.x & (D - 1);
        const int group = threadIdx.x >> bits, groups = D < kTileThreads ? kTileThreads >> bits : 1;
        for (int t = digit; t < D; t += kTileThreads) {
            uint32_t all = 0, before = 0;
#pragma unroll 16
            for (int b = group; b < tiles; b += groups) {
                const uint32_t c = counts[b * D + t];
                all += c;
                before += b < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&sum_all[t], all);
            atomicAdd(&sum_before[t], before);
        }
    }
#pragma unroll
    for (int r = 0; r < kTileRounds; ++r)
        if (ent[r] >= 0) atomicAdd(&at[w][(key[r] >> shift) & (D - 1)], 1u);
    __syncthreads();

    // digit starts: exclusive scan of the totals; then each wave's own start
    uint32_t carry = 0;
    for (int t0 = 0; t0 < D; t0 += kTileThreads) {
        const int t = t0 + threadIdx.x;
        const uint32_t own = t < D ? sum_all[t] : 0;
        uint32_t inc = own;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t up = __shfl_up(inc, s);
            if (lane >= s) inc += up;
        }
        if (lane == 63) wsum[w] = inc;
        __syncthreads();
        uint32_t before = carry, all = 0;
#pragma unroll
        for (int v = 0; v < kTileWaves; ++v) {
            if (v < w) before += wsum[v];
            all += wsum[v];
        }
        if (t < D) {
            const uint32_t start = before + inc - own;
            if (starts && blockIdx.x == 0 && t < n_starts) starts[t] = (int32_t)start;
            uint32_t run = start + sum_before[t];
#pragma unroll
            for (int v = 0; v < kTileWaves; ++v) {
                const uint32_t c = at[v][t];
                at[v][t] = run;
                run += c;
            }
        }
        carry += all;
        __syncthreads();
    }
    if (starts && blockIdx.x == 0 && threadIdx.x == 0 && D < n_starts) starts[D] = (int32_t)n;

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
        if (keys_out) keys_out[p] = key[r];
        if (last) {
            entry_out[p] = key[r] < G ? ent[r] : -1;
            if (slot) slot[ent[r]] = key[r] < G ? (int32_t)p : -1;
        } else {
            entry_out[p] = ent[r];
        }
    }
}

// offsets[g] = #{p : sorted key < g}, by bisection between the starts of g's
// last digit and of the next one (over all keys without starts)
__global__ __launch_bounds__(256) void k_group_offsets(const uint32_t *__restrict__ keys,
                                                       int64_t n, int64_t G, int shift,
                                                       const int32_t *__restrict__ starts,
                                                       int32_t *__restrict__ offsets) {
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g <= G;
         g += (int64_t)gridDim.x * 256) {
        int64_t lo = 0, hi = 0;
        if (!starts) {
            hi = n;
        } else if (n > 0) {
            lo = (uint32_t)starts[g >> shift];
            hi = (uint32_t)starts[(g >> shift) + 1];
        }
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (keys[mid] < (uint64_t)g) lo = mid + 1;
            else hi = mid;
        }
        offsets[g] = (int32_t)lo;
    }
}

// Where each way wins (us, measured on MI355X; counting / radix): n = 2,000
// with 64 units 4.3 / 7.5, with 16,384 units 8.4 / 17.6; n = 4,096 with 64
// units 8.5 / 8.1, with 16,384 units 10.0 / 19.6; n = 8,192 with 64 units
// 18.5 / 8.3, with 1,000 units 18.7 / 11.5.  Units counted in the same launch
// against a second one that bisects: 2,000 entries with 4,096 units 6.6 / 8.2,
// with 8,192 units 9.0 / 8.3.
constexpr int64_t kRankMost = 4096;
constexpr int64_t kRankUnits = 4096;

int key_bits(int64_t G) {  // bits of the largest key, G
    int b = 1;
    while ((G >> b) != 0) ++b;
    return b;
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// keys and entries twice, counts of the tiles, totals and starts of the digits
size_t group_workspace(int64_t n, int64_t G) {
    if (n <= kRankMost) return G <= kRankUnits ? 0 : up256((size_t)n * 4);
    const size_t arr = up256((size_t)n * 4);
    const size_t tiles = (size_t)((n + kTile - 1) / kTile);
    return 4 * arr + up256(tiles * (4u << kMaxBits)) + (4u << kMaxBits) + up256((4u << kMaxBits) + 4);
}

hipError_t launch_group(const int32_t *ids, int64_t n, int64_t G, int32_t *order,
                        int32_t *offsets, int32_t *slot, void *ws, hipStream_t st) {
    const unsigned offset_grid = (unsigned)((G + 256) / 256 < 65536 ? (G + 256) / 256 : 65536);
    if (n <= kRankMost) {
        const int32_t eb = (int32_t)((n + kRankEntries - 1) / kRankEntries);
        const bool in_one = G <= kRankUnits;
        const int64_t ub = in_one ? (G + 1 + kRankEntries - 1) / kRankEntries : 0;
        uint32_t *sorted = static_cast<uint32_t *>(ws);
        timing_before(st, "k_group_rank");
        if (eb + ub > 0)
            hipLaunchKernelGGL(k_group_rank, dim3((unsigned)(eb + ub)), dim3(kRankWaves * 64), 0,
                               st, ids, (int32_t)n, (uint32_t)G, eb, order, offsets, slot,
                               in_one ? nullptr : sorted);
        timing_after(st);
        if (!in_one)
            hipLaunchKernelGGL(k_group_offsets, dim3(offset_grid), dim3(256), 0, st, sorted, n, G,
                               0, nullptr, offsets);
        return hipGetLastError();
    }
    const size_t arr = up256((size_t)n * 4);
    const int64_t tiles = (n + kTile - 1) / kTile;
    char *p = static_cast<char *>(ws);
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(p), reinterpret_cast<uint32_t *>(p + arr)};
    int32_t *ent[2] = {reinterpret_cast<int32_t *>(p + 2 * arr),
                       reinterpret_cast<int32_t *>(p + 3 * arr)};
    uint32_t *counts = reinterpret_cast<uint32_t *>(p + 4 * arr);
    char *tail = p + 4 * arr + up256((size_t)tiles * (4u << kMaxBits));
    uint32_t *total = reinterpret_cast<uint32_t *>(tail);
    int32_t *starts = reinterpret_cast<int32_t *>(tail + (4u << kMaxBits));
    const int tb = key_bits(G);
    const int passes = (tb + kMaxBits - 1) / kMaxBits;
    const int bits = (tb + passes - 1) / passes;
    const int64_t D = int64_t(1) << bits;
    const bool scan = tiles * D > kFusedCounts;
    const dim3 grid((unsigned)tiles), block(kTileThreads);
    const uint32_t *kin = nullptr;
    const int32_t *ein = nullptr;
    for (int q = 0; q < passes; ++q) {
        const bool last = q == passes - 1;
        // one digit holds the whole key: its starts are the offsets
        const bool direct = passes == 1;
        uint32_t *kout = direct ? nullptr : keys[q & 1];
        int32_t *eout = last ? order : ent[q & 1];
        hipLaunchKernelGGL(k_group_hist, grid, block, 0, st, ids, kin, n, (uint32_t)G, q * bits,
                           bits, counts);
        if (scan)
            hipLaunchKernelGGL(k_group_scan, dim3((unsigned)((D + 63) / 64)), dim3(1024), 0, st,
                               counts, tiles, bits, total);
        if (last) timing_before(st, "k_group_scatter");
        hipLaunchKernelGGL(k_group_scatter, grid, block, 0, st, ids, kin, ein, n, (uint32_t)G,
                           q * bits, bits, counts, total, (int)scan, (int)tiles, kout, eout,
                           (int)last, slot, direct ? offsets : last ? starts : nullptr,
                           direct ? G + 1 : D + 1);
        if (last) timing_after(st);
        if (direct) return hipGetLastError();
        kin = kout;
        ein = eout;
    }
    hipLaunchKernelGGL(k_group_offsets, dim3(offset_grid), dim3(256), 0, st, kin, n, G,
                       (passes - 1) * bits, starts, offsets);
    return hipGetLastError();
}

}  // namespace vs
