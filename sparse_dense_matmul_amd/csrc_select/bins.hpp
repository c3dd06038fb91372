// Stable sort of ids on the device, in few launches: the sort behind the
// routing of tokens to experts (a bin per expert) and behind the embedding's
// gradient (tokens by id). Places depend only on the ids: the order is unique,
// equal to a sequential counting sort's.
//
//  - k_bin_count / k_bin_place: one pass of a counting sort over tiles.
//    k_bin_count counts every tile's digits; in k_bin_place each block sums the
//    counts of the tiles before its own (at most kBinBlocks of them, so no
//    third launch scans them), then ranks its elements. Each wave owns a
//    contiguous piece of the tile and counters of its own, so ranking needs no
//    barrier between rounds: a round's 64 lanes rank equal digits by ballots,
//    in lane order. A list of one tile needs no k_bin_count. Bound by latency:
//    4.2 us in one launch at 512 slots over 128 experts, 11 at 4,096, 5.4 + 10.5
//    us at 131,072, 4 + 19 at 524,288 over 256.
//  - k_rank: every element's place counted directly, one launch: 3.8 us at 64
//    elements and 4.4 at 1,024, a launch and two dependent reads; 7.0 at 4,096 and
//    11.4 at 8,192, of which the compares' issue (below) explains 3.4.
//  - k_chunk_rank / k_merge_rank: chunks of 1,024 placed directly, then every
//    element's place found by binary searches in the other chunks, two launches:
//    6.7 + 4.4 us at 12,289 elements, 11.9 + 14.8 at 65,536, the second bound by
//    LDS reads.
// Times are the kernels' own, in a trace, without the zeroing beside them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rows.hpp"

namespace vspmm {

constexpr int kBinThreads = 512;
constexpr int kBinWaves = kBinThreads / 64;
constexpr int kBinBlocks = 256;   // most tiles of a pass
constexpr int kBinPiece = 256;    // fewest elements of a wave's piece
constexpr int kBinMax = 4097;     // most bins (counters of 8 waves: 131,104 bytes of LDS)

// Dynamic LDS of k_bin_place.
inline size_t bin_lds(int bins) { return size_t(kBinWaves) * (bins + 1) * 4; }

// Elements per wave's piece: the least multiple of 64 that keeps the tiles
// within kBinBlocks; one tile, and so one launch, for up to 4,096 elements.
inline int bin_piece(int64_t n) {
    if (n <= 2 * kBinPiece * kBinWaves)
        return n <= 0 ? 64 : int((n + kBinWaves * 64 - 1) / (kBinWaves * 64)) * 64;
    const int64_t per = (n + int64_t(kBinBlocks) * kBinWaves - 1) / (int64_t(kBinBlocks) * kBinWaves);
    const int64_t p = (per + 63) / 64 * 64;
    return int(p < kBinPiece ? kBinPiece : p);
}
inline int bin_blocks(int64_t n) {
    const int64_t tile = int64_t(bin_piece(n)) * kBinWaves;
    return int((n + tile - 1) / tile);
}

// No list of at most n elements has more tiles.
inline int bin_blocks_most(int64_t n) {
    const int64_t tiles = (n + kBinPiece * kBinWaves - 1) / (kBinPiece * kBinWaves);
    return int(tiles < kBinBlocks ? tiles : kBinBlocks);
}

// The sort key of element i: its id, or `limit` for an id outside
// [0, limit), which sorts such elements last.
template <typename I>
__device__ __forceinline__ uint32_t bin_key(const I *ids, int64_t i, int64_t limit) {
    const int64_t id = int64_t(ids[i]);
    return uint32_t(id >= 0 && id < limit ? id : limit);
}

// One pass: the keys, the digit it sorts by (shift < 0: the whole key), and the
// launch's tiles (its first nb blocks).
template <typename I>
struct BinPass {
    const I *ids;
    int64_t n, limit;
    int shift, bins, piece, nb;
    __device__ __forceinline__ int digit(uint32_t key) const {
        return shift < 0 ? int(key) : int((key >> shift) & uint32_t(bins - 1));
    }
};

// counts[b * bins + d] = elements of tile b whose digit is d. Blocks past the
// tiles zero rows; *clear (may be null) = 0.
template <typename I>
__global__ void __launch_bounds__(kBinThreads)
k_bin_count(BinPass<I> ps, int *__restrict__ counts, int *clear, ZeroRows zero) {
    extern __shared__ int hist[];
    if (int(blockIdx.x) >= ps.nb) {
        zero.run(ps.nb);
        return;
    }
    if (clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
    for (int d = threadIdx.x; d < ps.bins; d += kBinThreads) hist[d] = 0;
    __syncthreads();
    const int64_t tile = int64_t(ps.piece) * kBinWaves, lo = blockIdx.x * tile;
    const int64_t hi = lo + tile < ps.n ? lo + tile : ps.n;
    for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += 4 * kBinThreads) {
        uint32_t key[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t i = i0 + r * kBinThreads;
            if (i < hi) key[r] = bin_key(ps.ids, i, ps.limit);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (i0 + r * kBinThreads < hi) atomicAdd(&hist[ps.digit(key[r])], 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < ps.bins; d += kBinThreads)
        counts[int64_t(blockIdx.x) * ps.bins + d] = hist[d];
}

// Exclusive scan over a block of kBinThreads threads.
__device__ __forceinline__ int bin_block_scan(int x, int *sh /*[kBinWaves]*/, int &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(inc, d);
        if (lane >= d) inc += y;
    }
    if (lane == 63) sh[wave] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int k = 0; k < kBinWaves; ++k) {
        const int s = sh[k];
        if (k < wave) before += s;
        total += s;
    }
    __syncthreads();
    return before + inc - x;
}

// What a pass writes for element i of place p, whose key and payload it holds.
struct PlaceRoute {  // order[p] = i, position[i] = p, or ~p for a dropped slot
    int *order, *position;
    __device__ __forceinline__ int pay_of(int64_t i) const { return int(i); }
    __device__ __forceinline__ void put(int64_t i, int p, uint32_t key, int pay, int64_t limit) const {
        order[p] = pay;
        position[i] = key == uint32_t(limit) ? ~p : p;
    }
};
struct PlaceKeys {  // keys[p] = key, pay[p] = from ? from[i] : i
    uint32_t *keys;
    int *pay;
    const int *from;
    __device__ __forceinline__ int pay_of(int64_t i) const { return from ? from[i] : int(i); }
    __device__ __forceinline__ void put(int64_t, int p, uint32_t key, int value, int64_t) const {
        keys[p] = key;
        pay[p] = value;
    }
};

// `bits` bits hold a digit. offsets (may be null): the first place of every
// bin, written by block 0. counts is not read when there is one tile.
template <typename I, typename Out>
__global__ void __launch_bounds__(kBinThreads)
k_bin_place(BinPass<I> ps, int bits, const int *__restrict__ counts, Out out,
            int *__restrict__ offsets) {
    extern __shared__ int wc[];             // [kBinWaves][bins], then
    int *const sh = wc + kBinWaves * ps.bins;  // [kBinWaves] for the scan
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = gridDim.x, blk = blockIdx.x, bins = ps.bins;
    // a piece is walked 4 rounds of 64 at a time, their loads issued together;
    // the first four rounds' keys (all of a short list's) are loaded once. The
    // choice between the two arrays in the counting loop puts them in scratch
    // memory (48 bytes a lane), not in registers.
    const int64_t lo = (int64_t(blk) * kBinWaves + wave) * ps.piece;
    const int64_t hi = lo + ps.piece < ps.n ? lo + ps.piece : ps.n;
    uint32_t first_keys[4];
    auto load4 = [&](uint32_t (&key)[4], int64_t i0) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            key[r] = i0 + r * 64 + lane < hi ? bin_key(ps.ids, i0 + r * 64 + lane, ps.limit) : 0u;
    };
    load4(first_keys, lo);
    for (int d = tid; d < kBinWaves * bins; d += kBinThreads) wc[d] = 0;
    __syncthreads();
    int *mine = wc + wave * bins;
    for (int64_t i0 = lo; i0 < hi; i0 += 256) {
        uint32_t key[4];
        if (i0 > lo) load4(key, i0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (i0 + r * 64 + lane < hi)
                atomicAdd(&mine[ps.digit(i0 > lo ? key[r] : first_keys[r])], 1);
    }
    __syncthreads();
    int carry = 0;  // elements of all lower digits
    for (int d0 = 0; d0 < bins; d0 += kBinThreads) {
        const int d = d0 + tid;
        int before = 0, total = 0;
        if (d < bins) {
            if (nb == 1) {
#pragma unroll
                for (int w = 0; w < kBinWaves; ++w) total += wc[w * bins + d];
            } else {
                for (int b0 = 0; b0 < nb; b0 += 32) {
                    int c[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        c[j] = b0 + j < nb ? counts[int64_t(b0 + j) * bins + d] : 0;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        before += b0 + j < blk ? c[j] : 0;
                        total += c[j];
                    }
                }
            }
        }
        int all;
        const int first = carry + bin_block_scan(total, sh, all);
        carry += all;
        if (d < bins) {
            if (offsets && blk == 0) offsets[d] = first;
            int run = first + before;
#pragma unroll
            for (int w = 0; w < kBinWaves; ++w) {
                const int c = wc[w * bins + d];
                wc[w * bins + d] = run;
                run += c;
            }
        }
    }
    __syncthreads();
    const uint64_t lt = lane == 0 ? 0ull : (~0ull >> (64 - lane));
    volatile int *next = mine;  // this wave alone reads and writes its counters
    for (int64_t i0 = lo; i0 < hi; i0 += 256) {
        uint32_t key[4];
        if (i0 > lo) load4(key, i0);
        else
#pragma unroll
            for (int r = 0; r < 4; ++r) key[r] = first_keys[r];
        int pay[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) pay[r] = i0 + r * 64 + lane < hi ? out.pay_of(i0 + r * 64 + lane) : 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t i = i0 + r * 64 + lane;
            const bool live = i < hi;
            const int d = ps.digit(key[r]);
            uint64_t same = __ballot(live);
            if (!same) break;
            for (int b = 0; b < bits; ++b) {
                const bool bit = (d >> b) & 1;
                const uint64_t with = __ballot(bit);
                same &= bit ? with : ~with;
            }
            const int rank = __popcll(same & lt);
            if (live) {
                const int at = next[d];
                if (rank == 0) next[d] = at + __popcll(same);
                out.put(i, at + rank, key[r], pay[r], ps.limit);
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// Every element's place, counted directly: the keys below its own, and the
// equal ones before it. A block holds all keys in LDS and places kRankTile
// elements: a lane holds kRankHeld of them, so that a quad of keys read from
// LDS serves four, and the block's lanes share the keys out between them. Two
// integer operations a pair: over the card's 16,384 lanes n^2 / 8,192 cycles, 0.05
// us at 1,024 elements and 3.4 at 8,192. What else the time grows by there (every
// block reads the whole list, and one block fills a CU) was not measured apart.
// kRankMax: the whole gradient of width 8 takes 17.5 us so at 4,096 elements, 19.4
// at 6,144, 21.6 at 8,192 and 29.2 at 10,240; by chunks and their merge 19.7, 20.1,
// 20.8 and 21.5.
constexpr int kRankThreads = 1024;
constexpr int kRankHeld = 4;
constexpr int kRankTile = 32;
constexpr int kRankMax = 8192;   // most elements

// The held elements' places among keys[0, padded) (in LDS, padded with ~0 to
// whole quads), `first` the index of the block's first element there; left in
// place[kRankTile]. All THREADS threads call it.
template <int THREADS>
__device__ __forceinline__ void rank_tile(const uint32_t *keys, int padded, int first, int *place) {
    constexpr int LANES = kRankTile / kRankHeld;  // lanes that hold the tile
    constexpr int SHARES = THREADS / LANES;       // shares of the keys
    const int tid = threadIdx.x;
    const int mine = (tid % LANES) * kRankHeld;
    const uint4 held = *reinterpret_cast<const uint4 *>(&keys[first + mine]);
    const uint32_t key[kRankHeld] = {held.x, held.y, held.z, held.w};
    int below[kRankHeld] = {};
    for (int q = tid / LANES; q < padded / 4; q += SHARES) {
        const uint4 k = *reinterpret_cast<const uint4 *>(&keys[4 * q]);
        // keys before the tile count when equal, too; those after it (and the
        // tile's own, whose equal ones are added below) only when smaller
        const uint32_t equal = 4 * q < first ? 1u : 0u;
#pragma unroll
        for (int h = 0; h < kRankHeld; ++h) {
            const uint32_t bound = key[h] + equal;
            below[h] += (k.x < bound) + (k.y < bound) + (k.z < bound) + (k.w < bound);
        }
    }
#pragma unroll
    for (int h = 0; h < kRankHeld; ++h) {
#pragma unroll
        for (int m = LANES; m < 64; m *= 2) below[h] += __shfl_xor(below[h], m);
        if ((tid & 63) < LANES && below[h]) atomicAdd(&place[mine + h], below[h]);
    }
    if (tid < kRankTile) {
        int equal = 0;
        for (int j = 0; j < tid; ++j) equal += keys[first + j] == keys[first + tid];
        if (equal) atomicAdd(&place[tid], equal);
    }
    __syncthreads();
}

template <typename I>
__global__ void __launch_bounds__(kRankThreads)
k_rank(const I *__restrict__ ids, int n, int64_t limit, int n_blocks, PlaceKeys out, int *clear,
       ZeroRows zero) {
    __shared__ __align__(16) uint32_t keys[kRankMax];
    __shared__ int place[kRankTile];
    const int tid = threadIdx.x;
    if (int(blockIdx.x) >= n_blocks) {
        zero.run(n_blocks);
        return;
    }
    if (clear && blockIdx.x == 0 && tid == 0) *clear = 0;
    const int padded = (n + kRankTile - 1) & ~(kRankTile - 1);
    for (int i = tid; i < padded; i += kRankThreads)
        keys[i] = i < n ? bin_key(ids, i, limit) : ~0u;
    if (tid < kRankTile) place[tid] = 0;
    __syncthreads();
    const int first = blockIdx.x * kRankTile, i = first + tid;
    rank_tile<kRankThreads>(keys, padded, first, place);
    if (tid < kRankTile && i < n) out.put(i, place[tid], keys[i], i, limit);
}

// Chunks of kChunkKeys elements sorted on their own: element i of chunk c goes
// to the chunk's place of it.
constexpr int kChunkKeys = 1024;
constexpr int kChunkThreads = 256;

template <typename I>
__global__ void __launch_bounds__(kChunkThreads)
k_chunk_rank(const I *__restrict__ ids, int n, int64_t limit, int n_blocks, PlaceKeys out, int *clear,
             ZeroRows zero) {
    __shared__ __align__(16) uint32_t keys[kChunkKeys];
    __shared__ int place[kRankTile];
    const int tid = threadIdx.x;
    if (int(blockIdx.x) >= n_blocks) {
        zero.run(n_blocks);
        return;
    }
    if (clear && blockIdx.x == 0 && tid == 0) *clear = 0;
    const int block0 = blockIdx.x * kRankTile;
    const int chunk0 = block0 & ~(kChunkKeys - 1);
#pragma unroll
    for (int r = 0; r < kChunkKeys / kChunkThreads; ++r) {
        const int i = chunk0 + r * kChunkThreads + tid;
        keys[r * kChunkThreads + tid] = i < n ? bin_key(ids, i, limit) : ~0u;
    }
    if (tid < kRankTile) place[tid] = 0;
    __syncthreads();
    const int first = block0 - chunk0, i = block0 + tid;
    rank_tile<kChunkThreads>(keys, kChunkKeys, first, place);
    if (tid < kRankTile && i < n) out.put(i, chunk0 + place[tid], keys[first + tid], i, limit);
}

// The sorted chunks merged: an element's place is its place in its chunk, plus
// the keys at or below its own in the chunks before, and below it in those
// after. A block places TILE elements (neighbours in a chunk, whose searches
// take nearly the same path), the chunks' keys in LDS kMergeStage at a time, the
// next stage's on their way in registers; 1,024 / TILE threads share an
// element's chunks and search several at once.
constexpr int kMergeThreads = 1024;
constexpr int kMergeStage = 16;
// Most elements. The whole gradient of width 8 over a table of 50,021 rows takes 41
// us so at 49,152 elements, 49.6 at 65,536 and 69 at 98,304; by digits, two passes,
// 45, 49.4 and 53. Over 400 rows, one pass, the digits are ahead from 32,768 on: 27
// for 29.5, at 65,536 32 for 45; the limit does not look at the table.
constexpr int kMergeMax = 65536;

constexpr size_t kMergeLds = size_t(kMergeStage * kChunkKeys) * 4;  // 64 KB

template <int TILE>
__global__ void __launch_bounds__(kMergeThreads)
k_merge_rank(const uint32_t *__restrict__ chunk_keys, const int *__restrict__ chunk_pay, int n,
             PlaceKeys out) {
    constexpr int SLOTS = kMergeThreads / TILE, PER = kMergeStage / SLOTS;
    constexpr int QUADS = kMergeStage * kChunkKeys / 4 / kMergeThreads;  // a thread's of a stage
    extern __shared__ __align__(16) uint32_t keys[];
    const int tid = threadIdx.x;
    const int e = blockIdx.x * TILE + (tid & (TILE - 1));
    const int slot = tid / TILE;
    const uint32_t key = e < n ? chunk_keys[e] : 0u;
    const int home = e / kChunkKeys, chunks = (n + kChunkKeys - 1) / kChunkKeys;
    uint4 next[QUADS];
    auto fetch = [&](int c0) {  // past the list: above every key
#pragma unroll
        for (int r = 0; r < QUADS; ++r) {
            const int64_t g = int64_t(c0) * kChunkKeys + (r * kMergeThreads + tid) * 4;
            next[r] = uint4{~0u, ~0u, ~0u, ~0u};
            if (g + 3 < n) {
                next[r] = *reinterpret_cast<const uint4 *>(chunk_keys + g);
            } else if (g < n) {
                next[r].x = chunk_keys[g];
                if (g + 1 < n) next[r].y = chunk_keys[g + 1];
                if (g + 2 < n) next[r].z = chunk_keys[g + 2];
            }
        }
    };
    fetch(0);
    int sum = 0;
    for (int c0 = 0; c0 < chunks; c0 += kMergeStage) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < QUADS; ++r)
            *reinterpret_cast<uint4 *>(&keys[(r * kMergeThreads + tid) * 4]) = next[r];
        __syncthreads();
        if (c0 + kMergeStage < chunks) fetch(c0 + kMergeStage);
        // the keys below `bound` among each chunk's 1,024
        int at[PER];
        uint32_t bound[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            at[j] = (j * SLOTS + slot) * kChunkKeys;
            bound[j] = key + (c0 + j * SLOTS + slot < home ? 1u : 0u);
        }
#pragma unroll
        for (int step = kChunkKeys / 2; step >= 1; step /= 2)
#pragma unroll
            for (int j = 0; j < PER; ++j) at[j] += keys[at[j] + step - 1] < bound[j] ? step : 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            at[j] += keys[at[j]] < bound[j] ? 1 : 0;
            if (c0 + j * SLOTS + slot != home) sum += at[j] - (j * SLOTS + slot) * kChunkKeys;
        }
    }
    __syncthreads();
    int *const place = reinterpret_cast<int *>(keys);  // [TILE]
    if (tid < TILE) place[tid] = e & (kChunkKeys - 1);
    __syncthreads();
    if (sum) atomicAdd(&place[tid & (TILE - 1)], sum);
    __syncthreads();
    if (tid < TILE && e < n) out.put(e, place[tid], key, chunk_pay[e], 0);
}

}  // namespace vspmm
