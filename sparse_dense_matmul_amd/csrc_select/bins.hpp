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
//    in lane order. A list of one tile needs no k_bin_count.
//  - k_rank: every element's place counted directly, one launch.
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
// within kBinBlocks.
inline int bin_piece(int64_t n) {
    const int64_t per = (n + int64_t(kBinBlocks) * kBinWaves - 1) / (int64_t(kBinBlocks) * kBinWaves);
    const int64_t p = (per + 63) / 64 * 64;
    return int(p < kBinPiece ? kBinPiece : p);
}
inline int bin_blocks(int64_t n) {
    const int64_t tile = int64_t(bin_piece(n)) * kBinWaves;
    return int((n + tile - 1) / tile);
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
// tiles zero their share of rows; *clear (may be null) = 0.
template <typename I>
__global__ void __launch_bounds__(kBinThreads)
k_bin_count(BinPass<I> ps, int *__restrict__ counts, int *clear, ZeroShare zero) {
    extern __shared__ int hist[];
    if (int(blockIdx.x) >= ps.nb) {
        zero.rows.range(zero.lo, zero.hi, int64_t(blockIdx.x - ps.nb) * kBinWaves + threadIdx.x / 64,
                        int64_t(gridDim.x - ps.nb) * kBinWaves);
        return;
    }
    if (clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
    for (int d = threadIdx.x; d < ps.bins; d += kBinThreads) hist[d] = 0;
    __syncthreads();
    const int64_t tile = int64_t(ps.piece) * kBinWaves, lo = blockIdx.x * tile;
    const int64_t hi = lo + tile < ps.n ? lo + tile : ps.n;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kBinThreads)
        atomicAdd(&hist[ps.digit(bin_key(ps.ids, i, ps.limit))], 1);
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

// Where a pass puts element i of place p.
struct PlaceRoute {  // order[p] = i, position[i] = p, or ~p for a dropped slot
    int *order, *position;
    __device__ __forceinline__ void put(int64_t i, int p, uint32_t key, int64_t limit) const {
        order[p] = int(i);
        position[i] = key == uint32_t(limit) ? ~p : p;
    }
};
struct PlaceKeys {  // keys[p] = key, pay[p] = from ? from[i] : i
    uint32_t *keys;
    int *pay;
    const int *from;
    __device__ __forceinline__ void put(int64_t i, int p, uint32_t key, int64_t) const {
        keys[p] = key;
        pay[p] = from ? from[i] : int(i);
    }
};

// `bits` bits hold a digit. offsets (may be null): the first place of every
// bin, written by block 0. counts is not read when there is one tile.
template <typename I, typename Out>
__global__ void __launch_bounds__(kBinThreads)
k_bin_place(BinPass<I> ps, int bits, const int *__restrict__ counts, Out out,
            int *__restrict__ offsets, ZeroShare zero) {
    extern __shared__ int wc[];             // [kBinWaves][bins], then
    int *const sh = wc + kBinWaves * ps.bins;  // [kBinWaves] for the scan
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = ps.nb, blk = blockIdx.x, bins = ps.bins;
    if (blk >= nb) {
        zero.rows.range(zero.lo, zero.hi, int64_t(blk - nb) * kBinWaves + wave,
                        int64_t(gridDim.x - nb) * kBinWaves);
        return;
    }
    for (int d = tid; d < kBinWaves * bins; d += kBinThreads) wc[d] = 0;
    __syncthreads();
    const int64_t lo = (int64_t(blk) * kBinWaves + wave) * ps.piece;
    const int64_t hi = lo + ps.piece < ps.n ? lo + ps.piece : ps.n;
    int *mine = wc + wave * bins;
    for (int64_t i = lo + lane; i < hi; i += 64)
        atomicAdd(&mine[ps.digit(bin_key(ps.ids, i, ps.limit))], 1);
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
#pragma unroll 8
                for (int b = 0; b < nb; ++b) {
                    const int c = counts[int64_t(b) * bins + d];
                    before += b < blk ? c : 0;
                    total += c;
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
    for (int64_t i0 = lo; i0 < hi; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool live = i < hi;
        const uint32_t key = live ? bin_key(ps.ids, i, ps.limit) : 0u;
        const int d = ps.digit(key);
        uint64_t same = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (d >> b) & 1;
            const uint64_t with = __ballot(bit);
            same &= bit ? with : ~with;
        }
        const int rank = __popcll(same & lt);
        if (live) {
            const int at = next[d];
            if (rank == 0) next[d] = at + __popcll(same);
            out.put(i, at + rank, key, ps.limit);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Every element's place, counted directly: the keys below its own, and the
// equal ones before it. A block holds all keys in LDS and places kRankTile
// elements, a lane each, both halves of every wave on the same elements; the
// 32 half waves count a piece of the keys each. Two integer operations per
// pair: n^2 pairs over the card's 16,384 lanes take n^2 / 8,192 cycles, 3.4 us
// for the most elements it is used at (8,192).
constexpr int kRankThreads = 1024;
constexpr int kRankTile = 32;
constexpr int kRankMax = 8192;

template <typename I>
__global__ void __launch_bounds__(kRankThreads)
k_rank(const I *__restrict__ ids, int n, int64_t limit, int n_blocks, PlaceKeys out, int *clear,
       ZeroShare zero) {
    __shared__ __align__(16) uint32_t keys[kRankMax];
    __shared__ int place[kRankTile];
    const int tid = threadIdx.x;
    if (int(blockIdx.x) >= n_blocks) {
        zero.rows.range(zero.lo, zero.hi,
                        int64_t(blockIdx.x - n_blocks) * (kRankThreads / 64) + tid / 64,
                        int64_t(gridDim.x - n_blocks) * (kRankThreads / 64));
        return;
    }
    if (clear && blockIdx.x == 0 && tid == 0) *clear = 0;
    // padded with keys above every other, so the counting reads whole vectors
    const int padded = (n + 127) & ~127;
    for (int i = tid; i < padded; i += kRankThreads)
        keys[i] = i < n ? bin_key(ids, i, limit) : ~0u;
    if (tid < kRankTile) place[tid] = 0;
    __syncthreads();
    const int first = blockIdx.x * kRankTile;      // a multiple of 4
    const int i = first + (tid & (kRankTile - 1));
    const uint32_t key = i < n ? keys[i] : ~0u;
    // this half wave's keys: quads q, q + 32, ... of four keys
    const int half = tid / kRankTile;
    int below = 0;
    for (int q = half; q < padded / 4; q += kRankThreads / kRankTile) {
        const uint4 k = *reinterpret_cast<const uint4 *>(&keys[4 * q]);
        if (4 * q >= first && 4 * q < first + kRankTile) {  // the tile's own elements
            below += k.x < key + (4 * q + 0 < i) ? 1 : 0;
            below += k.y < key + (4 * q + 1 < i) ? 1 : 0;
            below += k.z < key + (4 * q + 2 < i) ? 1 : 0;
            below += k.w < key + (4 * q + 3 < i) ? 1 : 0;
        } else {
            const uint32_t bound = key + (4 * q < first ? 1u : 0u);
            below += (k.x < bound) + (k.y < bound) + (k.z < bound) + (k.w < bound);
        }
    }
    if (below) atomicAdd(&place[tid & (kRankTile - 1)], below);
    __syncthreads();
    if (tid < kRankTile && i < n) out.put(i, place[tid], key, limit);
}

}  // namespace vspmm
