// Stable counting sort of ids into bins, over blocks: the sort behind the
// routing of tokens to experts (one pass, a bin per expert) and behind the
// embedding's gradient (tokens by id, one pass per digit). Two launches a
// pass: k_bin_count counts every tile's digits; k_bin_place has each block
// sum the counts of the tiles before its own (at most kBinBlocks of them, so
// no third launch scans them), then ranks its elements. Each wave owns a
// contiguous piece of the tile and counters of its own, so ranking needs no
// barrier between rounds: a round's 64 lanes rank equal digits by ballots,
// in lane order. Places depend only on the ids: the order is unique, equal to
// a sequential counting sort's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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
__host__ __device__ inline int bin_piece(int64_t n) {
    const int64_t per = (n + int64_t(kBinBlocks) * kBinWaves - 1) / (int64_t(kBinBlocks) * kBinWaves);
    const int64_t p = (per + 63) / 64 * 64;
    return int(p < kBinPiece ? kBinPiece : p);
}
__host__ __device__ inline int bin_blocks(int64_t n) {
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

// counts[b * bins + d] = elements of tile b whose digit is d.
template <typename I>
__global__ void __launch_bounds__(kBinThreads)
k_bin_count(const I *__restrict__ ids, int64_t n, int64_t limit, int shift, int bins, int piece,
            int *__restrict__ counts) {
    extern __shared__ int hist[];
    for (int d = threadIdx.x; d < bins; d += kBinThreads) hist[d] = 0;
    __syncthreads();
    const int64_t lo = int64_t(blockIdx.x) * piece * kBinWaves;
    const int64_t hi = lo + int64_t(piece) * kBinWaves < n ? lo + int64_t(piece) * kBinWaves : n;
    const uint32_t mask = shift < 0 ? ~0u : uint32_t(bins - 1);
    const int sh = shift < 0 ? 0 : shift;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kBinThreads)
        atomicAdd(&hist[(bin_key(ids, i, limit) >> sh) & mask], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kBinThreads)
        counts[int64_t(blockIdx.x) * bins + d] = hist[d];
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

// offsets (may be null): the first place of every bin, written by block 0.
template <typename I, typename Out>
__global__ void __launch_bounds__(kBinThreads)
k_bin_place(const I *__restrict__ ids, int64_t n, int64_t limit, int shift, int bins, int bits,
            int piece, const int *__restrict__ counts, Out out, int *__restrict__ offsets) {
    extern __shared__ int wc[];          // [kBinWaves][bins], then
    int *const sh = wc + kBinWaves * bins;  // [kBinWaves] for the scan
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = gridDim.x, blk = blockIdx.x;
    const uint32_t mask = shift < 0 ? ~0u : uint32_t(bins - 1);
    const int sft = shift < 0 ? 0 : shift;
    for (int d = tid; d < kBinWaves * bins; d += kBinThreads) wc[d] = 0;
    __syncthreads();
    const int64_t lo = (int64_t(blk) * kBinWaves + wave) * piece;
    const int64_t hi = lo + piece < n ? lo + piece : n;
    int *mine = wc + wave * bins;
    for (int64_t i = lo + lane; i < hi; i += 64)
        atomicAdd(&mine[(bin_key(ids, i, limit) >> sft) & mask], 1);
    __syncthreads();
    int carry = 0;  // elements of all lower digits
    for (int d0 = 0; d0 < bins; d0 += kBinThreads) {
        const int d = d0 + tid;
        int before = 0, total = 0;
        if (d < bins) {
#pragma unroll 8
            for (int b = 0; b < nb; ++b) {
                const int c = counts[int64_t(b) * bins + d];
                before += b < blk ? c : 0;
                total += c;
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
        const uint32_t key = live ? bin_key(ids, i, limit) : 0u;
        const int d = int((key >> sft) & mask);
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
            out.put(i, at + rank, key, limit);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

}  // namespace vspmm
