// Dense rows of 16-, 32- and 64-bit elements for the selection products: a
// row is cut into 16-byte chunks, a lane takes whole chunks, and arithmetic
// runs in float (double for double elements) with one rounding on the way
// out. Chunks are loaded and stored at the element's own alignment (gfx950
// serves unaligned global accesses of 16 bytes), so odd widths, row strides
// and offset views take the same path as aligned ones. A row whose width is no
// multiple of the chunk ends in a chunk moved left to end with the row: its
// first elements are the chunk before's last ones, computed and written twice
// with the same value. Rows shorter than a chunk go element by element (C = 1).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vspmm {

using bf16 = __bf16;
using f16 = _Float16;

template <typename T>
struct Sum {
    using type = float;
};
template <>
struct Sum<double> {
    using type = double;
};

template <typename T>
constexpr int kChunk = int(16 / sizeof(T));  // elements per 16-byte chunk

// C elements at the alignment of one.
template <typename T, int C>
using Vec = T __attribute__((ext_vector_type(C), aligned(alignof(T))));

template <int C, typename T>
__device__ __forceinline__ Vec<T, C> load_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, C> *>(p);
}
template <int C, typename T>
__device__ __forceinline__ void store_vec(T *p, Vec<T, C> v) {
    *reinterpret_cast<Vec<T, C> *>(p) = v;
}

// The same past the caches' replacement order, for streams read or written once.
template <int C, typename T>
__device__ __forceinline__ Vec<T, C> load_once(const T *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const Vec<T, C> *>(p));
}
template <int C, typename T>
__device__ __forceinline__ void store_once(T *p, Vec<T, C> v) {
    __builtin_nontemporal_store(v, reinterpret_cast<Vec<T, C> *>(p));
}

template <bool ONCE, int C, typename T>
__device__ __forceinline__ Vec<T, C> load_as(const T *p) {
    if constexpr (ONCE) return load_once<C>(p);
    else return load_vec<C>(p);
}

// Chunk c of a row starts at element c * C, moved left where the row's end
// cuts it (width >= C).
template <int C>
__device__ __forceinline__ uint32_t chunk_col(uint32_t c, uint32_t width) {
    const uint32_t col = c * C;
    return col + C <= width ? col : width - C;
}

// n / d for n < 2^31 by a multiplication: with l = ceil(log2 d) and m =
// floor(2^(31+l) / d) + 1, n m / 2^(31+l) exceeds n / d by less than 1 / d,
// so the floor is exact.
struct FastDiv {
    uint32_t m;
    int shift;
    explicit FastDiv(uint32_t d) {
        int l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        shift = 31 + l;
        m = uint32_t((uint64_t(1) << shift) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return uint32_t((uint64_t(n) * m) >> shift);
    }
};

// The zeroing of rows of any element type. Rows that nothing else writes go in
// units of `unit_rows` rows, one wave each, which skip the rows they are told
// to keep; whole ranges go as flat memory when the rows leave no gap.
constexpr int kZeroRows = 64;            // most rows of a unit
constexpr int kZeroWaveBytes = 1 << 14;  // about what one wave of a launch zeroes

struct ZeroRows {
    char *base = nullptr;
    int64_t ld = 0;          // bytes from row to row
    int64_t n_rows = 0;
    uint32_t row_bytes = 0;  // even
    uint32_t cpr = 0;        // 16-byte chunks per row, the last one maybe cut
    FastDiv by_cpr{1};
    int unit_rows = 1;       // a power of two
    bool once = false;       // nontemporal stores

    ZeroRows() = default;
    ZeroRows(void *p, int64_t ld_bytes, int64_t rows, int64_t bytes, bool nontemporal)
        : base(static_cast<char *>(p)), ld(rows > 1 ? ld_bytes : bytes), n_rows(rows),
          row_bytes(uint32_t(bytes)), cpr(uint32_t((bytes + 15) / 16)), by_cpr(cpr), once(nontemporal) {
        while (unit_rows < kZeroRows && 2 * unit_rows * bytes <= kZeroWaveBytes) unit_rows *= 2;
    }
    __host__ __device__ int64_t units() const { return (n_rows + unit_rows - 1) / unit_rows; }

    template <bool ONCE>
    __device__ __forceinline__ static void chunk(char *p, int64_t left) {
        if (left >= 16) {
            using Z = uint16_t __attribute__((ext_vector_type(8), aligned(2)));
            if (ONCE) __builtin_nontemporal_store(Z{}, reinterpret_cast<Z *>(p));
            else *reinterpret_cast<Z *>(p) = Z{};
        } else {
            for (int b = 0; b < left; b += 2) *reinterpret_cast<uint16_t *>(p + b) = 0;
        }
    }
    // Zeroes the rows of unit u whose bit in `keep` is 0.
    template <bool ONCE>
    __device__ __forceinline__ void unit(int64_t u, uint64_t keep) const {
        const int lane = threadIdx.x & 63;
        const int64_t r0 = u * unit_rows;
        const int rows = int(n_rows - r0 < unit_rows ? n_rows - r0 : unit_rows);
        if (cpr >= 64) {  // a row at a time
            for (int r = 0; r < rows; ++r) {
                if ((keep >> r) & 1) continue;
                char *p = base + (r0 + r) * ld;
#pragma unroll 4
                for (uint32_t at = lane * 16; at < row_bytes; at += 1024)
                    chunk<ONCE>(p + at, int64_t(row_bytes) - at);
            }
            return;
        }
        for (uint32_t c = lane; c < uint32_t(rows) * cpr; c += 64) {
            const uint32_t r = by_cpr.div(c), at = (c - r * cpr) * 16;
            if (!((keep >> r) & 1)) chunk<ONCE>(base + (r0 + r) * ld + at, int64_t(row_bytes) - at);
        }
    }
    // Zeroes all rows of units [lo, hi) by `waves` waves, of which this is
    // number `wave`.
    template <bool ONCE>
    __device__ __forceinline__ void range(int64_t lo, int64_t hi, int64_t wave, int64_t waves) const {
        if (ld != row_bytes) {
            for (int64_t u = lo + wave; u < hi; u += waves) unit<ONCE>(u, 0);
            return;
        }
        const int64_t r1 = hi * unit_rows < n_rows ? hi * unit_rows : n_rows;
        char *p = base + lo * unit_rows * ld;
        const int64_t bytes = (r1 - lo * unit_rows) * ld;
        for (int64_t at = wave * 4096 + (threadIdx.x & 63) * 16; at < bytes; at += waves * 4096) {
#pragma unroll
            for (int k = 0; k < 4; ++k) chunk<ONCE>(p + at + k * 1024, bytes - at - k * 1024);
        }
    }
    __device__ __forceinline__ void range(int64_t lo, int64_t hi, int64_t wave, int64_t waves) const {
        if (once) range<true>(lo, hi, wave, waves);
        else range<false>(lo, hi, wave, waves);
    }
};

// A share of the zeroing that a launch of another kernel carries: its blocks
// past its own work zero units [lo, hi).
struct ZeroShare {
    ZeroRows rows;
    int64_t lo = 0, hi = 0;
    // blocks of `waves` waves for it
    unsigned blocks(int waves) const {
        const int64_t bytes = (hi - lo) * rows.unit_rows * int64_t(rows.row_bytes);
        const int64_t per = int64_t(waves) * kZeroWaveBytes;
        const int64_t n = (bytes + per - 1) / per;
        return unsigned(n < (1 << 20) ? n : 1 << 20);
    }
};

}  // namespace vspmm
