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

#include <type_traits>

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

// A finished sum or product rounded to the type written. The empty asm keeps the
// compiler from contracting the operation before it with a float16's conversion
// (v_fma_mixlo_f16), which it does in some instances and not in others: that adds
// +0 to a product, which takes a zero's sign, and rounds the exact result straight
// to float16, so that a halfway case would depend on the width.
template <typename T, typename A>
__device__ __forceinline__ T rounded(A x) {
    if constexpr (std::is_same_v<T, f16>) asm("" : "+v"(x));
    return T(x);
}

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

// Rows of any element type to zero, by the blocks of a launch past its own
// `first` ones: one 16-byte store a thread, consecutive threads consecutive
// chunks. 1.07 GB take 159 us so (6.8 TB/s), 181 with four stores a thread, 186
// with sixteen: the fewer bytes a wave holds, the narrower the window of
// addresses being written at a time.
struct ZeroRows {
    char *base = nullptr;
    int64_t ld = 0;          // bytes from row to row
    int64_t chunks = 0;      // 16-byte chunks of all rows, a row's last one maybe cut;
                             // of all bytes when no gap is left between rows
    int64_t bytes = 0;       // of a row, or of all rows; even
    uint32_t cpr = 0;        // chunks per row, 0 for no gaps
    FastDiv by_cpr{1};

    ZeroRows() = default;
    ZeroRows(void *p, int64_t ld_bytes, int64_t rows, int64_t row_bytes)
        : base(static_cast<char *>(p)), ld(ld_bytes) {
        if (rows <= 1 || ld_bytes == row_bytes) {
            bytes = rows * row_bytes;
            chunks = (bytes + 15) / 16;
        } else {
            bytes = row_bytes;
            cpr = uint32_t((row_bytes + 15) / 16);
            by_cpr = FastDiv(cpr);
            chunks = rows * cpr;
        }
    }
    // blocks of `threads` threads for it
    unsigned blocks(int threads) const {
        const int64_t n = (chunks + threads - 1) / threads;
        return unsigned(n < (1 << 21) ? n : 1 << 21);
    }
    __device__ __forceinline__ void run(unsigned first) const {
        const int64_t threads = int64_t(gridDim.x - first) * blockDim.x;
        for (int64_t c = int64_t(blockIdx.x - first) * blockDim.x + threadIdx.x; c < chunks;
             c += threads) {
            int64_t row = 0, chunk = c;
            if (cpr) {
                row = c < (int64_t(1) << 31) ? by_cpr.div(uint32_t(c)) : c / cpr;
                chunk = c - row * cpr;
            }
            char *p = base + row * ld + chunk * 16;
            const int64_t left = bytes - chunk * 16;
            if (left >= 16) {
                using Z = uint16_t __attribute__((ext_vector_type(8), aligned(2)));
                *reinterpret_cast<Z *>(p) = Z{};
            } else {
                for (int b = 0; b < left; b += 2) *reinterpret_cast<uint16_t *>(p + b) = 0;
            }
        }
    }
};

}  // namespace vspmm
