// Dense rows of 16-, 32- and 64-bit elements for the selection products: a
// row is cut into 16-byte chunks, a lane takes whole chunks, and arithmetic
// runs in float (double for double elements) with one rounding on the way
// out. Chunks are loaded at the element's own alignment (gfx950 serves
// unaligned global accesses of 16 bytes), so odd widths, row strides and
// offset views take the same path as aligned ones.
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

template <typename T>
using ChunkOf = T __attribute__((ext_vector_type(16 / sizeof(T))));
// the same, at the alignment of one element
template <typename T>
using LooseChunk = T __attribute__((ext_vector_type(16 / sizeof(T)), aligned(alignof(T))));

// N elements at p as one access, or the first `live` of them one by one (the
// rest zero): a row's last chunk may be cut by the row's end.
template <typename T>
__device__ __forceinline__ ChunkOf<T> load_chunk(const T *p, int live = kChunk<T>) {
    if (live >= kChunk<T>) return *reinterpret_cast<const LooseChunk<T> *>(p);
    ChunkOf<T> v{};
#pragma unroll
    for (int i = 0; i < kChunk<T>; ++i)
        if (i < live) v[i] = p[i];
    return v;
}

template <typename T>
__device__ __forceinline__ void store_chunk(T *p, ChunkOf<T> v, int live = kChunk<T>) {
    if (live >= kChunk<T>) {
        *reinterpret_cast<LooseChunk<T> *>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < kChunk<T>; ++i)
        if (i < live) p[i] = v[i];
}

// n / d for n < 2^31 by a multiplication: with l = ceil(log2 d) and m =
// floor(2^(31+l) / d) + 1, n m / 2^(31+l) exceeds n / d by less than 1 / d,
// so the floor is exact.
struct FastDiv {
    uint32_t m;
    int shift;
    FastDiv() = default;
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

}  // namespace vspmm
