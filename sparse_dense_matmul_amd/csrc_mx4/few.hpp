// Products with few tokens: one wave takes 16 rows of each of R matrices and 16 MT tokens over a range of the
// contraction, the rows as the first operand of the 16 x 16 matrix instructions and the tokens as the second, so that
// weights go from memory to registers once and are bound by memory, whatever the number of tokens.
//
// A chunk is 128 values of the contraction, four instructions. Lane (r, g) = (lane % 16, lane / 16) holds row r (token
// r) at 32 values of the chunk. Which ones is free as long as both operands agree: for 4-bit rows it is block g, 16
// bytes under one scale; for 16-bit rows instruction j takes 8 values at 32 j + 8 g, so that the four lanes of a row
// read 64 bytes in a row. A result's lane (t, q) holds rows 4 q .. 4 q + 3 for token t.
#pragma once

#include "mx4.hpp"

namespace vspmm {

constexpr int kChunkK = 128;

template <typename T>
struct Row {  // 16-bit values
    const T *p;
};
template <>
struct Row<Mx4> {
    const uint8_t *codes, *scales;
};
template <>
struct Row<Planes> {
    const bf16 *hi, *lo;
    bool live;  // a row that is not counts as zeros and is not read
};

template <typename T>
struct Piece {  // a lane's part of a chunk
    i32x4 v[4];
};
template <>
struct Piece<Mx4> {
    i32x4 codes;
    uint32_t scale;
};
template <>
struct Piece<Planes> {
    i32x4 hi[4], lo[4];
};

// A lane's 8 values of 16 bits at p, those from the width on as zeros.
template <typename T>
__device__ __forceinline__ i32x4 load_half(const T *p, int k, int width) {
    if (k + 8 <= width) return *reinterpret_cast<const Half16 *>(p + k);
    i32x4 v{};
    if (k >= width) return v;
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t e = k + i < width ? h[k + i] : 0;
        v[i / 2] |= int32_t(e << (16 * (i & 1)));
    }
    return v;
}

// WHOLE: the chunk at k lies within the width. BY_BLOCKS: the lanes' values go by blocks of 32.
template <bool WHOLE, bool BY_BLOCKS, typename T>
__device__ __forceinline__ void load_piece(Piece<T> &out, const Row<T> &row, int k, int width, int g) {
    if constexpr (std::is_same_v<T, Mx4>) {
        const int b = k / kBlock + g;
        if (WHOLE || b * kBlock < width) {
            out.codes = *reinterpret_cast<const Byte16 *>(row.codes + int64_t(b) * kBlockBytes);
            out.scale = row.scales[b];
        } else {
            out.codes = i32x4{};
            out.scale = 127;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = k + (BY_BLOCKS ? 32 * g + 8 * j : 32 * j + 8 * g);
            if constexpr (std::is_same_v<T, Planes>) {
                if (!row.live) {
                    out.hi[j] = out.lo[j] = i32x4{};
                } else if (WHOLE) {
                    out.hi[j] = *reinterpret_cast<const Half16 *>(row.hi + at);
                    out.lo[j] = *reinterpret_cast<const Half16 *>(row.lo + at);
                } else {
                    out.hi[j] = load_half(row.hi, at, width);
                    out.lo[j] = load_half(row.lo, at, width);
                }
            } else {
                if (WHOLE) out.v[j] = *reinterpret_cast<const Half16 *>(row.p + at);
                else out.v[j] = load_half(row.p, at, width);
            }
        }
    }
}

// One tile of 16 tokens, number m of the sums. Conversions of the weights that another tile repeats are the same
// expressions, made once.
template <typename W, typename X, int R, int MT>
__device__ __forceinline__ void multiply(f32x4 (&acc)[R][MT], int m, const Piece<W> (&w)[R], const Piece<X> &x) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
        f32x4 &a = acc[i][m];
        if constexpr (std::is_same_v<X, Mx4>) {
            a = mma16_mx4<0>(w[i].codes, w[i].scale, x.codes, x.scale, a);
        } else if constexpr (std::is_same_v<W, Mx4>) {
            const float s = scale_operand(w[i].scale);
            if constexpr (std::is_same_v<X, f16>) {
                // float16 tokens meet the weights in float16 where it holds them exactly, which it does for all but
                // far scales; else in two bfloat16 parts
                const i32x4 c = w[i].codes;
                const bool none = (c[0] | c[1] | c[2] | c[3]) == 0 && w[i].scale != 255;
                if (__all(f16_scale(w[i].scale) || none)) {
                    const float s16 = none ? 1.0f : s;
#pragma unroll
                    for (int j = 0; j < 4; ++j) a = mma16<f16>(widen<f16>(uint32_t(c[j]), s16), x.v[j], a);
                    continue;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const i32x4 v = widen<bf16>(uint32_t(w[i].codes[j]), s);
                if constexpr (std::is_same_v<X, bf16>) {
                    a = mma16<bf16>(v, x.v[j], a);
                } else {
                    i32x4 hi, lo;
                    if constexpr (std::is_same_v<X, Planes>) hi = x.hi[j], lo = x.lo[j];
                    else split(x.v[j], hi, lo);
                    a = mma16<bf16>(v, hi, a);
                    a = mma16<bf16>(v, lo, a);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (!std::is_same_v<X, Planes>) {
                    a = mma16<W>(w[i].v[j], x.v[j], a);
                } else if constexpr (std::is_same_v<W, bf16>) {
                    a = mma16<bf16>(w[i].v[j], x.hi[j], a);
                    a = mma16<bf16>(w[i].v[j], x.lo[j], a);
                } else {
                    i32x4 hi, lo;
                    split(w[i].v[j], hi, lo);
                    a = mma16<bf16>(hi, x.hi[j], a);
                    a = mma16<bf16>(hi, x.lo[j], a);
                    // the product of both second parts lies 2^-16 and less under that of the first
                    a = mma16<bf16>(lo, x.hi[j], a);
                }
            }
        }
    }
}

// acc += rows times tokens over the chunks [c0, c1) of a contraction of `width` values. tiles: a bit for each tile of
// 16 tokens that counts; the others are neither read nor multiplied.
template <int U, typename W, typename X, int R, int MT>
__device__ __forceinline__ void accumulate(f32x4 (&acc)[R][MT], const Row<W> (&rows)[R], const Row<X> (&x)[MT], int c0,
                                           int c1, int width, int g, uint32_t tiles) {
    constexpr bool BY_BLOCKS = std::is_same_v<W, Mx4>;
    const int whole = width / kChunkK < c1 ? width / kChunkK : c1;
    // tokens that fill more registers than this are loaded tile by tile beside the products
    constexpr bool AT_ONCE = U * MT * sizeof(Piece<X>) <= 64 * 4;
    int c = c0;
    for (; c + U <= whole; c += U) {
        Piece<W> w[U][R];
        Piece<X> t[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < R; ++i) load_piece<true, BY_BLOCKS>(w[u][i], rows[i], (c + u) * kChunkK, width, g);
            if constexpr (AT_ONCE) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    if (tiles >> m & 1) load_piece<true, BY_BLOCKS>(t[u][m], x[m], (c + u) * kChunkK, width, g);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (!(tiles >> m & 1)) continue;
                if constexpr (!AT_ONCE) load_piece<true, BY_BLOCKS>(t[u][m], x[m], (c + u) * kChunkK, width, g);
                multiply<W, X>(acc, m, w[u], t[u][m]);
            }
    }
    for (; c < c1; ++c) {
        Piece<W> w[R];
#pragma unroll
        for (int i = 0; i < R; ++i) load_piece<false, BY_BLOCKS>(w[i], rows[i], c * kChunkK, width, g);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (!(tiles >> m & 1)) continue;
            Piece<X> t;
            load_piece<false, BY_BLOCKS>(t, x[m], c * kChunkK, width, g);
            multiply<W, X>(acc, m, w, t);
        }
    }
}

}  // namespace vspmm
