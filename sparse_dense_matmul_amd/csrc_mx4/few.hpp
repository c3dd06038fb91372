// Products with few tokens: one wave takes 16 rows of each of R matrices and 16 MT tokens over a range of the
// contraction, the rows as the first operand of the 16 x 16 matrix instructions and the tokens as the second. Weights
// go from memory to registers once; what bounds such a product is their bytes, whatever the number of tokens.
//
// A chunk is 128 values of the contraction, four instructions. Lane (r, g) = (lane % 16, lane / 16) holds row r (token
// r); instruction j takes its 8 values at 32 j + 8 g, so that the four lanes of a row read 64 bytes in a row. 4-bit
// rows are read as one block a lane, 16 bytes, and four exchanges between lanes turn block g into a part of every
// block: with a block a lane instead, the tokens would come in pieces of 16 bytes 64 apart, twice as many cache lines
// an instruction (which took an earlier form from 17 to 30 us at 37 tokens and 5,003 x 4,001).
// A result's lane (t, q) holds rows 4 q .. 4 q + 3 for token t. One bfloat16 token through 4,096 x 4,096: 4.9 us, 1.3 us
// of bytes, bound by the latency of one round of loads and the sum over the waves.
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
struct Row<Planes> {  // whole chunks: zeros past the width
    const bf16 *p;
    bool live;  // whether the lane's token counts: where not, chunks need not be loaded
};
// Where eight values at k lie in such a row: 3 x 8 bfloat16 numbers in a row, so that one address serves all three (64
// tokens to 8 of 128 experts in 676 us, 682 with the parts in three rows, in 4 bits 410 and 420).
__host__ __device__ constexpr int64_t at_planes(int64_t k) { return 3 * k; }

template <typename T>
struct Staged {};  // rows of T that lie in LDS, whole chunks with zeros at the end
template <typename T>
using LdsPtr = const __attribute__((address_space(3))) T *;
template <typename T>
struct Row<Staged<T>> {
    LdsPtr<T> p;
};
template <>
struct Row<Staged<Planes>> {
    LdsPtr<bf16> p;
};
template <typename X>
struct Plain {  // what a row's values are, wherever they lie
    using type = X;
    static constexpr bool staged = false;
};
template <typename T>
struct Plain<Staged<T>> {
    using type = T;
    static constexpr bool staged = true;
};

template <typename T>
struct Piece {  // a lane's part of a chunk
    i32x4 v[4];
};
template <>
struct Piece<Mx4> {
    i32x4 codes;
    uint32_t scale;  // of block g; as a matrix of 16-bit tokens, of the four blocks
};
template <>
struct Piece<Planes> {
    i32x4 hi[4], mid[4], lo[4];
};

// Eight 16-bit values at k of a row, those from the width on as zeros: loaded where the row still has eight and moved.
__device__ __forceinline__ i32x4 load_half(const uint16_t *p, int k, int width) {
    using Wide = unsigned __int128;
    if (width < 8) {
        i32x4 v{};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t e = p[min(i, width - 1)];
            v[i / 2] |= int32_t((k + i < width ? e : 0) << (16 * (i & 1)));
        }
        return v;
    }
    const int at = min(k, width - 8);
    const Wide v = bits_as<Wide>(i32x4(*reinterpret_cast<const Half16 *>(p + at)));
    return bits_as<i32x4>(k - at < 8 ? v >> (16 * (k - at)) : Wide(0));
}

// A whole chunk of a row or token. BOTH: both sides are of 4 bits.
template <bool BOTH, typename T>
__device__ __forceinline__ void load_piece(Piece<T> &out, const Row<T> &row, int k, int g) {
    if constexpr (std::is_same_v<T, Mx4>) {
        const int b = k / kBlock;
        out.codes = *reinterpret_cast<const Byte16 *>(row.codes + int64_t(b + g) * kBlockBytes);
        if constexpr (BOTH) out.scale = row.scales[b + g];
        else out.scale = *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(row.scales + b);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = k + 32 * j + 8 * g;
            if constexpr (std::is_same_v<T, Planes>) {
                const i32x4 *p = reinterpret_cast<const i32x4 *>(row.p + at_planes(at));
                out.hi[j] = p[0], out.mid[j] = p[1], out.lo[j] = p[2];
            } else {
                out.v[j] = *reinterpret_cast<const Half16 *>(row.p + at);
            }
        }
    }
}

// A lane's 8 values of a token for one instruction.
template <typename T>
struct Step {
    i32x4 hi, mid, lo;  // 16-bit tokens: hi alone
};

template <bool WHOLE, typename T>
__device__ __forceinline__ Step<T> load_step(const Row<T> &row, int k, int width) {
    Step<T> s;
    if constexpr (std::is_same_v<T, Staged<Planes>>) {
        const auto p = reinterpret_cast<LdsPtr<i32x4>>(row.p + int(at_planes(k)));
        s = {p[0], p[1], p[2]};
    } else if constexpr (Plain<T>::staged) {
        s.hi = *reinterpret_cast<LdsPtr<i32x4>>(row.p + k);
    } else if constexpr (std::is_same_v<T, Planes>) {
        const i32x4 *p = reinterpret_cast<const i32x4 *>(row.p + at_planes(k));
        s = {p[0], p[1], p[2]};
    } else if (WHOLE) {
        s.hi = *reinterpret_cast<const Half16 *>(row.p + k);
    } else {
        s.hi = load_half(reinterpret_cast<const uint16_t *>(row.p), k, width);
    }
    return s;
}

// Word w of lane g becomes word g of lane w.
__device__ __forceinline__ i32x4 exchange(i32x4 v) {
    using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
    const u32x2 a = __builtin_amdgcn_permlane32_swap(uint32_t(v[0]), uint32_t(v[2]), false, false);
    const u32x2 b = __builtin_amdgcn_permlane32_swap(uint32_t(v[1]), uint32_t(v[3]), false, false);
    const u32x2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const u32x2 d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return i32x4{int32_t(c[0]), int32_t(c[1]), int32_t(d[0]), int32_t(d[1])};
}

__device__ __forceinline__ float scale_operand_of(uint32_t scales, int j) {
    return scale_operand(scales >> (8 * j) & 255);
}

// One instruction's worth of a matrix's rows, a (of type T: its own, or what its codes were widened to), and a token
// tile: as many instructions as the two have parts. CAREFUL: a factor in parts may meet infinities.
template <typename T, bool CAREFUL, typename X>
__device__ __forceinline__ f32x4 multiply_step(i32x4 a, const Step<X> &x, f32x4 c) {
    using V = typename Plain<X>::type;
    if constexpr (std::is_same_v<V, T>) {
        return mma16<T>(a, x.hi, c);
    } else if constexpr (std::is_same_v<V, Planes>) {
        i32x4 hi = a, lo;
        if constexpr (std::is_same_v<T, f16>) split(a, hi, lo);
        c = mma16<bf16>(hi, x.hi, c);
        if constexpr (CAREFUL) hi = finite(hi);
        c = mma16<bf16>(hi, x.mid, c);
        c = mma16<bf16>(hi, x.lo, c);
        if constexpr (std::is_same_v<T, f16>) {
            c = mma16<bf16>(lo, CAREFUL ? finite(x.hi) : x.hi, c);
            c = mma16<bf16>(lo, x.mid, c);
            c = mma16<bf16>(lo, x.lo, c);
        }
        return c;
    } else {  // float16 tokens, bfloat16 rows
        i32x4 hi, lo;
        split(x.hi, hi, lo);
        c = mma16<bf16>(a, hi, c);
        asm volatile("" : "+v"(a));  // found anew for each tile of tokens, not kept in registers between
        return mma16<bf16>(finite(a), lo, c);
    }
}

// Whether a wave's chunk of a matrix may meet its tokens in float16: each lane answers for the block it loaded.
__device__ __forceinline__ bool f16_holds(const Piece<Mx4> &w, int g) {
    const uint32_t b = w.scale >> (8 * g) & 255;
    return __all(f16_scale(b) || f16_zeros(b, w.codes));
}

// acc += rows times tokens over the chunks [c0, c1) of a contraction of `width` values, U at a time. One tile's tokens are
// loaded by chunks; those of several, which would need more registers than there are, and those in LDS beside the
// products. CAREFUL: see multiply_step; all of the range goes by blocks of 32, in few registers.
template <int U, bool CAREFUL = false, typename W, typename X, int R, int MT>
__device__ __forceinline__ void accumulate(f32x4 (&acc)[R][MT], const Row<W> (&rows)[R], const Row<X> (&x)[MT], int c0,
                                           int c1, int width, int g) {
    constexpr bool BOTH = std::is_same_v<X, Mx4>, CODES = std::is_same_v<W, Mx4>;
    constexpr bool BY_CHUNKS = BOTH || (MT == 1 && !Plain<X>::staged);
    using V = typename Plain<X>::type;
    const int whole = CAREFUL ? c0 : min(width / kChunkK, c1);
    int c = c0;
    // N chunks: all are on their way before the first is waited for, as far as the compiler leaves it so
    auto load_rows = [&](auto &w, int at) {
#pragma unroll
        for (auto &u : w) {
#pragma unroll
            for (int i = 0; i < R; ++i) load_piece<BOTH>(u[i], rows[i], at * kChunkK, g);
            ++at;
        }
    };
    auto load_tokens = [&](auto &t, int at) {
        if constexpr (BY_CHUNKS && std::is_same_v<X, Planes>) {
            // A lane without a token loads nothing and leaves its registers as they are: a column of the product depends
            // on its own token alone. (64 tokens to 8 of 128 experts, four a tile: the layer in 676 us, 776 with all lanes'
            // loads, in float16 685 and 834.)
#pragma unroll
            for (auto &u : t)
#pragma unroll
                for (int j = 0; j < 4; ++j) asm("" : "=v"(u[0].hi[j]), "=v"(u[0].mid[j]), "=v"(u[0].lo[j]));
            if (x[0].live) {
#pragma unroll
                for (auto &u : t) load_piece<BOTH>(u[0], x[0], at++ * kChunkK, g);
            }
        } else if constexpr (BY_CHUNKS) {
#pragma unroll
            for (auto &u : t) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    load_piece<BOTH>(u[m], x[m], at * kChunkK, g);
                ++at;
            }
        }
    };
    auto multiply = [&](const Piece<W> (&w)[R], const Piece<V> (&t)[BY_CHUNKS ? MT : 1], int at) {
        if constexpr (BOTH) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    acc[i][m] = mma16_mx4<0>(w[i].codes, w[i].scale, t[m].codes, t[m].scale, acc[i][m]);
        } else {
            i32x4 codes[R];
            if constexpr (CODES) {
#pragma unroll
                for (int i = 0; i < R; ++i) codes[i] = exchange(w[i].codes);
            }
            auto chunk = [&](auto type) {
                using T = decltype(type);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    i32x4 a[R];
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        if constexpr (CODES) a[i] = widen<T>(uint32_t(codes[i][j]), scale_operand_of(w[i].scale, j));
                        else a[i] = w[i].v[j];
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        Step<X> s;
                        if constexpr (!BY_CHUNKS) s = load_step<true>(x[m], at * kChunkK + 32 * j + 8 * g, width);
                        else if constexpr (std::is_same_v<V, Planes>) s = {t[m].hi[j], t[m].mid[j], t[m].lo[j]};
                        else s.hi = t[m].v[j];
#pragma unroll
                        for (int i = 0; i < R; ++i) acc[i][m] = multiply_step<T, CAREFUL>(a[i], s, acc[i][m]);
                    }
                }
            };
            if constexpr (!CODES) {
                chunk(W{});
            } else if constexpr (std::is_same_v<V, f16>) {
                // float16 tokens meet the weights in float16 where it holds them exactly, which it does for all but far
                // scales; else in two bfloat16 parts
                bool exact = true;
#pragma unroll
                for (int i = 0; i < R; ++i) exact = exact && f16_holds(w[i], g);
                if (exact) chunk(f16{});
                else chunk(bf16{});
            } else {
                chunk(bf16{});
            }
        }
    };
    auto some = [&](auto count) {
        constexpr int N = decltype(count)::value;
        Piece<W> w[N][R];
        Piece<V> t[N][BY_CHUNKS ? MT : 1];
        load_rows(w, c);
        load_tokens(t, c);
#pragma unroll
        for (int u = 0; u < N; ++u) multiply(w[u], t[u], c + u);
        c += N;
    };
    if constexpr (!CAREFUL) {
        while (c + U <= whole) some(std::integral_constant<int, U>{});
        if constexpr (U > 2)
            if (c + 2 <= whole) some(std::integral_constant<int, 2>{});
        if constexpr (U > 1)
            if (c < whole) some(std::integral_constant<int, 1>{});
    }
    if (c >= c1) {
        settle(acc);
        return;
    }
    // the last chunk, in parts: what lies past the width is zeros on both sides
    if constexpr (BOTH) {
        const int b = c * (kChunkK / kBlock) + g;
        const bool here = b * kBlock < width;
        auto part = [&](const Row<Mx4> &row) {
            Piece<Mx4> p{i32x4{}, 127};
            if (here) {
                p.codes = *reinterpret_cast<const Byte16 *>(row.codes + int64_t(b) * kBlockBytes);
                p.scale = row.scales[b];
            }
            return p;
        };
        Piece<Mx4> w[R];
#pragma unroll
        for (int i = 0; i < R; ++i) w[i] = part(rows[i]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const Piece<Mx4> t = part(x[m]);
#pragma unroll
            for (int i = 0; i < R; ++i) acc[i][m] = mma16_mx4<0>(w[i].codes, w[i].scale, t.codes, t.scale, acc[i][m]);
        }
    } else {
        // blocks of 32 one after another, or, where registers allow, two or all loaded first; those past the end are zeros
        constexpr int N = CAREFUL || MT > 1 ? 1 : CODES ? kChunkK / kBlock : 2;
        const int end = CAREFUL ? min(width, c1 * kChunkK) : width;
#pragma unroll 1
        for (int k0 = c * kChunkK; k0 < end; k0 += N * kBlock) {
            i32x4 a[N][R];
            uint32_t word[N][R], top[N][R];
            Step<X> s[N][MT];
            bool exact = true;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int k = k0 + n * kBlock;
                const bool here = k < width;
                const int at = here ? k : k0;  // a block that is there: its values are not used
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if constexpr (CODES) {
                        const uint8_t *p = rows[i].codes + int64_t(at / kBlock) * kBlockBytes + 4 * g;
                        word[n][i] = *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(p);
                        top[n][i] = rows[i].scales[at / kBlock];
                    } else {
                        a[n][i] = load_half(reinterpret_cast<const uint16_t *>(rows[i].p), k + 8 * g, width);
                    }
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    s[n][m] = load_step<false>(x[m], (Plain<X>::staged || std::is_same_v<V, Planes> ? at : k) + 8 * g,
                                               width);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const bool here = k0 + n * kBlock < width;
                if constexpr (CODES) {
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        word[n][i] = here ? word[n][i] : 0;
                        top[n][i] = here ? top[n][i] : 127;
                        if constexpr (std::is_same_v<V, f16>)
                            exact = exact && (f16_scale(top[n][i]) || f16_zeros(top[n][i], word[n][i]));
                    }
                }
                if constexpr (Plain<X>::staged || std::is_same_v<V, Planes>) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[n][m].hi[e] = here ? s[n][m].hi[e] : 0;
                            if constexpr (std::is_same_v<V, Planes>) {
                                s[n][m].mid[e] = here ? s[n][m].mid[e] : 0;
                                s[n][m].lo[e] = here ? s[n][m].lo[e] : 0;
                            }
                        }
                }
            }
            auto part = [&](auto type) {
                using T = decltype(type);
#pragma unroll
                for (int n = 0; n < N; ++n) {
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        if constexpr (CODES) a[n][i] = widen<T>(word[n][i], scale_operand(top[n][i]));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < R; ++i) acc[i][m] = multiply_step<T, CAREFUL>(a[n][i], s[n][m], acc[i][m]);
                }
            };
            if constexpr (!CODES) {
                part(W{});
            } else if constexpr (std::is_same_v<V, f16>) {
                if (__all(exact)) part(f16{});
                else part(bf16{});
            } else {
                part(bf16{});
            }
        }
    }
    settle(acc);
}

}  // namespace vspmm
