// Microscaled 4-bit matrices: quantisation and back, products with dense and with 4-bit tokens, and the gradient of
// the tokens. Declared in include/vspmm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "few.hpp"
#include "host.hpp"
#include "quantize.hpp"
#include "stream.hpp"
#include "tile.hpp"

using namespace vspmm;

namespace {

// ------------------------------------------------------------------ kernels

// Eight waves share 16 R rows and 16 MT tokens, each over an eighth of the contraction; their sums meet in LDS.
constexpr int kFewWaves = 8;
template <typename X, typename O, int R, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void k_few(Row<X> x, int64_t ld_x, int64_t ld_xs, Row<Mx4> w,
                                                        int64_t ld_codes, int64_t ld_scales, O *__restrict__ out,
                                                        int64_t ld_out, int m, int n, int k) {
    __shared__ f32x4 parts[kFewWaves][R][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = int(blockIdx.x) * 16 * R, m0 = int(blockIdx.y) * 16 * MT;
    Row<Mx4> rows[R];
    Row<X> tokens[MT];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t row = min(n0 + 16 * i + r, n - 1);
        rows[i] = {w.codes + row * ld_codes, w.scales + row * ld_scales};
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t row = min(m0 + 16 * t + r, m - 1);
        if constexpr (std::is_same_v<X, Mx4>) tokens[t] = {x.codes + row * ld_x, x.scales + row * ld_xs};
        else tokens[t] = {x.p + row * ld_x};
    }
    const int chunks = (k + kChunkK - 1) / kChunkK;
    f32x4 acc[R][MT] = {};
    accumulate<(MT == 1 ? 4 : 2)>(acc, rows, tokens, chunks * wave / kFewWaves,
                                                chunks * (wave + 1) / kFewWaves, k, g);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t) __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i) parts[wave][i][lane] = acc[i][t];
        __syncthreads();
        if (int(threadIdx.x) < 64 * R) {
            f32x4 sum = parts[0][wave][lane];
#pragma unroll
            for (int v = 1; v < kFewWaves; ++v) sum += parts[v][wave][lane];
            const int mm = m0 + 16 * t + r, nn = n0 + 16 * wave + 4 * g;
            if (mm < m) {
                Vec<O, 4> o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = rounded<O>(sum[e]);
                O *at = out + mm * ld_out + nn;
                if (nn + 4 <= n) {
                    store_vec<4>(at, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nn + e < n) at[e] = o[e];
                }
            }
        }
    }
}

__global__ __launch_bounds__(256) void k_zero_rows(ZeroRows z) { z.run(0); }

// --------------------------------------------------------------------- host

template <typename O>
vspmm_status zero_rows(O *out, int64_t ld, int64_t rows, int64_t width, hipStream_t s) {
    const ZeroRows z(out, ld * int64_t(sizeof(O)), rows, width * int64_t(sizeof(O)));
    hipLaunchKernelGGL(k_zero_rows, dim3(z.blocks(256)), dim3(256), 0, s, z);
    return launched();
}

// Whether tiles of 128, taken for any large product, are more than one launch has threads for: 2^24 of them, whose results
// are up to 2^38. (Few tokens take fewer blocks: the result's rows are of 2^24 values at most.)
bool too_many(int64_t m, int64_t n) {
    return ((m + 127) / 128) * ((n + 127) / 128) > kThreadsMax / kTileThreads;
}

// The few-token kernel, which reads the tokens once for 32 rows, takes up to 32 tokens, and dense ones up to 64 where its
// blocks of 32 x 32 find a compute unit each (64 tokens through 4,096 x 4,096: 12.4 us, by tiles 17.6; 2,048 x 8,192: 23
// and 29; through 5,003 x 4,001 rows, past that, 37 tokens 29 to 36 and 22 to 25). Tiles beyond. With both sides in 4 bits
// tiles are as fast from 33 on (2,048 x 8,192: 12.4 us, 16.5 by this kernel).
constexpr int64_t kFewTokens = 32;
bool few_dense_tokens(int64_t m, int64_t n) {
    return m <= kFewTokens || (m <= 2 * kFewTokens && ((m + 31) / 32) * ((n + 31) / 32) <= 256);
}

template <typename X, typename O>
void launch_few(Row<X> x, int64_t ld_x, int64_t ld_xs, const vspmm_mx4 &w, O *out, int64_t ld_out, int m, int n, int k,
                hipStream_t s) {
    const Row<Mx4> rows{w.codes, w.scales};
    auto go = [&](auto r, auto mt) {
        constexpr int R = decltype(r)::value, MT = decltype(mt)::value;
        hipLaunchKernelGGL((k_few<X, O, R, MT>), dim3((n + 16 * R - 1) / (16 * R), (m + 16 * MT - 1) / (16 * MT)),
                           dim3(64 * kFewWaves), 0, s, x, ld_x, ld_xs, rows, w.ld_codes, w.ld_scales, out, ld_out, m, n,
                           k);
    };
    using std::integral_constant;
    if (m <= 16) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
}

// Tiles of 64 TW x 64 TW results by KS groups: the 128-wide ones, which read each operand half as often, where two to a
// compute unit come together (2,000 tokens of 4,000 to 4,096 rows: 91 us, 137 with 64-wide ones); one with its steps
// shared by two groups where there is one for each (1,000 tokens: 54, 62 with one group, 68); below that 64-wide ones,
// shared by two groups (300: 31, 34 with one, 35 with four) or, where even they leave units idle, by four (128: 19, 21
// with two, 27 with one).
template <typename F>
void with_tile(int64_t m, int64_t n, F &&f) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one{};
    constexpr integral_constant<int, 2> two{};
    constexpr integral_constant<int, 4> four{};
    const int64_t wide = ((m + 127) / 128) * ((n + 127) / 128), narrow = ((m + 63) / 64) * ((n + 63) / 64);
    if (wide >= 400) return f(two, one);
    if (wide >= 192) return f(two, two);
    if (narrow >= 256) return f(one, two);
    return f(one, four);
}

// Whether tiles of 256 x 256 occupy the 256 compute units.
bool fill(int64_t m, int64_t n) { return ((m + 255) / 256) * ((n + 255) / 256) >= 224; }

bool streams(const void *x, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (ld & 7) == 0 && ld < (1 << 22);
}

bool streams(const vspmm_mx4 &a) {
    const auto bits = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    return ((bits(a.codes) | a.ld_codes) & 15) == 0 && ((bits(a.scales) | a.ld_scales) & 3) == 0 &&
           a.ld_codes < (1 << 24) && a.ld_scales < (1 << 24);
}

TileShape tile_shape(int64_t m, int64_t n, int64_t k, int edge, unsigned &tiles) {
    const int64_t tn = (n + edge - 1) / edge;
    tiles = unsigned(((m + edge - 1) / edge) * tn);
    return TileShape{int(m), int(n), int(k), uint32_t(tn)};
}

}  // namespace

extern "C" {

vspmm_status vspmm_mx4_quantize(vspmm_elt elt, int32_t transpose, int64_t rows, int64_t width, const void *x,
                                int64_t ld_x, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
    if (!dense_elt(elt) && elt != VSPMM_ELT_F32) return VSPMM_ERR_ENUM;
    if (vspmm_status st = check_dense(rows, width, ld_x, x)) return st;
    if (transpose && rows > kWidthMax) return VSPMM_ERR_UNSUPPORTED;
    const int64_t n = transpose ? width : rows, blocks = blocks_of_width(transpose ? rows : width);
    if (n == 0 || blocks == 0) return VSPMM_OK;
    if (!codes || !scales) return VSPMM_ERR_NULL;
    auto run = [&](auto e) {
        using T = decltype(e);
        const T *p = static_cast<const T *>(x);
        if (transpose) {
            const int64_t col_tiles = (width + kTransposeCols - 1) / kTransposeCols;
            const int64_t row_tiles = (blocks + kTransposeWaves - 1) / kTransposeWaves;
            const int64_t most = kThreadsMax / (64 * kTransposeWaves) / col_tiles;
            for (int64_t first = 0; first < row_tiles; first += most) {
                const int64_t tiles = col_tiles * std::min(most, row_tiles - first);
                hipLaunchKernelGGL(k_quantize_transposed<T>, dim3(unsigned(tiles)), dim3(64 * kTransposeWaves), 0, stream,
                                   p, ld_x, int(rows), int(width), int(blocks), int(first), uint32_t(col_tiles), codes,
                                   scales);
            }
            return launched();
        }
        const uint32_t per_row = uint32_t(4 * blocks);
        const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per_row);
        for (int64_t r = 0; r < rows; r += most) {
            const uint32_t lanes = uint32_t(std::min(most, rows - r)) * per_row;
            hipLaunchKernelGGL(k_quantize<T>, dim3((lanes + 255) / 256), dim3(256), 0, stream, p + r * ld_x, ld_x, lanes,
                               FastDiv(per_row), per_row, int(width), codes + r * blocks * kBlockBytes,
                               scales + r * blocks);
        }
        return launched();
    };
    return elt == VSPMM_ELT_F32 ? run(float{}) : with_dense(elt, run);
}

vspmm_status vspmm_mx4_dequantize(vspmm_elt elt, int64_t rows, int64_t width, const vspmm_mx4 *x, void *out,
                                  int64_t ld_out, hipStream_t stream) {
    if (!dense_elt(elt) && elt != VSPMM_ELT_F32) return VSPMM_ERR_ENUM;
    if (vspmm_status st = check_mx4(x, rows, width)) return st;
    if (vspmm_status st = check_written(rows, width, ld_out, out)) return st;
    if (rows == 0 || width == 0) return VSPMM_OK;
    auto run = [&](auto e) {
        using T = decltype(e);
        const uint32_t per_row = uint32_t(4 * blocks_of_width(width));
        const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per_row);
        for (int64_t r = 0; r < rows; r += most) {
            const uint32_t lanes = uint32_t(std::min(most, rows - r)) * per_row;
            hipLaunchKernelGGL(k_dequantize<T>, dim3((lanes + 255) / 256), dim3(256), 0, stream,
                               x->codes + r * x->ld_codes, x->ld_codes, x->scales + r * x->ld_scales, x->ld_scales,
                               lanes, FastDiv(per_row), per_row, int(width), static_cast<T *>(out) + r * ld_out, ld_out);
        }
        return launched();
    };
    return elt == VSPMM_ELT_F32 ? run(float{}) : with_dense(elt, run);
}

vspmm_status vspmm_mx4_matmul(vspmm_elt elt, int64_t m, int64_t n, int64_t width, const void *x, int64_t ld_x,
                              const vspmm_mx4 *w, void *out, int64_t ld_out, hipStream_t stream) {
    if (!dense_elt(elt)) return VSPMM_ERR_ENUM;
    if (vspmm_status st = check_dense(m, width, ld_x, x)) return st;
    if (vspmm_status st = check_mx4(w, n, width)) return st;
    if (vspmm_status st = check_written(m, n, ld_out, out)) return st;
    if (m == 0 || n == 0) return VSPMM_OK;
    if (too_many(m, n)) return VSPMM_ERR_UNSUPPORTED;
    return with_dense(elt, [&](auto e) {
        using T = decltype(e);
        T *o = static_cast<T *>(out);
        if (width == 0) return zero_rows(o, ld_out, m, n, stream);
        if (few_dense_tokens(m, n)) {
            launch_few(Row<T>{static_cast<const T *>(x)}, ld_x, 0, *w, o, ld_out, int(m), int(n), int(width), stream);
            return launched();
        }
        if (m >= 256 && n >= 256 && width % kChunkK == 0 && fill(m, n) && streams(x, ld_x) && streams(*w)) {
            unsigned tiles;
            const TileShape s = tile_shape(m, n, width, 256, tiles);
            allow_lds<&k_stream<T>>(kStreamLds);
            hipLaunchKernelGGL((k_stream<T>), dim3(tiles), dim3(256), kStreamLds, stream, static_cast<const T *>(x), ld_x,
                               w->codes, w->ld_codes, w->scales, w->ld_scales, o, ld_out, s);
            return launched();
        }
        with_tile(m, n, [&](auto tw, auto ks) {
            constexpr int TW = decltype(tw)::value, KS = decltype(ks)::value;
            unsigned tiles;
            const TileShape s = tile_shape(m, n, width, 64 * TW, tiles);
            allow_lds<&k_tile<TW, KS, T, T>>(KS * tile_lds<TW>());
            hipLaunchKernelGGL((k_tile<TW, KS, T, T>), dim3(tiles), dim3(kTileThreads * KS), KS * tile_lds<TW>(), stream,
                               static_cast<const T *>(x), ld_x, w->codes, w->ld_codes, w->scales, w->ld_scales, o,
                               ld_out, s);
        });
        return launched();
    });
}

vspmm_status vspmm_mx4_matmul_grad(vspmm_elt elt, int64_t m, int64_t n, int64_t width, const void *dout, int64_t ld_dout,
                                   const vspmm_mx4 *w, void *grad, int64_t ld_grad, hipStream_t stream) {
    if (!dense_elt(elt)) return VSPMM_ERR_ENUM;
    if (vspmm_status st = check_dense(m, n, ld_dout, dout)) return st;
    if (vspmm_status st = check_mx4(w, n, width)) return st;
    if (vspmm_status st = check_written(m, width, ld_grad, grad)) return st;
    if (m == 0 || width == 0) return VSPMM_OK;
    if (too_many(m, width)) return VSPMM_ERR_UNSUPPORTED;
    return with_dense(elt, [&](auto e) {
        using T = decltype(e);
        T *o = static_cast<T *>(grad);
        if (n == 0) return zero_rows(o, ld_grad, m, width, stream);
        // (a wave's copies of 64 rows reach 2^31 bytes past the first)
        if (m >= 256 && n % kStepHalf == 0 && fill(m, width) && streams(dout, ld_dout) && n + 64 * ld_dout <= 1 << 30) {
            unsigned tiles;
            const TileShape s = tile_shape(m, width, n, 256, tiles);
            allow_lds<&k_stream_grad<T>>(kStreamGradLds);
            hipLaunchKernelGGL((k_stream_grad<T>), dim3(tiles), dim3(256), kStreamGradLds, stream,
                               static_cast<const T *>(dout), ld_dout, w->codes, w->ld_codes, w->scales, w->ld_scales, o,
                               ld_grad, s);
            return launched();
        }
        with_tile(m, width, [&](auto tw, auto ks) {
            constexpr int TW = decltype(tw)::value, KS = decltype(ks)::value;
            unsigned tiles;
            const TileShape s = tile_shape(m, width, n, 64 * TW, tiles);
            allow_lds<&k_tile_grad<TW, KS, T>>(KS * grad_lds<TW>());
            hipLaunchKernelGGL((k_tile_grad<TW, KS, T>), dim3(tiles), dim3(kTileThreads * KS), KS * grad_lds<TW>(), stream,
                               static_cast<const T *>(dout), ld_dout, w->codes, w->ld_codes, w->scales, w->ld_scales, o,
                               ld_grad, s);
        });
        return launched();
    });
}

vspmm_status vspmm_mx4_matmul_mx4(vspmm_elt elt, int64_t m, int64_t n, int64_t width, const vspmm_mx4 *x,
                                  const vspmm_mx4 *w, void *out, int64_t ld_out, hipStream_t stream) {
    if (!dense_elt(elt) && elt != VSPMM_ELT_F32) return VSPMM_ERR_ENUM;
    if (vspmm_status st = check_mx4(x, m, width)) return st;
    if (vspmm_status st = check_mx4(w, n, width)) return st;
    if (vspmm_status st = check_written(m, n, ld_out, out)) return st;
    if (m == 0 || n == 0) return VSPMM_OK;
    if (too_many(m, n)) return VSPMM_ERR_UNSUPPORTED;
    auto run = [&](auto e) {
        using T = decltype(e);
        T *o = static_cast<T *>(out);
        if (width == 0) return zero_rows(o, ld_out, m, n, stream);
        if (m <= kFewTokens) {
            launch_few(Row<Mx4>{x->codes, x->scales}, x->ld_codes, x->ld_scales, *w, o, ld_out, int(m), int(n),
                       int(width), stream);
            return launched();
        }
        if (m >= 256 && n >= 256 && width % kStepCodes == 0 && fill(m, n) && streams(*x) && streams(*w)) {
            unsigned tiles;
            const TileShape s = tile_shape(m, n, width, 256, tiles);
            allow_lds<&k_stream_both<T>>(kStreamBothLds);
            hipLaunchKernelGGL((k_stream_both<T>), dim3(tiles), dim3(256), kStreamBothLds, stream, x->codes,
                               x->ld_codes, x->scales, x->ld_scales, w->codes, w->ld_codes, w->scales, w->ld_scales, o,
                               ld_out, s);
            return launched();
        }
        with_tile(m, n, [&](auto tw, auto ks) {
            constexpr int TW = decltype(tw)::value, KS = decltype(ks)::value;
            unsigned tiles;
            const TileShape s = tile_shape(m, n, width, 64 * TW, tiles);
            allow_lds<&k_tile_both<TW, KS, T>>(KS * both_lds<TW>());
            hipLaunchKernelGGL((k_tile_both<TW, KS, T>), dim3(tiles), dim3(kTileThreads * KS), KS * both_lds<TW>(), stream, x->codes,
                               x->ld_codes, x->scales, x->ld_scales, w->codes, w->ld_codes, w->scales, w->ld_scales, o,
                               ld_out, s);
        });
        return launched();
    };
    return elt == VSPMM_ELT_F32 ? run(float{}) : with_dense(elt, run);
}

}  // extern "C"
