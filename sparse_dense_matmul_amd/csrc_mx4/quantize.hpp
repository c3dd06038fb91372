// Rows to microscaled 4-bit codes and back. The scale of a block of 32 has the exponent of its largest magnitude less
// 2 (the codes' largest exponent), at least 2^-127; a value over its scale is rounded to the nearest code, ties to
// even, and those past 6 become 6. A block with an infinity or NaN becomes NaN (scale byte 255, codes 0).
#pragma once

#include "mx4.hpp"

namespace vspmm {

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_of(uint32_t most) {
    if (most >= 0x7f800000u) return 255;
    const uint32_t e = most >> 23;
    return e > 2 ? e - 2 : 0;
}

// Eight values as a word of codes. The conversion reads the exponent field alone: 0 stands for 2^-127.
__device__ __forceinline__ uint32_t encode(const float (&v)[8], uint32_t scale) {
    if (scale == 255) return 0;
    const float s = scale_operand(scale);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
    return r;
}

// A lane takes 8 values of a row, four lanes a block: 16-byte loads of 16-bit values and 4-byte stores of codes, both
// without gaps over the lanes. Bound by memory, and at a few rows by the launch (32 x 4,096 bfloat16: 2.6 us). per_row:
// lanes of a row, 4 * blocks.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize(const T *__restrict__ x, int64_t ld, uint32_t n, FastDiv by_row,
                                                  uint32_t per_row, int width, uint8_t *__restrict__ codes,
                                                  uint8_t *__restrict__ scales) {
    const uint32_t c = blockIdx.x * 256u + threadIdx.x;
    if (c >= n) return;  // n is a multiple of 4: a block's lanes leave together
    const uint32_t row = by_row.div(c), part = c - row * per_row;
    const T *p = x + row * ld;
    const int k = int(part) * 8;
    float v[8];
    if (k + 8 <= width) {
        const Vec<T, 8> t = load_vec<8>(p + k);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = float(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < width ? float(p[k + i]) : 0.0f;
    }
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, magnitude(v[i]));
    most = max(most, uint32_t(__shfl_xor(int(most), 1)));
    most = max(most, uint32_t(__shfl_xor(int(most), 2)));
    const uint32_t s = scale_of(most);
    reinterpret_cast<uint32_t __attribute__((aligned(1))) *>(codes)[c] = encode(v, s);
    if ((c & 3) == 0) scales[c >> 2] = uint8_t(s);
}

// The transpose's rows: a lane takes two columns of x over the 32 rows of one of their blocks, so a wave reads 128
// columns in a row. Eight waves take eight blocks in a row of the same columns, whose codes meet in LDS and leave as
// 128 bytes a column. Bound by memory: 16,384 x 8,192 bfloat16 in 71 to 93 us, 3.6 to 4.8 TB/s.
constexpr int kTransposeWaves = 8, kTransposeCols = 128;
template <typename T>
__global__ __launch_bounds__(64 * kTransposeWaves) void k_quantize_transposed(
    const T *__restrict__ x, int64_t ld, int rows, int width, int blocks, int first_tile, uint32_t col_tiles,
    uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    // a column's blocks, 16 bytes further for every column so that the lanes' stores spread over the banks
    __shared__ i32x4 tile[kTransposeCols][kTransposeWaves + 1];
    __shared__ uint8_t tops[kTransposeCols][kTransposeWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int b0 = (first_tile + int(blockIdx.x / col_tiles)) * kTransposeWaves;
    const int col0 = int(blockIdx.x % col_tiles) * kTransposeCols, col = col0 + 2 * lane;
    const int64_t r0 = int64_t(b0 + wave) * kBlock;
    const T *p = x + r0 * ld + col;
    float v[2][kBlock];
    uint32_t most[2] = {0, 0};
    if (r0 + kBlock <= rows && col + 2 <= width) {
        Vec<T, 2> t[kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i) t[i] = load_vec<2>(p + i * ld);
#pragma unroll
        for (int i = 0; i < kBlock; ++i) v[0][i] = float(t[i][0]), v[1][i] = float(t[i][1]);
    } else {
#pragma unroll
        for (int i = 0; i < kBlock; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[h][i] = r0 + i < rows && col + h < width ? float(p[i * ld + h]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kBlock; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) most[h] = max(most[h], magnitude(v[h][i]));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t s = scale_of(most[h]);
        i32x4 c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float part[8] = {v[h][8 * j],     v[h][8 * j + 1], v[h][8 * j + 2], v[h][8 * j + 3],
                                   v[h][8 * j + 4], v[h][8 * j + 5], v[h][8 * j + 6], v[h][8 * j + 7]};
            c[j] = int32_t(encode(part, s));
        }
        tile[2 * lane + h][wave] = c;
        tops[2 * lane + h][wave] = uint8_t(s);
    }
    __syncthreads();
    for (int s = threadIdx.x; s < kTransposeCols * kTransposeWaves; s += 64 * kTransposeWaves) {
        const int c = s / kTransposeWaves, w = s % kTransposeWaves;
        if (col0 + c < width && b0 + w < blocks) {
            const int64_t at = int64_t(col0 + c) * blocks + b0 + w;
            *reinterpret_cast<Byte16 *>(codes + at * kBlockBytes) = tile[c][w];
            scales[at] = tops[c][w];
        }
    }
}

// A lane takes 8 codes: 4-byte loads, 16-byte stores of 16-bit values. Bound by memory: 8,192 x 16,384 to bfloat16 in
// 68 us, 5.0 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                    const uint8_t *__restrict__ scales, int64_t ld_scales, uint32_t n,
                                                    FastDiv by_row, uint32_t per_row, int width, T *__restrict__ out,
                                                    int64_t ld) {
    const uint32_t c = blockIdx.x * 256u + threadIdx.x;
    if (c >= n) return;
    const uint32_t row = by_row.div(c), part = c - row * per_row;
    const int k = int(part) * 8;
    if (k >= width) return;
    const uint32_t word =
        *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(codes + row * ld_codes + 4 * part);
    const float s = scale_operand(scales[row * ld_scales + part / 4]);
    Vec<T, 8> v;
    if constexpr (sizeof(T) == 2) {
        v = bits_as<Vec<T, 8>>(widen<T>(word, s));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 t = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 0)
                            : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 1)
                            : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 2)
                                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 3);
            v[2 * j] = t[0];
            v[2 * j + 1] = t[1];
        }
    }
    T *o = out + row * ld + k;
    if (k + 8 <= width) {
        store_vec<8>(o, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < width) o[i] = v[i];
    }
}

}  // namespace vspmm
