// Microscaled 4-bit matrices: codes of 4 bits (sign, two exponent bits, one mantissa bit), 32 to a 16-byte block of a
// row with value 2 j in the low half of byte j, and one power of two 2^(b - 127) a block (b = 255: not a number).
// gfx950 converts between the codes and 16- or 32-bit floats with the scale applied (v_cvt_scalef32_pk_*; the scale
// operand's exponent field is the byte b) and multiplies them in its matrix instructions. Both were checked here for
// every code and scale: values are exact where the type holds them, b = 255 gives NaN, conversions to codes round to
// nearest even and saturate, and the matrix instructions keep subnormal operands and results.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../csrc_select/rows.hpp"

namespace vspmm {

constexpr int kBlock = 32;       // values of a block
constexpr int kBlockBytes = 16;  // their codes

using i32x4 = int32_t __attribute__((ext_vector_type(4)));
using i32x8 = int32_t __attribute__((ext_vector_type(8)));
using f32x2 = float __attribute__((ext_vector_type(2)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x4 = __bf16 __attribute__((ext_vector_type(4)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));

// 16 bytes at the alignment of one element of 16 bits, or of a byte.
using Half16 = i32x4 __attribute__((aligned(2)));
using Byte16 = i32x4 __attribute__((aligned(1)));

struct Mx4 {};     // element type of a microscaled matrix
struct Planes {};  // float32 values as the sum of three bfloat16 ones, eight values' first, second and third parts in turn

template <typename T, typename F>
__device__ __forceinline__ T bits_as(F x) {
    static_assert(sizeof(T) == sizeof(F));
    return __builtin_bit_cast(T, x);
}

// The scale operand of the conversions.
__device__ __forceinline__ float scale_operand(uint32_t b) { return __uint_as_float(b << 23); }

// Codes 2 H and 2 H + 1 of a word of eight as two values of 16 bits.
template <typename T, int H>
__device__ __forceinline__ int32_t widen_two(uint32_t codes, float scale) {
    if constexpr (std::is_same_v<T, bf16>)
        return bits_as<int32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, H));
    else return bits_as<int32_t>(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, H));
}
template <typename T>
__device__ __forceinline__ int32_t widen_pair(uint32_t codes, float scale, int h) {  // h: known when compiled
    return h == 0   ? widen_two<T, 0>(codes, scale)
           : h == 1 ? widen_two<T, 1>(codes, scale)
           : h == 2 ? widen_two<T, 2>(codes, scale)
                    : widen_two<T, 3>(codes, scale);
}

// Eight codes (a word) as eight values of 16 bits.
template <typename T>
__device__ __forceinline__ i32x4 widen(uint32_t codes, float scale) {
    return i32x4{widen_two<T, 0>(codes, scale), widen_two<T, 1>(codes, scale), widen_two<T, 2>(codes, scale),
                 widen_two<T, 3>(codes, scale)};
}

// Whether a product with float16 tokens may take a block in float16, which has to hold all of its values: it does at
// scales from 2^-23 to 2^13 (0.5 * 2^-23 is its least subnormal, 6 * 2^13 lies below its largest number), and at smaller
// ones where all are zero, as those of a block of zeros are.
__device__ __forceinline__ bool f16_scale(uint32_t b) { return b - 104u <= 36u; }
__device__ __forceinline__ bool f16_zeros(uint32_t b, uint32_t codes) { return b < 104u && (codes & 0x77777777u) == 0; }
__device__ __forceinline__ bool f16_zeros(uint32_t b, i32x4 codes) {
    return f16_zeros(b, uint32_t(codes[0] | codes[1] | codes[2] | codes[3]));
}
// Whether it holds the blocks that a thread block's threads walk between them: each(ok) says whether ok(scale, codes)
// holds for all of this thread's. Their scales nearly always settle it (with codes looked at in the same walk 4,096 tokens
// through 8,192 x 8,192 took 472 us, 446 so).
template <typename Each>
__device__ __forceinline__ bool f16_holds(Each &&each) {
    if (__syncthreads_and(each([](uint32_t b, const uint8_t *) { return f16_scale(b); }))) return true;
    return __syncthreads_and(each([](uint32_t b, const uint8_t *codes) {
        return f16_scale(b) || (b < 104u && f16_zeros(b, i32x4(*reinterpret_cast<const Byte16 *>(codes))));
    }));
}

// Eight float16 values as the sum of two bfloat16 each: the upper eight bits of the significand, and the rest, which
// has at most three. Exact: float16's least subnormal is a normal bfloat16. An infinity or NaN goes into the first.
__device__ __forceinline__ void split(i32x4 v, i32x4 &hi, i32x4 &lo) {
    const f16x8 x = bits_as<f16x8>(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = float(x[2 * i]), b = float(x[2 * i + 1]);
        const uint32_t ua = __float_as_uint(a) & 0xffff0000u, ub = __float_as_uint(b) & 0xffff0000u;
        hi[i] = int32_t((ua >> 16) | ub);
        // x - x for an infinity: its second part is zero
        const float la = __builtin_isinf(a) ? 0.0f : a - __uint_as_float(ua);
        const float lb = __builtin_isinf(b) ? 0.0f : b - __uint_as_float(ub);
        lo[i] = int32_t((__float_as_uint(la) >> 16) | (__float_as_uint(lb) & 0xffff0000u));
    }
}

// Eight bfloat16 values, zeros in the place of infinities and NaN. Where a factor goes in parts, an infinity of the other
// meets the first part alone: the others may be zero, and infinity times zero is not a number.
__device__ __forceinline__ i32x4 finite(i32x4 v) {
    i32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = uint32_t(v[i]);
        const uint32_t top = ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // of a half: its exponent is the largest
        out[i] = int32_t(w & ~(top - (top >> 15)));
    }
    return out;
}

template <typename T>
__device__ __forceinline__ f32x4 mma16(i32x4 a, i32x4 b, f32x4 c) {
    if constexpr (std::is_same_v<T, bf16>)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bits_as<bf16x8>(a), bits_as<bf16x8>(b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(bits_as<f16x8>(a), bits_as<f16x8>(b), c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ f32x16 mma32(i32x4 a, i32x4 b, f32x16 c) {
    if constexpr (std::is_same_v<T, bf16>)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bits_as<bf16x8>(a), bits_as<bf16x8>(b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(bits_as<f16x8>(a), bits_as<f16x8>(b), c, 0, 0, 0);
}

// The product of two blocks of 4-bit codes, each with its scales in byte I of a word.
template <int I>
__device__ __forceinline__ f32x4 mma16_mx4(i32x4 a, uint32_t sa, i32x4 b, uint32_t sb, f32x4 c) {
    const i32x8 a8 = __builtin_shufflevector(a, i32x4{}, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 b8 = __builtin_shufflevector(b, i32x4{}, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, I, int(sa), I, int(sb));
}
template <int I>
__device__ __forceinline__ f32x16 mma32_mx4(i32x4 a, uint32_t sa, i32x4 b, uint32_t sb, f32x16 c) {
    const i32x8 a8 = __builtin_shufflevector(a, i32x4{}, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 b8 = __builtin_shufflevector(b, i32x4{}, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, I, int(sa), I, int(sb));
}

// Waits until the matrix instructions have written their sums. The compiler puts waits between such an instruction and
// a use of its result, but here it was seen to leave them out: where a branch leads past a short block straight from
// the instruction to the use, the first registers of the sum were read too early. So a sum goes through here before any
// use but another product. Branches between products (float16 tokens choose their type at every chunk, the last chunks go
// by size) lead from products to products on the same sums, or to here. In the assembly of every kernel, along every
// path, no other instruction reads a product's result before 8 wait states (16 x 16) or 12 (32 x 32).
template <typename V, int A, int B>
__device__ __forceinline__ void settle(V (&acc)[A][B]) {
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j) asm volatile("" : "+v"(acc[i][j]));
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// A barrier for what lies in LDS: loads to registers stay on their way (__syncthreads waits for them).
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__host__ __device__ constexpr int64_t blocks_of_width(int64_t width) { return (width + kBlock - 1) / kBlock; }

}  // namespace vspmm
