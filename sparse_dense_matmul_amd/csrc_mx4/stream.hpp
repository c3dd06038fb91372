// Products with many tokens whose operands lie as the loads to LDS want them.
#pragma once

#include "tile.hpp"

namespace vspmm {

using Lds = __attribute__((address_space(3))) char;

// A wave's 64 pieces of BYTES bytes, each lane's at its own offset from a base and `more` beyond it, to consecutive
// ones in LDS. The address's common part stays in scalar registers.
using Buffer = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Buffer buffer_of(const uint8_t *p, uint32_t bytes = 0x80000000u) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, int(bytes), 0x00020000);
}
// Rows of `width` bytes from row0 on whose copies run past a row's end: past the last row's are zeros.
__device__ __forceinline__ Buffer rows_of(const uint8_t *p, int64_t ld, int row0, int rows, int width) {
    const int64_t bytes = int64_t(rows - 1 - row0) * ld + width;
    return buffer_of(p + row0 * ld, bytes < 0x80000000ll ? uint32_t(bytes) : 0x80000000u);
}
__device__ __forceinline__ void copy16(Buffer from, uint32_t offset, uint32_t more, Lds *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, int(offset),
                                             int(more), 0, 0);
}
__device__ __forceinline__ void copy4(Buffer from, uint32_t offset, uint32_t more, Lds *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 4, int(offset),
                                             int(more), 0, 0);
}

// Keeps the sums' products on their side of here: the compiler moves them over scheduling barriers otherwise. No
// instruction is made.
template <int A, int B>
__device__ __forceinline__ void pin(f32x16 (&acc)[A][B]) {
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// The order of a part of a step, 16 products: READS loads from LDS behind each of the first eight, so that they are
// there at the next part's first product, and one of COPIES loads to LDS behind every other of the rest and then of all
// (a wave waits to issue them while others' are on their way, its products with it).
template <int READS, int COPIES, int LOADS = 0>
__device__ __forceinline__ void mix() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (READS > 0)
            if (i < 8) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        if constexpr (LOADS > 0) {
            if (i >= 8) __builtin_amdgcn_sched_group_barrier(0x010, LOADS, 0);
        } else if constexpr (COPIES > 0) {
            if (i % 3 == 2 && i / 3 < COPIES) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        }
    }
}

// The same where an instruction's rows are widened beside the products, by VALU operations behind each from the
// FIRST on.
template <int READS, int COPIES, int FIRST, int VALU>
__device__ __forceinline__ void mix_widening() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (i % 3 == 2 && i / 3 < COPIES) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        if (i >= FIRST) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    }
}

// Both sides in 4 bits: a step is 256 codes, 128 bytes of a row of each side. One wave a SIMD holds 128 x 128 results, so
// that a step's 64 products need 16 loads from LDS; smaller tiles read as much for a quarter of the products. 8,192^3 in
// 308 to 333 us, 3.3 to 3.6 PFLOP/s, where the instructions alone reach 6.5 on random codes. Every step waits for all of
// its copies at its barrier, whose last ones leave 12 products before it; what the waits cost was not told apart.
constexpr int kStreamEdge = 256;
constexpr size_t kStreamBothLds = 2 * 512 * (128 + 16);

template <typename O>
__global__ __launch_bounds__(256, 1) void k_stream_both(const uint8_t *__restrict__ x_codes, int64_t ld_x,
                                                     const uint8_t *__restrict__ x_scales, int64_t ld_xs,
                                                     const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                     const uint8_t *__restrict__ scales, int64_t ld_scales,
                                                     O *__restrict__ out, int64_t ld_out, TileShape s) {
    constexpr int TW = 4;
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5;
    uint32_t tm, tn;
    tile_of(s, (uint32_t(s.m) + 255) / 256, tm, tn);
    const int m0 = min(int(tm) * 256, s.m - 256), n0 = min(int(tn) * 256, s.n - 256);

    // waves 0 and 1 copy the tokens' rows, 2 and 3 the matrix's: 16 times 8 rows each
    const bool mine = wave < 2;
    const int64_t ld = mine ? ld_x : ld_codes;
    const int row0 = (mine ? m0 : n0) + (wave & 1) * 128;
    const Buffer src = buffer_of((mine ? x_codes : codes) + row0 * ld);
    const uint32_t rows8 = 8 * uint32_t(ld);
    const uint32_t off[2] = {uint32_t(lane >> 3) * uint32_t(ld) + 16 * ((lane & 7) ^ (lane >> 3)),
                             uint32_t(lane >> 3) * uint32_t(ld) + 16 * ((lane & 7) ^ (lane >> 3) ^ 1)};
    Lds *base = (Lds *)smem;
    Lds *to = base + wave * 128 * 128;
    auto copy = [&](int it, int buf, int i) {
        copy16(src, off[i & 1], uint32_t(it) * 128 + i * rows8, to + buf * 512 * 128 + i * 1024);
    };
    // scales go by two steps, 16 bytes a row: in each of the two a wave copies those of 64 of its 128 rows
    const int64_t lds_ = mine ? ld_xs : ld_scales;
    const Buffer src_s = rows_of(mine ? x_scales : scales, lds_, row0, mine ? s.m : s.n, s.k / kBlock);
    const uint32_t off_s = uint32_t(lane) * uint32_t(lds_), rows64 = 64 * uint32_t(lds_);
    const char *tops = smem + 2 * 512 * 128;
    Lds *to_s = (Lds *)tops + wave * 128 * 16;
    auto copy_s = [&](int pair, int buf, int half) {
        copy16(src_s, off_s, uint32_t(pair) * 16 + half * rows64, to_s + buf * 512 * 16 + half * 1024);
    };

    f32x16 acc[TW][TW] = {};
    const int wm = (wave & 1) * 128, wn = (wave >> 1) * 128;
    const uint32_t pick = 0x06040200u + uint32_t(g) * 0x01010101u;
    const int steps = s.k / kStepCodes;
    const int turn = (r ^ (r >> 3 & 1)) & 7;
    i32x4 p[2][TW], q[2][TW];
    uint2 tx[TW], tw[TW];      // scales as they lie
    uint32_t sx[TW], sw[TW];   // the four that this lane's blocks of a step have
    auto read = [&](int buf, int set, int j) {
        const i32x4 *bx = reinterpret_cast<const i32x4 *>(smem + buf * 512 * 128), *bw = bx + 256 * 8;
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            q[set][t] = bx[(wm + 32 * t + r) * 8 + ((2 * j + g) ^ turn)];
            p[set][t] = bw[(wn + 32 * t + r) * 8 + ((2 * j + g) ^ turn)];
        }
    };
    auto read_s = [&](int buf, int half) {
        const uint2 *b = reinterpret_cast<const uint2 *>(tops + buf * 512 * 16) + half;
#pragma unroll
        for (int t = 0; t < TW; ++t) tx[t] = b[2 * (wm + 32 * t + r)], tw[t] = b[2 * (256 + wn + 32 * t + r)];
    };
    auto multiply = [&](auto index) {
        constexpr int J = decltype(index)::value;
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
            for (int i = 0; i < TW; ++i)
                acc[i][j] = mma32_mx4<J>(p[J & 1][i], sw[i], q[J & 1][j], sx[j], acc[i][j]);
    };
    using std::integral_constant;
    // At step `it`'s start its first operands are in registers, its copies have arrived, the first of the next
    // step's are on their way. Behind the last step the copies repeat it: nothing reads them.
    const int last = steps - 1;
#pragma unroll
    for (int i = 0; i < 16; ++i) copy(0, 0, i);
    copy_s(0, 0, 0);
    copy_s(0, 0, 1);
    __syncthreads();
    read(0, 0, 0);
    read_s(0, 0);
#pragma unroll
    for (int i = 0; i < 5; ++i) copy(min(1, last), 1, i);
    for (int it = 0; it < steps; ++it) {
        const int P = it & 1, B = it >> 1 & 1;
        const int next = min(it + 1, last), second = min(it + 2, last), pair = min((it >> 1) + 1, last >> 1);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            sx[t] = __builtin_amdgcn_perm(tx[t].y, tx[t].x, pick);
            sw[t] = __builtin_amdgcn_perm(tw[t].y, tw[t].x, pick);
        }
        __builtin_amdgcn_sched_barrier(0);
        read(P, 1, 1);
        copy_s(pair, 1 - B, P);
#pragma unroll
        for (int i = 5; i < 9; ++i) copy(next, 1 - P, i);
        multiply(integral_constant<int, 0>{});
        mix<1, 5>();
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
        read(P, 0, 2);
#pragma unroll
        for (int i = 9; i < 13; ++i) copy(next, 1 - P, i);
        multiply(integral_constant<int, 1>{});
        mix<1, 4>();
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
        read(P, 1, 3);
#pragma unroll
        for (int i = 13; i < 16; ++i) copy(next, 1 - P, i);
        multiply(integral_constant<int, 2>{});
        mix<1, 3>();
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        read(1 - P, 0, 0);
        read_s(P ? 1 - B : B, 1 - P);
#pragma unroll
        for (int i = 0; i < 5; ++i) copy(second, P, i);
        multiply(integral_constant<int, 3>{});
        mix<2, 5>();
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
    }
    pin(acc);
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");  // as settle() does
    pin(acc);
    __syncthreads();  // no copy is on its way when the block ends
    store_tile<TW>(acc, out, ld_out, m0 + wm, n0 + wn, s.m, s.n, lane);
}

// Dense tokens. A step is 64 values: 128 bytes of a token's row, copied for every step, and a quarter of the 128 bytes
// of codes of a row, copied for every four. An instruction's part of the rows is widened while the part before it is
// multiplied. Bound by the clock under the matrix instructions and by what the conversions take beside them: 4,096 tokens
// through 8,192 x 8,192 in 405 to 467 us, 1.18 to 1.36 PFLOP/s (1.7 by the instructions alone on random operands); float16
// 434 to 450 us.
constexpr size_t kStreamLds = 2 * 256 * (128 + 128 + 16);

template <typename X>
__global__ __launch_bounds__(256, 1) void k_stream(const X *__restrict__ x, int64_t ld_x,
                                                   const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                   const uint8_t *__restrict__ scales, int64_t ld_scales,
                                                   X *__restrict__ out, int64_t ld_out, TileShape s) {
    constexpr int TW = 4;
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5;
    uint32_t tm, tn;
    tile_of(s, (uint32_t(s.m) + 255) / 256, tm, tn);
    // The last tile of either side is moved to end with the matrix. Columns stay those of the tile that they would lie in:
    // the route of float16 tokens is chosen by a tile's own rows, and the two tiles' sums of a column may differ.
    const int own = int(tn) * 256;
    const int m0 = min(int(tm) * 256, s.m - 256), n0 = min(own, s.n - 256);

    // a wave copies 64 tokens' rows and 64 of the matrix's, eight at a time
    const char *lds_x = smem, *lds_w = smem + 2 * 256 * 128, *lds_s = smem + 4 * 256 * 128;
    const int64_t ld_xb = ld_x * 2;
    const Buffer src_x = buffer_of(reinterpret_cast<const uint8_t *>(x) + (m0 + 64 * wave) * ld_xb);
    const Buffer src_w = rows_of(codes, ld_codes, n0 + 64 * wave, s.n, s.k / 2);
    const Buffer src_s = rows_of(scales, ld_scales, n0 + 64 * wave, s.n, s.k / kBlock);
    const uint32_t piece = 16 * ((lane & 7) ^ (lane >> 3));
    const uint32_t off_x = uint32_t(lane >> 3) * uint32_t(ld_xb), off_w = uint32_t(lane >> 3) * uint32_t(ld_codes);
    const uint32_t offs_x[2] = {off_x + piece, off_x + (piece ^ 16)}, offs_w[2] = {off_w + piece, off_w + (piece ^ 16)};
    const uint32_t off_s = uint32_t(lane) * uint32_t(ld_scales);
    const uint32_t rows_x = 8 * uint32_t(ld_xb), rows_w = 8 * uint32_t(ld_codes);
    Lds *to_x = (Lds *)lds_x + wave * 64 * 128, *to_w = (Lds *)lds_w + wave * 64 * 128;
    Lds *to_s = (Lds *)lds_s + wave * 64 * 16;
    auto copy_x = [&](int it, int buf, int i) {
        copy16(src_x, offs_x[i & 1], uint32_t(it) * 128 + i * rows_x, to_x + buf * 256 * 128 + i * 1024);
    };
    // two of the eight of a group of four steps; i: 0, 2, 4, 6
    auto copy_w = [&](int four, int buf, int i) {
        copy16(src_w, offs_w[0], uint32_t(four) * 128 + i * rows_w, to_w + buf * 256 * 128 + i * 1024);
        copy16(src_w, offs_w[1], uint32_t(four) * 128 + (i + 1) * rows_w, to_w + buf * 256 * 128 + i * 1024 + 1024);
    };
    auto copy_s = [&](int eight, int buf) { copy16(src_s, off_s, uint32_t(eight) * 16, to_s + buf * 256 * 16); };

    f32x16 acc[TW][TW] = {};
    const int wm = (wave & 1) * 128, wn = (wave >> 1) * 128;
    const int turn = (r ^ (r >> 3 & 1)) & 7;
    i32x4 q[2][TW], p[2][TW], c[2][TW];  // tokens and widened rows of an instruction, codes of a step
    uint32_t b[2][TW];                   // and their scales
    auto read = [&](int buf, int set, int j) {
        const i32x4 *bx = reinterpret_cast<const i32x4 *>(lds_x + buf * 256 * 128);
#pragma unroll
        for (int t = 0; t < TW; ++t) q[set][t] = bx[(wm + 32 * t + r) * 8 + ((4 * g + j) ^ turn)];
    };
    auto read_w = [&](int it, int set) {
        const i32x4 *bw = reinterpret_cast<const i32x4 *>(lds_w + (it >> 2 & 1) * 256 * 128);
        const uint8_t *bs = reinterpret_cast<const uint8_t *>(lds_s + (it >> 3 & 1) * 256 * 16) + 2 * (it & 7) + g;
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            c[set][t] = bw[(wn + 32 * t + r) * 8 + ((2 * (it & 3) + g) ^ turn)];
            b[set][t] = bs[16 * (wn + 32 * t + r)];
        }
    };
    const int steps = s.k / kStepHalf, last = steps - 1;
    auto run = [&](auto type) {
        using T = decltype(type);
        auto widen_rows = [&](int set, int from, int j) {
#pragma unroll
            for (int t = 0; t < TW; ++t) p[set][t] = widen<T>(uint32_t(c[from][t][j]), scale_operand(b[from][t]));
        };
        auto multiply = [&](int set) {
#pragma unroll
            for (int j = 0; j < TW; ++j) {
                i32x4 hi = q[set][j], lo;
                if constexpr (!std::is_same_v<T, X>) split(q[set][j], hi, lo);
#pragma unroll
                for (int i = 0; i < TW; ++i) {
                    acc[i][j] = mma32<T>(p[set][i], hi, acc[i][j]);
                    if constexpr (!std::is_same_v<T, X>) acc[i][j] = mma32<T>(finite(p[set][i]), lo, acc[i][j]);
                }
            }
        };
        read(0, 0, 0);
        read_w(0, 0);
        widen_rows(0, 0, 0);
#pragma unroll
        for (int i = 0; i < 3; ++i) copy_x(min(1, last), 1, i);
        for (int it = 0; it < steps; ++it) {
            const int P = it & 1, next = min(it + 1, last), second = min(it + 2, last);
            const int four = min((it >> 2) + 1, last >> 2);
            if ((it & 7) == wave) copy_s(min((it >> 3) + 1, last >> 3), ~(it >> 3) & 1);
            __builtin_amdgcn_sched_barrier(0);
            read(P, 1, 1);
            widen_rows(1, 0, 1);
#pragma unroll
            for (int i = 3; i < 6; ++i) copy_x(next, 1 - P, i);
            multiply(0);
            mix_widening<4, 3, 0, 1>();
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
            read(P, 0, 2);
            widen_rows(0, 0, 2);
#pragma unroll
            for (int i = 6; i < 8; ++i) copy_x(next, 1 - P, i);
            multiply(1);
            mix_widening<4, 2, 0, 1>();
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
            read(P, 1, 3);
            widen_rows(1, 0, 3);
            copy_w(four, ~(it >> 2) & 1, 2 * (it & 3));
            multiply(0);
            mix_widening<4, 2, 0, 1>();
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
            __syncthreads();
            read(1 - P, 0, 0);
            read_w(it + 1, 0);
            widen_rows(0, 0, 0);
#pragma unroll
            for (int i = 0; i < 3; ++i) copy_x(second, P, i);
            multiply(1);
            mix_widening<12, 3, 12, 5>();
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_x(0, 0, i);
#pragma unroll
    for (int i = 0; i < 8; i += 2) copy_w(0, 0, i);
    copy_s(0, 0);
    if constexpr (std::is_same_v<X, f16>) {
        // whether float16 holds the tile's own rows: a thread looks at one row's scales
        const int at = own + int(threadIdx.x);
        const uint8_t *row = scales + int64_t(min(at, s.n - 1)) * ld_scales;
        const uint8_t *row_codes = codes + int64_t(min(at, s.n - 1)) * ld_codes;
        const bool holds = f16_holds([&](auto &&ok) {
            bool fine = true;
#pragma unroll 8
            for (int i = 0; i < s.k / kBlock; i += 4) {
                const uint32_t v = *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(row + i);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    fine = fine && ok(v >> (8 * e) & 255, row_codes + int64_t(i + e) * kBlockBytes);
            }
            return fine;
        });
        if (holds) run(f16{});
        else run(bf16{});
    } else {
        __syncthreads();
        run(bf16{});
    }
    pin(acc);
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");  // as settle() does
    pin(acc);
    __syncthreads();  // no copy is on its way when the block ends
    store_tile<TW>(acc, out, ld_out, m0 + wm, n0 + wn, s.m, s.n, lane, own);
}

// The gradient: dx[m][c] = sum over n of dy[m][n] w[n][c], 256 tokens by 256 columns, 64 rows n a step. The tokens'
// rows are copied as above. The matrix's codes go through registers: a thread takes eight columns of eight rows, a word
// from each, widens them, joins pairs of rows and writes each column's eight values to its row in LDS. A step's words
// are loaded a step ahead of that. Bound as above, with the columns' stores to LDS: 4,096 tokens, 8,192 rows of 4,096 in
// 219 to 236 us, 1.16 to 1.26 PFLOP/s. float16 gradients 287 to 298 us: a look at the columns' scales comes first, one after
// another.
constexpr size_t kStreamGradLds = 2 * 256 * (128 + 128);

template <typename X>
__global__ __launch_bounds__(256, 1) void k_stream_grad(const X *__restrict__ dy, int64_t ld_dy,
                                                        const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                        const uint8_t *__restrict__ scales, int64_t ld_scales,
                                                        X *__restrict__ out, int64_t ld_out, TileShape s) {
    // s: tokens, the matrix's width, its rows
    constexpr int TW = 4;
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, g = lane >> 5;
    uint32_t tm, tn;
    tile_of(s, (uint32_t(s.m) + 255) / 256, tm, tn);
    const int m0 = min(int(tm) * 256, s.m - 256), c0 = int(tn) * 256;

    const int64_t ld_b = ld_dy * 2;
    const Buffer src = buffer_of(reinterpret_cast<const uint8_t *>(dy) + (m0 + 64 * wave) * ld_b);
    const uint32_t off = uint32_t(lane >> 3) * uint32_t(ld_b), piece = 16 * ((lane & 7) ^ (lane >> 3));
    const uint32_t offs[2] = {off + piece, off + (piece ^ 16)}, rows8 = 8 * uint32_t(ld_b);
    Lds *to = (Lds *)smem + wave * 64 * 128;
    auto copy = [&](int it, int buf, int i) {
        copy16(src, offs[i & 1], uint32_t(it) * 128 + i * rows8, to + buf * 256 * 128 + i * 1024);
    };
    // columns past the last block's are not stored: any of the matrix's will do
    const int group = tid & 31, octet = tid >> 5;
    const int col = c0 + 8 * group < int(blocks_of_width(s.n)) * kBlock ? c0 + 8 * group : 0;
    const uint8_t *wp = codes + int64_t(8 * octet) * ld_codes + col / 2;
    const uint8_t *sp = scales + int64_t(8 * octet) * ld_scales + col / kBlock;
    uint32_t word[8], top[8];
    auto load = [&](int it) {
        const uint8_t *w = wp + int64_t(it) * kStepHalf * ld_codes, *b = sp + int64_t(it) * kStepHalf * ld_scales;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            word[i] = *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(w + i * ld_codes);
            top[i] = b[i * ld_scales];
        }
    };
    i32x4 *lds_w = reinterpret_cast<i32x4 *>(smem + 2 * 256 * 128);

    f32x16 acc[TW][TW] = {};
    const int wm = (wave & 1) * 128, wn = (wave >> 1) * 128;
    const int turn = (r ^ (r >> 3 & 1)) & 7;
    i32x4 q[2][TW], p[2][TW];
    auto read = [&](int buf, int set, int j) {
        const i32x4 *bx = reinterpret_cast<const i32x4 *>(smem + buf * 256 * 128), *bw = lds_w + buf * 256 * 8;
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            q[set][t] = bx[(wm + 32 * t + r) * 8 + ((4 * g + j) ^ turn)];
            p[set][t] = bw[place(wn + 32 * t + r, 4 * g + j)];
        }
    };
    const int steps = s.k / kStepHalf, last = steps - 1;
    auto run = [&](auto type) {
        using T = decltype(type);
        // columns 2 h and 2 h + 1 of the eight
        auto store = [&](int buf, int h) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = uint32_t(widen_pair<T>(word[i], scale_operand(top[i]), h));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                i32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = int32_t(__builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], c ? 0x07060302u : 0x05040100u));
                lds_w[buf * 256 * 8 + place(8 * group + 2 * h + c, octet)] = o;
            }
        };
        auto multiply = [&](int set) {
#pragma unroll
            for (int j = 0; j < TW; ++j) {
                i32x4 hi = q[set][j], lo;
                if constexpr (!std::is_same_v<T, X>) split(q[set][j], hi, lo);
#pragma unroll
                for (int i = 0; i < TW; ++i) {
                    acc[i][j] = mma32<T>(p[set][i], hi, acc[i][j]);
                    if constexpr (!std::is_same_v<T, X>) acc[i][j] = mma32<T>(finite(p[set][i]), lo, acc[i][j]);
                }
            }
        };
        load(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) copy(0, 0, i);
#pragma unroll
        for (int h = 0; h < 4; ++h) store(0, h);
        __syncthreads();
        load(min(1, last));
        read(0, 0, 0);
#pragma unroll
        for (int i = 0; i < 3; ++i) copy(min(1, last), 1, i);
        for (int it = 0; it < steps; ++it) {
            const int P = it & 1, next = min(it + 1, last), second = min(it + 2, last);
            __builtin_amdgcn_sched_barrier(0);
            read(P, 1, 1);
#pragma unroll
            for (int i = 3; i < 8; ++i) copy(next, 1 - P, i);
            multiply(0);
            mix<1, 5>();
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
            read(P, 0, 2);
            store(1 - P, 0);
            store(1 - P, 1);
            multiply(1);
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
            read(P, 1, 3);
            store(1 - P, 2);
            store(1 - P, 3);
            multiply(0);
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
            __syncthreads();
            read(1 - P, 0, 0);
            load(second);
#pragma unroll
            for (int i = 0; i < 3; ++i) copy(second, P, i);
            multiply(1);
            mix<1, 0, 3>();
            pin(acc);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if constexpr (std::is_same_v<X, f16>) {
        // whether float16 holds the tile's columns: a thread looks at a block of every 32nd row
        const int b = c0 / kBlock + (tid & 7);
        const bool holds = f16_holds([&](auto &&ok) {
            bool fine = true;
            if (b < int(blocks_of_width(s.n))) {
#pragma unroll 8
                for (int row = tid >> 3; row < s.k; row += 32)
                    fine = fine && ok(scales[int64_t(row) * ld_scales + b],
                                      codes + int64_t(row) * ld_codes + b * kBlockBytes);
            }
            return fine;
        });
        if (holds) run(f16{});
        else run(bf16{});
    } else {
        run(bf16{});
    }
    pin(acc);
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");  // as settle() does
    pin(acc);
    __syncthreads();  // no copy is on its way when the block ends
    store_tile<TW>(acc, out, ld_out, m0 + wm, c0 + wn, s.m, s.n, lane);
}

}  // namespace vspmm
