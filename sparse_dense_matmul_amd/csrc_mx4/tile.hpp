// Products with many tokens: out[m][n] = sum over k of q[m][k] p[n][k], tiles of 64 TW rows n by 64 TW tokens m, four
// waves of 32 TW x 32 TW each. The rows are the first operand of the 32 x 32 matrix instructions, so a lane's results
// are runs of four along n.
//
// A step of the contraction takes 128 bytes of a token's row (64 values of 16 bits, 256 codes of 4). Its rows lie in
// LDS as eight 16-byte chunks, chunk c of row r at place c ^ spread(r): the eight rows that eight lanes read at a time
// then lie in eight different groups of banks, and so do the rows 8 apart that the transposing store writes. Steps are
// double buffered: a step's loads go to registers before the step before it is multiplied and to LDS behind it.
//
// Lane (r, g) = (lane % 32, lane / 32) of an instruction holds 8 values of row r. Which ones is free as long as both
// operands agree: instruction j of a step takes 32 g + 8 j, so that a lane's 32 values of a step are one block of
// codes under one scale.
//
// Bound by latency where there are few tiles (load, widen, store, barrier, multiply): 37 float16 tokens through 5,003 x
// 4,001 in 22 us, the gradient of 515 through 1,111 x 2,049 in 21 us, 64 4-bit tokens through 8,192 x 4,096 in 10 us.
#pragma once

#include "few.hpp"

namespace vspmm {

constexpr int kTileThreads = 256;
constexpr int kStepHalf = 64;    // values of a step of 16-bit rows
constexpr int kStepCodes = 256;  // codes of a step of 4-bit rows

__device__ __forceinline__ int spread(int row) { return (row ^ (row >> 3)) & 7; }
__device__ __forceinline__ int place(int row, int chunk) { return row * 8 + (chunk ^ spread(row)); }

struct TileShape {
    int m, n, k;            // tokens, rows and the contraction's length
    uint32_t tiles_n;       // tiles along n
};

// A block is KS groups of four waves, each over a part of the contraction's steps with buffers of its own.
__device__ __forceinline__ int group_thread() { return int(threadIdx.x) & (kTileThreads - 1); }
__device__ __forceinline__ int group_number() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kTileThreads); }

// Steps [first, first + steps) of a group: load(step) to registers, store(buffer) from there to LDS, compute(buffer). A
// step is loaded before the barrier that opens the one before it.
template <typename Load, typename Store, typename Compute>
__device__ __forceinline__ void run_steps(int first, int steps, Load &&load, Store &&store, Compute &&compute) {
    load(first);
    store(0);
    load(first + 1);
    lds_barrier();
    for (int it = 0; it < steps; ++it) {
        compute(it & 1);
        store((it + 1) & 1);
        load(first + it + 2);
        lds_barrier();
    }
}

// The groups' sums added up in the first, in order, through LDS that nothing else uses any more.
template <int KS, int TW>
__device__ __forceinline__ void join_groups(f32x16 (&acc)[TW][TW], char *smem) {
    if constexpr (KS > 1) {
        f32x4 *parts = reinterpret_cast<f32x4 *>(smem);  // [wave][4 TW][lane] of a group at a time
        const int tid = group_thread(), group = group_number();
#pragma unroll 1
        for (int k = 1; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                __syncthreads();
                if (group == k) {
#pragma unroll
                    for (int j = 0; j < TW; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            parts[(j * 4 + e) * kTileThreads + tid] =
                                f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
                }
                __syncthreads();
                if (group == 0) {
#pragma unroll
                    for (int j = 0; j < TW; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f32x4 v = parts[(j * 4 + e) * kTileThreads + tid];
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[i][j][4 * e + c] += v[c];
                        }
                }
            }
    }
}

// Consecutive blocks go to the eight chiplets in turn; each chiplet takes a run of tiles, down strips of 8 tiles of
// tokens, so that what its L2 holds is used by neighbours.
__device__ __forceinline__ void tile_of(const TileShape &s, uint32_t tiles_m, uint32_t &tm, uint32_t &tn) {
    const uint32_t total = gridDim.x, id = blockIdx.x;
    const uint32_t x = id % 8, each = total / 8, more = total % 8;
    const uint32_t l = x * each + (x < more ? x : more) + id / 8;
    const uint32_t strip = l / (8 * s.tiles_n), in = l - strip * 8 * s.tiles_n;
    const uint32_t high = tiles_m - strip * 8 < 8 ? tiles_m - strip * 8 : 8;
    tm = strip * 8 + in % high;
    tn = in / high;
}

// The tokens' side of a step: TW * 2 chunks a thread.
template <int TW>
struct Tokens {
    const uint16_t *row[2 * TW];
    i32x4 v[2 * TW];
    int chunk;

    __device__ __forceinline__ void init(const void *x, int64_t ld, int m0, int m) {
        chunk = group_thread() & 7;
#pragma unroll
        for (int i = 0; i < 2 * TW; ++i) {
            const int r = m0 + i * 32 + (group_thread() >> 3);
            row[i] = static_cast<const uint16_t *>(x) + int64_t(r < m ? r : m - 1) * ld;
        }
    }
    __device__ __forceinline__ void load(int k0, int width) {
        const int k = k0 + 8 * chunk;
        if (k0 + kStepHalf <= width) {
#pragma unroll
            for (int i = 0; i < 2 * TW; ++i) v[i] = *reinterpret_cast<const Half16 *>(row[i] + k);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * TW; ++i) v[i] = load_half(row[i], k, width);
        }
    }
    __device__ __forceinline__ void store(i32x4 *lds) const {
#pragma unroll
        for (int i = 0; i < 2 * TW; ++i) lds[place(i * 32 + (group_thread() >> 3), chunk)] = v[i];
    }
};

// The same for 4-bit rows, with their scales: eight bytes a row and step.
template <int TW>
struct Codes {
    static constexpr int kEdge = 64 * TW;
    const uint8_t *row[2 * TW], *tops;
    i32x4 v[2 * TW];
    uint32_t s[2];
    int chunk, blocks;

    __device__ __forceinline__ void init(const uint8_t *codes, int64_t ld, const uint8_t *scales, int64_t ld_scales,
                                         int r0, int rows, int width) {
        chunk = group_thread() & 7;
        blocks = int(blocks_of_width(width));
#pragma unroll
        for (int i = 0; i < 2 * TW; ++i) {
            const int r = r0 + i * 32 + (group_thread() >> 3);
            row[i] = codes + int64_t(r < rows ? r : rows - 1) * ld;
        }
        const int r = r0 + group_thread();
        tops = scales + int64_t(r < rows ? r : rows - 1) * ld_scales;
    }
    __device__ __forceinline__ void load(int b0) {
        const bool here = b0 + chunk < blocks;
#pragma unroll
        for (int i = 0; i < 2 * TW; ++i)
            v[i] = here ? *reinterpret_cast<const Byte16 *>(row[i] + int64_t(b0 + chunk) * kBlockBytes) : i32x4{};
        if (group_thread() >= kEdge) return;
        if (b0 + 8 <= blocks) {
            using Two = uint32_t __attribute__((ext_vector_type(2), aligned(1)));
            const Two t = *reinterpret_cast<const Two *>(tops + b0);
            s[0] = t[0], s[1] = t[1];
        } else {
            s[0] = s[1] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (b0 + i < blocks) s[i / 4] |= uint32_t(tops[b0 + i]) << (8 * (i & 3));
        }
    }
    __device__ __forceinline__ void store(i32x4 *lds, uint2 *lds_s) const {
#pragma unroll
        for (int i = 0; i < 2 * TW; ++i) lds[place(i * 32 + (group_thread() >> 3), chunk)] = v[i];
        if (group_thread() < kEdge) lds_s[group_thread()] = make_uint2(s[0], s[1]);
    }
};

// Results to out: out[m][n .. n + 3] for each run of four; columns before `from` are another tile's.
template <int TW, typename O>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[TW][TW], O *out, int64_t ld, int m0, int n0, int m, int n,
                                           int lane, int from = 0) {
    using V = Vec<O, 4>;
#pragma unroll
    for (int j = 0; j < TW; ++j) {
        const int mm = m0 + 32 * j + (lane & 31);
        if (mm >= m) continue;
        O *row = out + int64_t(mm) * ld;
#pragma unroll
        for (int i = 0; i < TW; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int nn = n0 + 32 * i + 8 * q + 4 * (lane >> 5);
                V v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = rounded<O>(acc[i][j][4 * q + e]);
                if (nn + 4 <= n && nn >= from) {
                    *reinterpret_cast<V *>(row + nn) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nn + e < n && nn + e >= from) row[nn + e] = v[e];
                }
            }
    }
}

// One instruction's worth of every tile of a wave. HALVES: the tokens in two bfloat16 parts.
template <typename T, bool HALVES, int TW>
__device__ __forceinline__ void multiply_tiles(f32x16 (&acc)[TW][TW], const i32x4 (&p)[TW], const i32x4 (&q)[TW]) {
#pragma unroll
    for (int j = 0; j < TW; ++j) {
        if constexpr (HALVES) {
            i32x4 hi, lo;
            split(q[j], hi, lo);
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                acc[i][j] = mma32<bf16>(p[i], hi, acc[i][j]);
                i32x4 rows = p[i];
                asm volatile("" : "+v"(rows));  // found anew for each j, not kept in registers between
                acc[i][j] = mma32<bf16>(finite(rows), lo, acc[i][j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < TW; ++i) acc[i][j] = mma32<T>(p[i], q[j], acc[i][j]);
        }
    }
}

// ---------------------------------------------------------------- 16-bit tokens, 4-bit rows

// A step's codes are two 16-byte blocks a row, at [tile of 32 rows][block][row]: a wave's reads are one run of 1 KB.
template <int TW>
constexpr size_t tile_lds() {  // bytes: two buffers of tokens, codes and scales
    return size_t(2) * 64 * TW * (128 + 32 + 2);
}

template <int TW, int KS, typename X, typename O>
__global__ __launch_bounds__(kTileThreads *KS) void k_tile(const X *__restrict__ x, int64_t ld_x,
                                                       const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                       const uint8_t *__restrict__ scales, int64_t ld_scales,
                                                       O *__restrict__ out, int64_t ld_out, TileShape s) {
    constexpr int EDGE = 64 * TW, SLOTS = EDGE * 2;  // 16-byte blocks of codes of a step
    constexpr int OWN = SLOTS / kTileThreads > 0 ? SLOTS / kTileThreads : 1;
    extern __shared__ __align__(16) char smem[];
    i32x4 *lds_x = reinterpret_cast<i32x4 *>(smem + group_number() * tile_lds<TW>());
    i32x4 *lds_w = lds_x + 2 * EDGE * 8;
    uint16_t *lds_s = reinterpret_cast<uint16_t *>(lds_w + 2 * SLOTS);
    const int tid = group_thread(), lane = tid & 63, wave = tid >> 6;
    const int r = lane & 31, g = lane >> 5;
    uint32_t tm, tn;
    tile_of(s, (uint32_t(s.m) + EDGE - 1) / EDGE, tm, tn);
    const int m0 = int(tm) * EDGE, n0 = int(tn) * EDGE;
    const int blocks = int(blocks_of_width(s.k));

    Tokens<TW> tok;
    tok.init(x, ld_x, m0, s.m);
    const uint8_t *wrow[OWN], *srow;
    i32x4 wv[OWN];
    uint32_t sv;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int slot = i * kTileThreads + tid;  // [row / 32][block][row % 32]
        const int row = n0 + (slot >> 6) * 32 + (slot & 31);
        wrow[i] = codes + int64_t(row < s.n ? row : s.n - 1) * ld_codes;
    }
    {
        const int row = n0 + tid;
        srow = scales + int64_t(row < s.n ? row : s.n - 1) * ld_scales;
    }
    const bool own_w = tid < SLOTS, own_s = tid < EDGE;
    const int wb = (tid >> 5) & 1;
    auto load = [&](int it) {
        tok.load(it * kStepHalf, s.k);
        const int b = 2 * it;
        if (own_w) {
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                wv[i] = b + wb < blocks
                               ? *reinterpret_cast<const Byte16 *>(wrow[i] + int64_t(b + wb) * kBlockBytes)
                               : i32x4{};
        }
        if (own_s) {
            // in one load: joining two would wait for them here
            if (b + 2 <= blocks) sv = *reinterpret_cast<const uint16_t __attribute__((aligned(1))) *>(srow + b);
            else sv = (b < blocks ? uint32_t(srow[b]) : 127u) | 127u << 8;
        }
    };
    auto store = [&](int buf) {
        tok.store(lds_x + buf * EDGE * 8);
        if (own_w) {
#pragma unroll
            for (int i = 0; i < OWN; ++i) lds_w[buf * SLOTS + i * kTileThreads + tid] = wv[i];
        }
        if (own_s) lds_s[buf * EDGE + tid] = uint16_t(sv);
    };

    f32x16 acc[TW][TW] = {};
    const int wm = (wave & 1) * 32 * TW, wn = (wave >> 1) * 32 * TW;
    // each group has as many steps as the first: those past the end are zeros
    const int all = (s.k + kStepHalf - 1) / kStepHalf, steps = (all + KS - 1) / KS, first = group_number() * steps;
    auto run = [&](auto type) {
        using T = decltype(type);
        run_steps(first, steps, load, store, [&](int buf) {
            const i32x4 *bx = lds_x + buf * EDGE * 8, *bw = lds_w + buf * SLOTS;
            i32x4 c[TW];
            float sc[TW];
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                c[i] = bw[(wn / 32 + i) * 64 + lane];
                sc[i] = scale_operand(reinterpret_cast<const uint8_t *>(lds_s + buf * EDGE + wn + 32 * i + r)[g]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                i32x4 p[TW], q[TW];
#pragma unroll
                for (int t = 0; t < TW; ++t) q[t] = bx[place(wm + 32 * t + r, 4 * g + j)];
#pragma unroll
                for (int i = 0; i < TW; ++i) p[i] = widen<T>(uint32_t(c[i][j]), sc[i]);
                multiply_tiles<T, !std::is_same_v<T, X>, TW>(acc, p, q);
            }
        });
    };
    if constexpr (std::is_same_v<X, f16>) {
        // float16 tokens meet the rows in float16 where it holds the tile's, else in two bfloat16 parts in bfloat16: the
        // block's threads share the rows' scales
        const int rows = min(EDGE, s.n - n0);
        const bool holds = f16_holds([&](auto &&ok) {
            bool fine = true;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < int64_t(rows) * blocks; i += kTileThreads * KS)
                fine = fine && ok(scales[(n0 + i / blocks) * ld_scales + i % blocks],
                                  codes + (n0 + i / blocks) * ld_codes + i % blocks * kBlockBytes);
            return fine;
        });
        if (holds) run(f16{});
        else run(bf16{});
    } else {
        run(bf16{});
    }
    settle(acc);
    join_groups<KS>(acc, smem);
    if (group_number() > 0) return;
    store_tile<TW>(acc, out, ld_out, m0 + wm, n0 + wn, s.m, s.n, lane);
}

// ---------------------------------------------------------------- the gradient

template <int TW>
constexpr size_t grad_lds() {  // bytes: two buffers of the gradient's rows and of widened columns
    return size_t(2) * 64 * TW * 256;
}

// dx[m][c] = sum over n of dy[m][n] w[n][c]: the matrix's columns c are the rows of the tile, widened on their
// way to LDS: a thread takes eight columns of eight rows n, a word of codes from each, and pairs of rows joined make each
// column's eight values 16 bytes of its LDS row. float16 gradients meet them in float16 where it holds the tile's
// columns, else, in two bfloat16 parts, in bfloat16, which holds every value.
template <int TW, int KS, typename X>
__global__ __launch_bounds__(kTileThreads *KS) void k_tile_grad(const X *__restrict__ dy, int64_t ld_dy,
                                                            const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                            const uint8_t *__restrict__ scales, int64_t ld_scales,
                                                            X *__restrict__ out, int64_t ld_out, TileShape s) {
    // s: tokens, the matrix's width, its rows
    constexpr int EDGE = 64 * TW;
    constexpr int GROUPS = EDGE / 8;  // groups of eight columns
    extern __shared__ __align__(16) char smem[];
    i32x4 *lds_x = reinterpret_cast<i32x4 *>(smem + group_number() * grad_lds<TW>());
    i32x4 *lds_w = lds_x + 2 * EDGE * 8;
    const int tid = group_thread(), lane = tid & 63, wave = tid >> 6;
    const int r = lane & 31, g = lane >> 5;
    uint32_t tm, tn;
    tile_of(s, (uint32_t(s.m) + EDGE - 1) / EDGE, tm, tn);
    const int m0 = int(tm) * EDGE, c0 = int(tn) * EDGE;

    Tokens<TW> tok;
    tok.init(dy, ld_dy, m0, s.m);
    const int group = tid % GROUPS, octet = tid / GROUPS;  // octet >= 8: the thread has none
    const bool own = octet < 8;
    // columns from the width on: the last block's, whose results are not stored
    const int blocks = int(blocks_of_width(s.n));
    const int col = c0 + 8 * group < blocks * kBlock ? c0 + 8 * group : 0;
    const uint8_t *wp = codes + col / 2, *sp = scales + col / kBlock;
    uint32_t word[8], top[8];
    auto load = [&](int it) {
        tok.load(it * kStepHalf, s.k);
        if (!own) return;
        const int row0 = it * kStepHalf + 8 * octet;
        const uint8_t *w = wp + row0 * ld_codes, *b = sp + row0 * ld_scales;
        if (row0 + 8 <= s.k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                word[i] = *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(w + i * ld_codes);
                top[i] = b[i * ld_scales];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                word[i] = 0;
                top[i] = 127;
                if (row0 + i < s.k) {
                    word[i] = *reinterpret_cast<const uint32_t __attribute__((aligned(1))) *>(w + i * ld_codes);
                    top[i] = b[i * ld_scales];
                }
            }
        }
    };
    f32x16 acc[TW][TW] = {};
    const int wm = (wave & 1) * 32 * TW, wn = (wave >> 1) * 32 * TW;
    // each group has as many steps as the first: those past the end are zeros
    const int all = (s.k + kStepHalf - 1) / kStepHalf, steps = (all + KS - 1) / KS, first = group_number() * steps;
    auto run = [&](auto type) {
        using T = decltype(type);
        auto store = [&](int buf) {
            tok.store(lds_x + buf * EDGE * 8);
            if (!own) return;
            i32x4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = widen<T>(word[i], scale_operand(top[i]));
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                i32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = int32_t(__builtin_amdgcn_perm(uint32_t(v[2 * i + 1][c / 2]), uint32_t(v[2 * i][c / 2]),
                                                         c & 1 ? 0x07060302u : 0x05040100u));
                lds_w[buf * EDGE * 8 + place(8 * group + c, octet)] = o;
            }
        };
        auto compute = [&](int buf) {
            const i32x4 *bx = lds_x + buf * EDGE * 8, *bw = lds_w + buf * EDGE * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                i32x4 p[TW], q[TW];
#pragma unroll
                for (int t = 0; t < TW; ++t) q[t] = bx[place(wm + 32 * t + r, 4 * g + j)];
#pragma unroll
                for (int t = 0; t < TW; ++t) p[t] = bw[place(wn + 32 * t + r, 4 * g + j)];
                multiply_tiles<T, !std::is_same_v<T, X>, TW>(acc, p, q);
            }
        };
        run_steps(first, steps, load, store, compute);
    };
    if constexpr (std::is_same_v<X, f16>) {
        // whether float16 holds the tile's columns: the block's threads share their scales
        constexpr int TOPS = EDGE / kBlock;
        const bool holds = f16_holds([&](auto &&ok) {
            bool fine = true;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < int64_t(s.k) * TOPS; i += kTileThreads * KS) {
                const int b = c0 / kBlock + int(i % TOPS);
                fine = fine && (b >= blocks || ok(scales[i / TOPS * ld_scales + b],
                                                  codes + i / TOPS * ld_codes + b * kBlockBytes));
            }
            return fine;
        });
        if (holds) run(f16{});
        else run(bf16{});
    } else {
        run(bf16{});
    }
    settle(acc);
    join_groups<KS>(acc, smem);
    if (group_number() > 0) return;
    store_tile<TW>(acc, out, ld_out, m0 + wm, c0 + wn, s.m, s.n, lane);
}

// ---------------------------------------------------------------- 4-bit tokens, 4-bit rows

template <int TW>
constexpr size_t both_lds() {  // bytes: two buffers of both sides' codes and scales
    return size_t(2) * 64 * TW * 2 * (128 + 8);
}

template <int TW, int KS, typename O>
__global__ __launch_bounds__(kTileThreads *KS) void k_tile_both(const uint8_t *__restrict__ x_codes, int64_t ld_x,
                                                            const uint8_t *__restrict__ x_scales, int64_t ld_xs,
                                                            const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                            const uint8_t *__restrict__ scales, int64_t ld_scales,
                                                            O *__restrict__ out, int64_t ld_out, TileShape s) {
    constexpr int EDGE = 64 * TW;
    extern __shared__ __align__(16) char smem[];
    i32x4 *lds_x = reinterpret_cast<i32x4 *>(smem + group_number() * both_lds<TW>());
    i32x4 *lds_w = lds_x + 2 * EDGE * 8;
    uint2 *lds_xs = reinterpret_cast<uint2 *>(lds_w + 2 * EDGE * 8);
    uint2 *lds_ws = lds_xs + 2 * EDGE;
    const int lane = group_thread() & 63, wave = group_thread() >> 6;
    const int r = lane & 31, g = lane >> 5;
    uint32_t tm, tn;
    tile_of(s, (uint32_t(s.m) + EDGE - 1) / EDGE, tm, tn);
    const int m0 = int(tm) * EDGE, n0 = int(tn) * EDGE;

    Codes<TW> cx, cw;
    cx.init(x_codes, ld_x, x_scales, ld_xs, m0, s.m, s.k);
    cw.init(codes, ld_codes, scales, ld_scales, n0, s.n, s.k);
    auto load = [&](int it) {
        cx.load(8 * it);
        cw.load(8 * it);
    };
    auto store = [&](int buf) {
        cx.store(lds_x + buf * EDGE * 8, lds_xs + buf * EDGE);
        cw.store(lds_w + buf * EDGE * 8, lds_ws + buf * EDGE);
    };

    f32x16 acc[TW][TW] = {};
    const int wm = (wave & 1) * 32 * TW, wn = (wave >> 1) * 32 * TW;
    // block 2 j + g of a row's eight scales to byte j
    const uint32_t pick = 0x06040200u + uint32_t(g) * 0x01010101u;
    auto compute = [&](int buf) {
        const i32x4 *bx = lds_x + buf * EDGE * 8, *bw = lds_w + buf * EDGE * 8;
        uint32_t sx[TW], sw[TW];
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            const uint2 a = lds_xs[buf * EDGE + wm + 32 * t + r], b = lds_ws[buf * EDGE + wn + 32 * t + r];
            sx[t] = __builtin_amdgcn_perm(a.y, a.x, pick);
            sw[t] = __builtin_amdgcn_perm(b.y, b.x, pick);
        }
        auto part = [&](auto index) {
            constexpr int J = decltype(index)::value;
            i32x4 p[TW], q[TW];
#pragma unroll
            for (int t = 0; t < TW; ++t) q[t] = bx[place(wm + 32 * t + r, 2 * J + g)];
#pragma unroll
            for (int t = 0; t < TW; ++t) p[t] = bw[place(wn + 32 * t + r, 2 * J + g)];
#pragma unroll
            for (int j = 0; j < TW; ++j)
#pragma unroll
                for (int i = 0; i < TW; ++i) acc[i][j] = mma32_mx4<J>(p[i], sw[i], q[j], sx[j], acc[i][j]);
        };
        part(std::integral_constant<int, 0>{});
        part(std::integral_constant<int, 1>{});
        part(std::integral_constant<int, 2>{});
        part(std::integral_constant<int, 3>{});
    };

    // each group has as many steps as the first: those past the end are zeros
    const int all = (s.k + kStepCodes - 1) / kStepCodes, steps = (all + KS - 1) / KS, first = group_number() * steps;
    run_steps(first, steps, load, store, compute);
    settle(acc);
    join_groups<KS>(acc, smem);
    if (group_number() > 0) return;
    store_tile<TW>(acc, out, ld_out, m0 + wm, n0 + wn, s.m, s.n, lane);
}

}  // namespace vspmm
