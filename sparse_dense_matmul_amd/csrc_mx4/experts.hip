// A whole mixture-of-experts layer for a few tokens in two launches: each token's experts' gated two-layer products,
// weighted and summed. Declared in include/vspmm.h.
//
// The work is reading the weights of every expert that a token is sent to, once. The first launch takes 16 hidden
// units of one expert for all its tokens (a block finds its expert, the a-th of those in use, and its tokens in the
// list of choices by itself) and writes act(gate x) (up x) times the router's weight. The second takes 16 columns of
// the result a block and sums over all experts in use; where there are few columns several blocks share them and the
// last adds their parts, in order. Every sum's order is fixed. Hidden values go between the launches as the sum of three
// bfloat16 numbers, which hold float32's 24 bits and which the second launch's matrix instructions take as they are.
//
// 64 tokens to 8 of 128 experts of 4,096 x 1,024, bfloat16: 419 and 267 us, 5.0 and 3.9 TB/s of weights; the second is
// bound by the hidden values, which every 16 columns read again, 6 bytes each (two parts of 17 bits: 235 us). One token, 4
// bits: 14 and 10 us, latency: 7.5 us of bytes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "few.hpp"
#include "host.hpp"

using namespace vspmm;

namespace {

constexpr int kTokensMax = 1024;
constexpr int kExpertsMax = 4096;
constexpr int kLogWaves = 3;
constexpr int kUpWaves = 1 << kLogWaves;  // of a block of the first launch
constexpr int kDownWaves = 8;             // of a block of the second
constexpr int kSplitsMax = 8;
constexpr size_t kStageMax = 48 * 1024;  // bytes of staged tokens that leave room for two blocks

// ------------------------------------------------------------------ kernels

struct Choices {
    const void *ids;  // [tokens, top_k], int32 or int64
    bool wide;
    const float *weights;
    int tokens, top_k, experts;
    __device__ __forceinline__ int expert(int slot) const {  // -1: none
        const int64_t e = wide ? static_cast<const int64_t *>(ids)[slot] : static_cast<const int32_t *>(ids)[slot];
        return e >= 0 && e < experts ? int(e) : -1;
    }
};

// Between the launches: how many experts are in use, which, how many of each group of kGroup tokens are sent to each and
// which, in order, with a slot of each (a token sent twice to an expert is listed once, with both weights), and the
// hidden values by slot, in whole chunks with zeros at the end. With few choices the second launch finds all but the
// hidden values by itself.
constexpr int kGroup = 128;
struct Between {
    int *count, *expert;  // [1], [most]
    int *counts;          // [most, groups]
    int2 *list;           // [most, groups, kGroup]: token, slot
    bf16 *hidden;         // [slots, padded / 8, part, 8]
    int64_t padded;
    int groups;
    // of a result whose experts are split over blocks: the parts, [splits, tokens, tiles, 16], and how many have come
    float *parts;
    int *arrived;  // [groups, tiles], zeroed by the first launch
    int tiles, splits;

    __device__ __forceinline__ void reset() const {
        if (splits > 1 && blockIdx.x == 0 && blockIdx.y == 0)
            for (int i = threadIdx.x; i < groups * tiles; i += blockDim.x) arrived[i] = 0;
    }
};

// Up to 64 choices of up to 16 tokens: a wave holds them all, one a lane, and finds the experts in use, in order of
// their first choice, and an expert's tokens by ballots.
struct Few {
    int expert;      // the lane's choice, -1: none
    float weight;    // and its weight
    uint64_t first;  // the lanes whose expert none before has chosen
    int top_k;

    __device__ __forceinline__ Few(const Choices &ch, int lane) : expert(-1), weight(0.0f), top_k(ch.top_k) {
        const int slots = ch.tokens * ch.top_k;
        if (lane < slots) expert = ch.expert(lane), weight = ch.weights[lane];
        bool again = expert < 0;
        for (int s = 0; s < slots; ++s) again = again || (lane > s && expert == __builtin_amdgcn_readlane(expert, s));
        first = __ballot(!again);
    }
    __device__ __forceinline__ int count() const { return __popcll(first); }
    // the a-th expert in use
    __device__ __forceinline__ int number(int a) const {
        uint64_t m = first;
        for (; a > 0; --a) m &= m - 1;
        return __builtin_amdgcn_readlane(expert, __builtin_ctzll(m));
    }
    // how many tokens expert e has; in lane r its r-th token and that one's choices of it, as bits from the first on
    __device__ __forceinline__ int tokens(int e, int lane, int &token, uint64_t &choices) const {
        const uint64_t all = __ballot(expert == e);
        const uint64_t own = top_k < 64 ? (uint64_t(1) << top_k) - 1 : ~uint64_t(0);
        const bool has = lane * top_k < 64 && (all >> (lane * top_k) & own) != 0;
        const uint64_t here = __ballot(has);
        const int rank = __popcll(here & ((uint64_t(1) << lane) - 1));
        token = __builtin_amdgcn_ds_permute((has ? rank : 63) * 4, lane);  // lane 63 has no token of 16
        choices = lane < __popcll(here) ? all >> (token * top_k) & own : 0;
        return __popcll(here);
    }
};

template <typename T>
struct Matrix {  // [experts, rows, width]
    const T *p;
    int64_t ld, stride;
    __device__ __forceinline__ Row<T> row(int64_t e, int64_t r) const { return {p + e * stride + r * ld}; }
};
template <>
struct Matrix<Mx4> {
    const uint8_t *codes, *scales;
    int64_t ld, stride, ld_scales, stride_scales;
    __device__ __forceinline__ Row<Mx4> row(int64_t e, int64_t r) const {
        return {codes + e * stride + r * ld, scales + e * stride_scales + r * ld_scales};
    }
};

template <bool GELU>
__device__ __forceinline__ float activate(float g) {
    if constexpr (GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
    else return g / (1.0f + expf(-g));
}

// The hidden values of 16 units of the weights' rows f0 .. for a tile of 16 tokens from the waves' parts, by one wave:
// lane (r, g) has token r's units f0 + 4 g .. + 3.
template <bool GELU>
__device__ __forceinline__ void store_hidden(const f32x4 (*parts)[2][64], int waves, int lane, int f0, int hidden,
                                             int slot, float weight, const Between &to) {
    f32x4 sg{}, su{};
#pragma unroll
    for (int v = 0; v < kUpWaves; ++v) {  // all loaded at once: those of other runs count as zeros
        const int from = min(v, waves - 1);
        const f32x4 a = parts[from][0][lane], b = parts[from][1][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sg[i] += v < waves ? a[i] : 0.0f, su[i] += v < waves ? b[i] : 0.0f;
    }
    const int f = f0 + 4 * (lane >> 4);
    bf16 *row = to.hidden + at_planes(slot * to.padded);
    bf16x4 hi, mid, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float h = f + i < hidden ? weight * (activate<GELU>(sg[i]) * su[i]) : 0.0f;
        // Eight bits of the significand, the next eight and the last, each with h's sign: exact down to bfloat16's least
        // number, 2^-133. An infinity or NaN has the first part alone.
        const float top = __uint_as_float(__float_as_uint(h) & 0xffff0000u), rest = __builtin_isfinite(h) ? h - top : 0.0f;
        const float next = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
        hi[i] = bf16(top);
        mid[i] = bf16(next);
        lo[i] = bf16(rest - next);
    }
    const auto store = [&](int64_t k, bf16x4 a, bf16x4 b, bf16x4 c) {
        bf16 *p = row + at_planes(k & ~int64_t(7)) + (k & 7);
        *reinterpret_cast<bf16x4 *>(p) = a;
        *reinterpret_cast<bf16x4 *>(p + 8) = b;
        *reinterpret_cast<bf16x4 *>(p + 16) = c;
    };
    store(f, hi, mid, lo);
    if (f0 + 16 >= hidden)  // zeros to the end of the last chunk
        for (int64_t k = f + 16; k < to.padded; k += 16) store(k, bf16x4{}, bf16x4{}, bf16x4{});
}

// 4-bit rows and float16 tokens, multiplied in either type, need more than the 128 registers that let two blocks share a
// compute unit (which takes the first launch of 13 tokens through 39 experts of 1,008 x 736 from 50 to 40 us).
template <typename W, typename X>
constexpr bool kWide = std::is_same_v<W, Mx4> && std::is_same_v<X, f16>;

// `share` of a block's waves take 16 hidden units of one expert, an equal part of the contraction each, so that the
// block has kUpWaves / share runs of units at once; it does so `own` times. ALL: `share` is all of them, which as a
// constant takes 64 tokens to 8 of 128 experts of 4,096 x 1,024 from 460 to 415 us. Fewer share narrow tokens, so that
// each wave has two chunks or more (13 tokens to 4 of 60 experts of 256 x 2,048: 24 us, 112 with all).
template <typename W, typename X, bool GELU, int MT, bool ALL>
__global__ __launch_bounds__(64 * kUpWaves, (MT == 1 && !kWide<W, X> ? 4 : 1)) void k_experts_up(Choices ch, const X *__restrict__ x, int64_t ld_x,
                                                              Matrix<W> gate, Matrix<W> up, int width, int hidden,
                                                              int log_share, int own, Between to) {
    __shared__ uint32_t used[kExpertsMax / 32];
    constexpr int RUNS = MT == 1 ? 1 : kTokensMax / 64 / kUpWaves;  // one tile: no more than 16 tokens
    __shared__ int s_expert, s_total, s_counts[RUNS * kUpWaves];
    __shared__ int s_slot[RUNS * kUpWaves * 64];
    __shared__ float s_weight[RUNS * kUpWaves * 64];
    __shared__ uint16_t s_token[RUNS * kUpWaves * 64];
    __shared__ f32x4 parts[2][kUpWaves][2][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slots = ch.tokens * ch.top_k, a = blockIdx.y;
    to.reset();

    // the experts in use as bits, and the a-th of them
    const int words = (ch.experts + 31) / 32;
    for (int i = tid; i < words; i += 64 * kUpWaves) used[i] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += 64 * kUpWaves) {
        const int e = ch.expert(i);
        if (e >= 0) atomicOr(&used[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (wave == 0) {
        const uint32_t w0 = 2 * lane < words ? used[2 * lane] : 0, w1 = 2 * lane + 1 < words ? used[2 * lane + 1] : 0;
        const int own_bits = __popc(w0) + __popc(w1);
        int before = own_bits;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int t = __shfl_up(before, d);
            if (lane >= d) before += t;
        }
        if (lane == 63) s_total = before;
        before -= own_bits;
        if (a >= before && a < before + own_bits) {
            int left = a - before, at = 64 * lane;
            uint32_t w = w0;
            if (left >= __popc(w0)) left -= __popc(w0), at += 32, w = w1;
            for (; left > 0; --left) w &= w - 1;
            s_expert = at + __ffs(int(w)) - 1;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && a == 0 && tid == 0) *to.count = s_total;
    if (a >= s_total) return;
    const int e = s_expert;

    // its tokens in order, each with its first slot here and the sum of its weights
    int slot[RUNS];
    float weight[RUNS];
    uint64_t here[RUNS];
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int t = (i * kUpWaves + wave) * 64 + lane;
        slot[i] = -1;
        weight[i] = 0.0f;
        if (t < ch.tokens) {
            for (int k = 0; k < ch.top_k; ++k) {
                const int s = t * ch.top_k + k;
                if (ch.expert(s) != e) continue;
                weight[i] = slot[i] < 0 ? ch.weights[s] : weight[i] + ch.weights[s];
                if (slot[i] < 0) slot[i] = s;
            }
        }
        here[i] = __ballot(slot[i] >= 0);
        if (lane == 0) s_counts[i * kUpWaves + wave] = __popcll(here[i]);
    }
    __syncthreads();
    const bool list = blockIdx.x == 0;  // this block writes the expert's list
    if (list && tid == 0) to.expert[a] = e;
    if (list && tid < to.groups)
        to.counts[int64_t(a) * to.groups + tid] = s_counts[2 * tid] + s_counts[2 * tid + 1];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int run = i * kUpWaves + wave;
        int at = 0;
        for (int c = 0; c < run; ++c) at += s_counts[c];
        if (slot[i] >= 0) {
            const int rank = __popcll(here[i] & ((uint64_t(1) << lane) - 1));
            s_token[at + rank] = uint16_t(run * 64 + lane);
            s_slot[at + rank] = slot[i];
            s_weight[at + rank] = weight[i];
            if (list)
                to.list[(int64_t(a) * to.groups + run / 2) * kGroup + rank + (run & 1 ? s_counts[run - 1] : 0)] =
                    make_int2(run * 64 + lane, slot[i]);
        }
    }
    for (int c = 0; c < RUNS * kUpWaves; ++c) mine += s_counts[c];
    __syncthreads();

    const int r = lane & 15, g = lane >> 4;
    const int chunks = (width + kChunkK - 1) / kChunkK;
    if constexpr (ALL) log_share = kLogWaves;
    const int share = 1 << log_share, sub = wave & (share - 1), lead = wave - sub;
    const int at_once = 16 * kUpWaves >> log_share;
    const int c0 = chunks * sub >> log_share, c1 = chunks * (sub + 1) >> log_share;
    int set = 0;
    for (int i = 0; i < own; ++i) {
        const int64_t start = (int64_t(blockIdx.x) * own + i) * at_once;
        if (start >= hidden) return;
        const int f0 = int(start) + 16 * (wave >> log_share), f = min(f0 + r, hidden - 1);
        const Row<W> rows[2] = {gate.row(e, f), up.row(e, f)};
        // up to 16 N tokens from `first` on
        auto pass = [&](auto mt, auto in_flight, int first) {
            constexpr int N = decltype(mt)::value;
            Row<X> tokens[N];
            const int tiles = min(N, (mine - first + 15) / 16);
#pragma unroll
            for (int m = 0; m < N; ++m)
                tokens[m] = {x + int64_t(s_token[min(first + 16 * m + r, mine - 1)]) * ld_x};
            f32x4 acc[2][N] = {};
            accumulate<decltype(in_flight)::value>(acc, rows, tokens, c0, c1, width, g);
#pragma unroll
            for (int m = 0; m < N; ++m) {
                if (m >= tiles) continue;
                // two sets in turn: who writes one again has passed the barrier behind its reading
                parts[set][wave][0][lane] = acc[0][m];
                parts[set][wave][1][lane] = acc[1][m];
                lds_barrier();
                const int at = first + 16 * m + r;
                if (sub == (set & (share - 1)) && at < mine && f0 < hidden)
                    store_hidden<GELU>(&parts[set][lead], share, lane, f0, hidden, s_slot[at], s_weight[at], to);
                set ^= 1;
            }
        };
        using std::integral_constant;
        for (int first = 0; first < mine; first += 16 * MT) {
            if (MT > 1 && mine - first > 16) pass(integral_constant<int, MT>{}, integral_constant<int, 1>{}, first);
            else pass(integral_constant<int, 1>{}, integral_constant<int, (std::is_same_v<W, Mx4> ? 4 : 2)>{}, first);
        }
    }
}

// A row of staged tokens: whole chunks, and 16 bytes so that the rows' starts lie in different banks.
__host__ __device__ constexpr int staged_row(int width) { return (width + kChunkK - 1) / kChunkK * kChunkK + 8; }
__host__ __device__ constexpr int staged_planes(int width) { return 3 * ((width + kChunkK - 1) / kChunkK * kChunkK) + 8; }

// The same with few choices: no list is built, and the weights are under way after one load. STAGE: the expert's tokens
// go to LDS first.
template <typename W, typename X, bool GELU, bool STAGE, bool ALL>
__global__ __launch_bounds__(64 * kUpWaves, (STAGE || !kWide<W, X> ? 4 : 1)) void k_experts_up_few(Choices ch, const X *__restrict__ x, int64_t ld_x,
                                                                     Matrix<W> gate, Matrix<W> up, int width, int hidden,
                                                                     int log_share, Between to) {
    extern __shared__ __align__(16) char smem[];  // the staged tokens
    __shared__ f32x4 parts[kUpWaves][2][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    to.reset();
    const Few few(ch, lane);
    if (int(blockIdx.y) >= few.count()) return;
    const int e = few.number(blockIdx.y);
    int token;
    uint64_t choices;
    const int mine = few.tokens(e, lane, token, choices);
    if constexpr (ALL) log_share = kLogWaves;
    const int share = 1 << log_share, sub = wave & (share - 1);
    const int f0 = 16 * (int(blockIdx.x) * (kUpWaves >> log_share) + (wave >> log_share));
    const int f = min(f0 + r, hidden - 1);
    const int chunks = (width + kChunkK - 1) / kChunkK;
    const Row<W> rows[2] = {gate.row(e, f), up.row(e, f)};
    f32x4 acc[2][1] = {};
    const int c0 = chunks * sub >> log_share, c1 = chunks * (sub + 1) >> log_share;
    constexpr int U = std::is_same_v<W, Mx4> ? 4 : 2;
    if constexpr (STAGE) {
        const int row = staged_row(width);
        X *staged = reinterpret_cast<X *>(smem);
        for (int t = 0; t < mine; ++t) {
            const uint16_t *from = reinterpret_cast<const uint16_t *>(x + int64_t(__shfl(token, t)) * ld_x);
            for (int k = 8 * int(threadIdx.x); k < chunks * kChunkK; k += 8 * 64 * kUpWaves)
                *reinterpret_cast<i32x4 *>(staged + t * row + k) = load_half(from, k, width);
        }
        lds_barrier();
        const Row<Staged<X>> tokens[1] = {{(LdsPtr<X>)(staged) + min(r, mine - 1) * row}};
        accumulate<U>(acc, rows, tokens, c0, c1, width, g);
    } else {
        const Row<X> tokens[1] = {{x + int64_t(__shfl(token, min(r, mine - 1))) * ld_x}};
        accumulate<U>(acc, rows, tokens, c0, c1, width, g);
    }
    parts[wave][0][lane] = acc[0][0];
    parts[wave][1][lane] = acc[1][0];
    __syncthreads();
    if (sub > 0 || f0 >= hidden) return;
    token = __shfl(token, r);
    choices = uint64_t(uint32_t(__shfl(int(choices >> 32), r))) << 32 | uint32_t(__shfl(int(choices), r));
    const int at = token * ch.top_k, slot = at + __builtin_ctzll(choices | uint64_t(1) << 63);
    float weight = __shfl(few.weight, slot);
    for (uint64_t more = choices & (choices - 1); __any(more != 0); more &= more - 1) {
        const float w = __shfl(few.weight, at + __builtin_ctzll(more | uint64_t(1) << 63));
        if (more) weight += w;
    }
    if (r >= mine) return;
    store_hidden<GELU>(&parts[wave], share, lane, f0, hidden, slot, weight, to);
}

// A wave takes an equal run of the contraction over (expert in use, chunk of hidden units) for 16 columns, the tokens
// of an expert 16 MT at a time, and adds each expert's results to its own sums of every token, in LDS. FEW: as above.
// STAGE: the hidden values of all slots go to LDS first.
template <typename W, typename X, int MT, bool FEW, bool STAGE>
__global__ __launch_bounds__(64 * kDownWaves) void k_experts_down(Choices ch, Between from, Matrix<W> down, int hidden,
                                                                  int width, X *__restrict__ out, int64_t ld_out) {
    extern __shared__ __align__(16) char smem[];
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);  // [wave][token][4 columns]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int n0 = int(blockIdx.x) * 16, group = blockIdx.y, t0 = group * kGroup;
    const int count = min(kGroup, ch.tokens - t0);
    const int n = min(n0 + r, width - 1);
    f32x4 *own = sums + wave * count * 4;
    for (int i = lane; i < count * 4; i += 64) own[i] = f32x4{};
    using H = std::conditional_t<STAGE, Staged<Planes>, Planes>;
    // Chunks on their way at once. One of hidden values and 16-bit weights takes 64 registers, and with two no second block
    // fits a unit (1,024 tokens to 2 of 8 experts of 2,048 x 1,408 in 587 us for 526, 64 to 8 of 128 in 677 for 676); with
    // 4-bit weights two take 410 us, one 425, four 413.
    constexpr int AT_ONCE = !STAGE ? (std::is_same_v<W, Mx4> ? 2 : 1) : std::is_same_v<W, f16> ? 2 : 4;
    bf16 *staged = reinterpret_cast<bf16 *>(sums + kDownWaves * count * 4);
    const int slots = ch.tokens * ch.top_k, row = staged_planes(hidden);
    if constexpr (STAGE) {
        const int per_row = 3 * int(from.padded) / 8;
        for (int i = threadIdx.x; i < slots * per_row; i += 64 * kDownWaves) {
            const int s = i / per_row, k = (i - s * per_row) * 8;
            *reinterpret_cast<i32x4 *>(staged + s * row + k) =
                *reinterpret_cast<const i32x4 *>(from.hidden + at_planes(s * from.padded) + k);
        }
        lds_barrier();
    }
    const int chunks = (hidden + kChunkK - 1) / kChunkK;
    // an expert's number, how many tokens it has, and of the first 16 the lane's token and slot
    struct Work {
        int expert, tokens, token, slot;
    };
    auto walk = [&](int used, auto &&look) {
        const int64_t all = int64_t(used) * chunks;
        const int part = int(blockIdx.z) * kDownWaves + wave, parts = from.splits * kDownWaves;
        const int64_t end = all * (part + 1) / parts;
        int64_t u = all * part / parts;
        int a = int(u / chunks);
        Work next{};
        if (u < end) next = look(a);
        for (; u < end; ++a) {
            const Work now = next;
            const int c0 = int(u - int64_t(a) * chunks), c1 = int(min(int64_t(chunks), c0 + (end - u)));
            u += c1 - c0;
            if (u < end) next = look(a + 1);  // loaded while this one is multiplied
            const Row<W> rows[1] = {down.row(now.expert, n)};
            // the lane's token and slot in a tile of the expert's tokens
            const auto entry_of = [&](int at) {
                int2 entry = make_int2(now.token, now.slot);
                if (!FEW && at > 0)
                    entry = from.list[(int64_t(a) * from.groups + group) * kGroup + min(at + r, now.tokens - 1)];
                return entry;
            };
            const auto hidden_of = [&](bool live, int slot) -> Row<H> {
                if constexpr (STAGE) return {(LdsPtr<bf16>)(staged) + (live ? slot : 0) * row};
                else return {from.hidden + at_planes((live ? slot : 0) * from.padded), live};
            };
            // which of N tiles from `first` on have to be done again
            auto pass = [&](auto mt, auto in_flight, int first) {
                constexpr int N = decltype(mt)::value;
                Row<H> x[N];
                int token[N];
                bool live[N];
#pragma unroll
                for (int m = 0; m < N; ++m) {
                    const int2 entry = entry_of(first + 16 * m);
                    token[m] = entry.x;
                    live[m] = first + 16 * m + r < now.tokens;
                    x[m] = hidden_of(live[m], entry.y);
                }
                f32x4 part[1][N] = {};
                accumulate<decltype(in_flight)::value>(part, rows, x, c0, c1, hidden, g);
                uint32_t again = 0;
#pragma unroll
                for (int m = 0; m < N; ++m) {
                    bool nan = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) nan = nan || __builtin_isnan(part[0][m][i]);
                    if (__any(live[m] && nan)) again |= 1u << m;
                    else if (live[m]) own[(token[m] - t0) * 4 + g] += part[0][m];
                }
                return again;
            };
            using std::integral_constant;
            for (int first = 0; first < now.tokens; first += 16 * MT) {
                uint32_t again;
                if (MT > 1 && now.tokens - first > 16)
                    again = pass(integral_constant<int, MT>{}, integral_constant<int, 1>{}, first);
                else again = pass(integral_constant<int, 1>{}, integral_constant<int, AT_ONCE>{}, first);
                // An infinite weight times a hidden value's parts is rightly infinite (all have the value's sign), or NaN if
                // a later part is zero; so is an infinite hidden value times a weight's. Rare: done again with care.
                for (; again; again &= again - 1) {
                    const int at = first + 16 * __builtin_ctz(again);
                    const bool live = at + r < now.tokens;
                    const int2 entry = entry_of(at);
                    const Row<H> x[1] = {hidden_of(live, entry.y)};
                    f32x4 part[1][1] = {};
                    accumulate<1, true>(part, rows, x, c0, c1, hidden, g);
                    if (live) own[(entry.x - t0) * 4 + g] += part[0][0];
                }
            }
        }
    };
    if constexpr (FEW) {
        const Few few(ch, lane);
        walk(few.count(), [&](int a) {
            Work w;
            uint64_t choices;
            w.expert = few.number(a);
            w.tokens = few.tokens(w.expert, lane, w.token, choices);
            w.slot = w.token * ch.top_k + __builtin_ctzll(choices | uint64_t(1) << 63);
            w.token = __shfl(w.token, r);
            w.slot = __shfl(w.slot, r);
            return w;
        });
    } else {
        walk(*from.count, [&](int a) {
            const int64_t at = int64_t(a) * from.groups + group;
            const int2 entry = from.list[at * kGroup + r];  // past the list's end: not used
            return Work{from.expert[a], from.counts[at], entry.x, entry.y};
        });
    }
    __syncthreads();
    auto store = [&](int i, f32x4 sum) {
        const int c = n0 + 4 * (i & 3);
        X *o = out + int64_t(t0 + i / 4) * ld_out + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < width) o[e] = rounded<X>(sum[e]);
    };
    // Parts of other blocks' sums: stores and loads of agent scope, past the caches of the compute dies. (Plain ones
    // between fences of that scope, which write a die's whole cache back, took 60 us more.)
    using Pair = uint64_t __attribute__((ext_vector_type(2)));
    auto part_of = [&](int z, int i) {
        return reinterpret_cast<uint64_t *>(from.parts) +
               (((int64_t(z) * ch.tokens + t0 + i / 4) * from.tiles + blockIdx.x) * 4 + (i & 3)) * 2;
    };
    auto load_part = [&](int z, int i) {
        uint64_t *p = part_of(z, i);
        Pair v;
        v[0] = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v[1] = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return bits_as<f32x4>(v);
    };
    for (int i = threadIdx.x; i < count * 4; i += 64 * kDownWaves) {
        f32x4 sum = sums[i];
#pragma unroll
        for (int v = 1; v < kDownWaves; ++v) sum += sums[v * count * 4 + i];
        if (from.splits == 1) store(i, sum);
        else {
            uint64_t *p = part_of(blockIdx.z, i);
            const Pair v = bits_as<Pair>(sum);
            __hip_atomic_store(p, v[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(p + 1, v[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (from.splits == 1) return;
    // the last block to come adds all parts, in their order: each wave's stores are acknowledged before the barrier
    int *last = reinterpret_cast<int *>(smem);  // the sums are no longer needed
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        *last = __hip_atomic_fetch_add(&from.arrived[group * from.tiles + int(blockIdx.x)], 1, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT) == from.splits - 1;
    __syncthreads();
    if (!*last) return;
    for (int i = threadIdx.x; i < count * 4; i += 64 * kDownWaves) {
        f32x4 sum = load_part(0, i);
        for (int z = 1; z < from.splits; ++z) sum += load_part(z, i);
        store(i, sum);
    }
}

__global__ __launch_bounds__(256) void k_zero_out(ZeroRows z) { z.run(0); }

// --------------------------------------------------------------------- host

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// How many blocks share 16 columns of the result: so many that there are two for each compute unit, while each wave
// has two chunks of hidden units if all choices are of different experts.
int splits(int64_t tokens, int64_t top_k, int64_t experts, int64_t width, int64_t hidden) {
    const int64_t blocks = (width + 15) / 16 * ((tokens + kGroup - 1) / kGroup);
    const int64_t work = std::min(tokens * top_k, experts) * ((hidden + kChunkK - 1) / kChunkK);
    return int(std::max<int64_t>(1, std::min({int64_t(kSplitsMax), 511 / blocks, work / (2 * kDownWaves)})));
}

size_t carve(int64_t tokens, int64_t top_k, int64_t experts, int64_t width, int64_t hidden, void *ws, Between *to) {
    const int64_t slots = tokens * top_k, most = std::min(slots, experts);
    const int64_t padded = (hidden + kChunkK - 1) / kChunkK * kChunkK;
    char *p = static_cast<char *>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t a = at;
        at += up256(bytes);
        return p + a;
    };
    const int64_t groups = (tokens + kGroup - 1) / kGroup;
    char *count = take(4), *expert = take(size_t(most) * 4), *counts = take(size_t(most * groups) * 4);
    char *list = take(size_t(most * groups) * kGroup * 8);
    char *values = take(size_t(slots) * size_t(padded) * 6);
    const int64_t tiles = (width + 15) / 16, n = splits(tokens, top_k, experts, width, hidden);
    char *parts = take(n > 1 ? size_t(n * tokens * tiles) * 64 : 0);
    char *arrived = take(n > 1 ? size_t(groups * tiles) * 4 : 0);
    if (to) {
        to->parts = reinterpret_cast<float *>(parts);
        to->arrived = reinterpret_cast<int *>(arrived);
        to->tiles = int(tiles);
        to->splits = int(n);
        to->count = reinterpret_cast<int *>(count);
        to->expert = reinterpret_cast<int *>(expert);
        to->counts = reinterpret_cast<int *>(counts);
        to->list = reinterpret_cast<int2 *>(list);
        to->hidden = reinterpret_cast<bf16 *>(values);
        to->padded = padded;
        to->groups = int(groups);
    }
    return at;
}

vspmm_status check_extents(int64_t tokens, int64_t top_k, int64_t experts, int64_t width, int64_t hidden) {
    if (!fits(tokens) || !fits(top_k) || !fits(experts) || !fits(width) || !fits(hidden)) return VSPMM_ERR_DIM;
    if (tokens > kTokensMax || experts > kExpertsMax || top_k > kExpertsMax || width > kWidthMax || hidden > kWidthMax)
        return VSPMM_ERR_UNSUPPORTED;
    return VSPMM_OK;
}

template <typename W>
Matrix<W> matrix(const vspmm_expert_matrix &m) {
    if constexpr (std::is_same_v<W, Mx4>)
        return {static_cast<const uint8_t *>(m.data), m.scales, m.ld, m.stride, m.ld_scales, m.stride_scales};
    else return {static_cast<const W *>(m.data), m.ld, m.stride};
}

template <typename W, typename X, bool GELU>
void launch(const Choices &ch, const X *x, int64_t ld_x, const vspmm_expert_matrix &gate, const vspmm_expert_matrix &up,
            const vspmm_expert_matrix &down, int width, int hidden, X *out, int64_t ld_out, const Between &b,
            hipStream_t s) {
    const int tiles = (hidden + 15) / 16, most = std::min(ch.tokens * ch.top_k, ch.experts);
    const bool few = ch.tokens <= 16 && ch.tokens * ch.top_k <= 64;
    const int chunks = (width + kChunkK - 1) / kChunkK;
    const size_t lds = size_t(ch.tokens) * staged_row(width) * 2;
    const bool stage = lds <= kStageMax;
    int log_share = kLogWaves;  // tokens too wide to be staged have chunks for all waves, or nearly
    while (log_share > 0 && chunks < 2 << log_share && !(few && !stage)) --log_share;
    const bool all = log_share == kLogWaves;
    const int64_t up_blocks = ((int64_t(tiles) << log_share) + kUpWaves - 1) / kUpWaves;
    if (few) {
        auto go = [&](auto stage, auto by_all, size_t lds) {
            hipLaunchKernelGGL((k_experts_up_few<W, X, GELU, decltype(stage)::value, decltype(by_all)::value>), dim3(unsigned(up_blocks), most), dim3(64 * kUpWaves), lds, s, ch, x, ld_x,
                               matrix<W>(gate), matrix<W>(up), width, hidden, log_share, b);
        };
        if (stage && all) go(std::true_type{}, std::true_type{}, lds);
        else if (stage) go(std::true_type{}, std::false_type{}, lds);
        else go(std::false_type{}, std::true_type{}, 0);
    } else {
        // a block builds its expert's list once for up to four runs of hidden units, while there are blocks for all
        const int own = std::max(1, std::min(4, int(up_blocks * most / 1024)));
        const dim3 grid(unsigned((up_blocks + own - 1) / own), most);
        auto go = [&](auto mt, auto by_all) {
            hipLaunchKernelGGL((k_experts_up<W, X, GELU, decltype(mt)::value, decltype(by_all)::value>), grid, dim3(64 * kUpWaves), 0, s, ch, x,
                               ld_x, matrix<W>(gate), matrix<W>(up), width, hidden, log_share, own, b);
        };
        auto with_tiles = [&](auto by_all) {
            if (ch.tokens <= 16) go(std::integral_constant<int, 1>{}, by_all);
            else go(std::integral_constant<int, 4>{}, by_all);
        };
        // (4-bit rows need more registers than there are with the constant)
        if (std::is_same_v<W, Mx4> || !all) with_tiles(std::false_type{});
        else if constexpr (!std::is_same_v<W, Mx4>) with_tiles(std::true_type{});
    }
    auto go = [&](auto mt, auto by_few, auto stage, size_t staged) {
        constexpr int MT = decltype(mt)::value;
        constexpr bool FEW = decltype(by_few)::value, STAGE = decltype(stage)::value;
        const size_t lds = size_t(kDownWaves) * std::min(ch.tokens, kGroup) * 64 + staged;
        allow_lds<&k_experts_down<W, X, MT, FEW, STAGE>>(size_t(kDownWaves) * (MT > 1 ? kGroup : 16) * 64 +
                                                         (STAGE ? 2 * kStageMax : 0));
        hipLaunchKernelGGL((k_experts_down<W, X, MT, FEW, STAGE>),
                           dim3(b.tiles, b.groups, b.splits), dim3(64 * kDownWaves), lds, s, ch,
                           b, matrix<W>(down), hidden, width, out, ld_out);
    };
    constexpr std::integral_constant<int, 1> one{};
    const size_t staged = size_t(ch.tokens) * ch.top_k * staged_planes(hidden) * 2;
    if (few && staged <= 2 * kStageMax) go(one, std::true_type{}, std::true_type{}, staged);
    else if (few) go(one, std::true_type{}, std::false_type{}, 0);
    else if (ch.tokens <= 16) go(one, std::false_type{}, std::false_type{}, 0);
    else go(std::integral_constant<int, 4>{}, std::false_type{}, std::false_type{}, 0);
}

}  // namespace

extern "C" {

vspmm_status vspmm_expert_mlp_workspace_size(int64_t n_tokens, int64_t top_k, int64_t n_experts, int64_t width,
                                             int64_t hidden, size_t *bytes) {
    if (!bytes) return VSPMM_ERR_NULL;
    if (vspmm_status st = check_extents(n_tokens, top_k, n_experts, width, hidden)) return st;
    const bool none = n_tokens == 0 || top_k == 0 || n_experts == 0 || width == 0 || hidden == 0;
    *bytes = none ? 0 : carve(n_tokens, top_k, n_experts, width, hidden, nullptr, nullptr);
    return VSPMM_OK;
}

vspmm_status vspmm_expert_mlp(vspmm_elt elt, vspmm_elt weights_elt, vspmm_index index, vspmm_activation activation,
                              int64_t n_tokens, int64_t top_k, int64_t n_experts, int64_t width, int64_t hidden,
                              const void *x, int64_t ld_x, const void *experts, const float *weight,
                              const vspmm_expert_matrix *gate, const vspmm_expert_matrix *up,
                              const vspmm_expert_matrix *down, void *out, int64_t ld_out, void *ws, size_t ws_bytes,
                              hipStream_t stream) {
    if (!dense_elt(elt) || (weights_elt != elt && weights_elt != VSPMM_ELT_MX4)) return VSPMM_ERR_ENUM;
    if (index != VSPMM_INDEX_I32 && index != VSPMM_INDEX_I64) return VSPMM_ERR_ENUM;
    if (activation != VSPMM_SILU && activation != VSPMM_GELU) return VSPMM_ERR_ENUM;
    size_t need = 0;
    if (vspmm_status st = vspmm_expert_mlp_workspace_size(n_tokens, top_k, n_experts, width, hidden, &need)) return st;
    if (vspmm_status st = check_dense(n_tokens, width, ld_x, x)) return st;
    if (vspmm_status st = check_written(n_tokens, width, ld_out, out)) return st;
    if (n_tokens == 0 || width == 0) return VSPMM_OK;
    const bool mx4 = weights_elt == VSPMM_ELT_MX4;
    if (need > 0) {
        if (!experts || !weight) return VSPMM_ERR_NULL;
        for (const vspmm_expert_matrix *m : {gate, up, down}) {
            if (!m || !m->data || (mx4 && !m->scales)) return VSPMM_ERR_NULL;
            if (m->ld < 0 || m->stride < 0 || (mx4 && (m->ld_scales < 0 || m->stride_scales < 0))) return VSPMM_ERR_DIM;
        }
        if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255)) return VSPMM_ERR_WORKSPACE;
    }
    return with_dense(elt, [&](auto e) {
        using T = decltype(e);
        T *o = static_cast<T *>(out);
        if (need == 0) {  // no expert, or none with a hidden unit
            const ZeroRows z(o, ld_out * 2, n_tokens, width * 2);
            hipLaunchKernelGGL(k_zero_out, dim3(z.blocks(256)), dim3(256), 0, stream, z);
            return launched();
        }
        Between b;
        carve(n_tokens, top_k, n_experts, width, hidden, ws, &b);
        const Choices ch{experts, index == VSPMM_INDEX_I64, weight, int(n_tokens), int(top_k), int(n_experts)};
        auto go = [&](auto w, auto gelu) {
            launch<decltype(w), T, decltype(gelu)::value>(ch, static_cast<const T *>(x), ld_x, *gate, *up, *down,
                                                          int(width), int(hidden), o, ld_out, b, stream);
        };
        auto with_weights = [&](auto gelu) {
            if (mx4) go(Mx4{}, gelu);
            else go(T{}, gelu);
        };
        if (activation == VSPMM_GELU) with_weights(std::true_type{});
        else with_weights(std::false_type{});
        return launched();
    });
}

}  // extern "C"
