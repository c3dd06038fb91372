// A whole mixture-of-experts layer for a few tokens in two launches: each token's experts' gated two-layer products,
// weighted and summed. Declared in include/vspmm.h.
//
// The work is reading the weights of every expert that a token is sent to, once. The first launch takes 16 hidden
// units of one expert a block (a block finds its expert, the a-th of those in use, and its tokens in the list of
// choices by itself) and writes act(gate x) (up x) times the router's weight. The second takes 16 columns of the result a block and
// sums over all experts in use, so that no sum crosses blocks: its order is fixed, and no third launch joins parts.
// Hidden values go between them as the sum of two bfloat16 numbers (17 bits, for float32's 24: far under the result's
// rounding), which the second launch's matrix instructions take as they are.
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
constexpr int kUpWaves = 8;     // of a block of the first launch
constexpr int kDownWaves = 16;  // of a block of the second

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

// Between the launches: how many experts are in use, which, the tokens sent to each in order with a slot of each (a
// token sent twice to an expert is listed once, with both weights), where the list passes each multiple of kGroup
// tokens, and the hidden values by slot, in whole chunks with zeros at the end.
constexpr int kGroup = 128, kGroups = kTokensMax / kGroup;
struct Between {
    int *count, *expert;  // [1], [most]
    int *bounds;          // [most, kGroups + 1]
    int2 *list;           // [most, tokens]: token, slot
    bf16 *hi, *lo;        // [slots, padded]
    int64_t padded;
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

template <typename W, typename X, bool GELU, int MT>
__global__ __launch_bounds__(64 * kUpWaves) void k_experts_up(Choices ch, const X *__restrict__ x, int64_t ld_x,
                                                              Matrix<W> gate, Matrix<W> up, int width, int hidden,
                                                              Between to) {
    __shared__ uint32_t used[kExpertsMax / 32];
    __shared__ int s_expert, s_total, s_counts[kTokensMax / 64];
    __shared__ int s_slot[kTokensMax];
    __shared__ float s_weight[kTokensMax];
    __shared__ uint16_t s_token[kTokensMax];
    __shared__ f32x4 parts[kUpWaves][2][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int slots = ch.tokens * ch.top_k, a = blockIdx.y;

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
        const int own = __popc(w0) + __popc(w1);
        int before = own;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int t = __shfl_up(before, d);
            if (lane >= d) before += t;
        }
        if (lane == 63) s_total = before;
        before -= own;
        if (a >= before && a < before + own) {
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
    constexpr int GROUPS = kTokensMax / 64 / kUpWaves;
    int slot[GROUPS];
    float weight[GROUPS];
    uint64_t here[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
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
    if (blockIdx.x == 0 && tid == 0) to.expert[a] = e;
    __syncthreads();
    int mine = 0;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        int at = 0;
        for (int c = 0; c < i * kUpWaves + wave; ++c) at += s_counts[c];
        const int group = i * kUpWaves + wave;
        if (blockIdx.x == 0 && lane == 0 && group % (kGroup / 64) == 0)
            to.bounds[int64_t(a) * (kGroups + 1) + group / (kGroup / 64)] = at;
        if (slot[i] >= 0) {
            at += __popcll(here[i] & ((uint64_t(1) << lane) - 1));
            s_token[at] = uint16_t(group * 64 + lane);
            s_slot[at] = slot[i];
            s_weight[at] = weight[i];
            if (blockIdx.x == 0) to.list[int64_t(a) * ch.tokens + at] = make_int2(group * 64 + lane, slot[i]);
        }
    }
    for (int c = 0; c < kTokensMax / 64; ++c) mine += s_counts[c];
    if (blockIdx.x == 0 && tid == 0) to.bounds[int64_t(a) * (kGroups + 1) + kGroups] = mine;
    __syncthreads();

    const int r = lane & 15, g = lane >> 4;
    const int f0 = int(blockIdx.x) * 16, f = min(f0 + r, hidden - 1);
    const Row<W> rows[2] = {gate.row(e, f), up.row(e, f)};
    const int chunks = (width + kChunkK - 1) / kChunkK;
    const int c0 = chunks * wave / kUpWaves, c1 = chunks * (wave + 1) / kUpWaves;
    const bool last = blockIdx.x == gridDim.x - 1;
    // up to 16 MT tokens from `first` on
    auto pass = [&](auto mt, auto in_flight, int first) {
        constexpr int N = decltype(mt)::value;
        Row<X> tokens[N];
        const int tiles = min(N, (mine - first + 15) / 16);
#pragma unroll
        for (int m = 0; m < N; ++m)
            tokens[m] = {x + int64_t(s_token[min(first + 16 * m + r, mine - 1)]) * ld_x};
        f32x4 acc[2][N] = {};
        accumulate<decltype(in_flight)::value>(acc, rows, tokens, c0, c1, width, g, tiles);
#pragma unroll
        for (int m = 0; m < N; ++m) {
            if (m >= tiles) continue;
            parts[wave][0][lane] = acc[0][m];
            parts[wave][1][lane] = acc[1][m];
            __syncthreads();
            const int at = first + 16 * m + r;
            if (wave == 0 && at < mine) {
                f32x4 sg = parts[0][0][lane], su = parts[0][1][lane];
#pragma unroll
                for (int v = 1; v < kUpWaves; ++v) sg += parts[v][0][lane], su += parts[v][1][lane];
                const int64_t base = s_slot[at] * to.padded + f0 + 4 * g;
                bf16x4 hi, lo;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float h = f0 + 4 * g + i < hidden ? s_weight[at] * (activate<GELU>(sg[i]) * su[i]) : 0.0f;
                    hi[i] = bf16(h);
                    // an infinity has no second part
                    lo[i] = __builtin_isinf(float(hi[i])) ? bf16(0.0f) : bf16(h - float(hi[i]));
                }
                *reinterpret_cast<bf16x4 *>(to.hi + base) = hi;
                *reinterpret_cast<bf16x4 *>(to.lo + base) = lo;
                if (last)  // zeros to the end of the last chunk
                    for (int64_t f = 16; f0 + f < to.padded; f += 16) {
                        *reinterpret_cast<bf16x4 *>(to.hi + base + f) = bf16x4{};
                        *reinterpret_cast<bf16x4 *>(to.lo + base + f) = bf16x4{};
                    }
            }
            __syncthreads();
        }
    };
    using std::integral_constant;
    for (int first = 0; first < mine; first += 16 * MT) {
        if (MT > 1 && mine - first > 16) pass(integral_constant<int, MT>{}, integral_constant<int, 1>{}, first);
        else pass(integral_constant<int, 1>{}, integral_constant<int, (std::is_same_v<W, Mx4> ? 4 : 2)>{}, first);
    }
}

// A wave takes an equal run of the contraction over (expert in use, chunk of hidden units) for 16 columns, the tokens
// of an expert 16 MT at a time, and adds each expert's results to its own sums of every token, in LDS.
template <typename W, typename X, int MT>
__global__ __launch_bounds__(64 * kDownWaves) void k_experts_down(Between from, Matrix<W> down, int tokens, int hidden,
                                                                  int width, X *__restrict__ out, int64_t ld_out) {
    extern __shared__ __align__(16) char smem[];
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);  // [wave][token][4 columns]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int n0 = int(blockIdx.x) * 16, group = blockIdx.y, t0 = group * kGroup;
    const int count = min(kGroup, tokens - t0);
    const int n = min(n0 + r, width - 1);
    f32x4 *own = sums + wave * count * 4;
    for (int i = lane; i < count * 4; i += 64) own[i] = f32x4{};
    const int chunks = (hidden + kChunkK - 1) / kChunkK;
    const int64_t all = int64_t(*from.count) * chunks;
    int64_t u = all * wave / kDownWaves;
    const int64_t end = all * (wave + 1) / kDownWaves;
    // an expert's number, list and first token of the list are loaded while the one before is multiplied
    struct Next {
        int expert, first, last;
        int2 entry;
    };
    auto look = [&](int a) {
        const int *b = from.bounds + int64_t(a) * (kGroups + 1) + group;
        Next x{from.expert[a], b[0], b[1], make_int2(0, 0)};
        x.entry = from.list[int64_t(a) * tokens + max(min(x.first + r, x.last - 1), 0)];
        return x;
    };
    int a = int(u / chunks);
    Next next{};
    if (u < end) next = look(a);
    for (; u < end; ++a) {
        const Next now = next;
        const int c0 = int(u - int64_t(a) * chunks), c1 = int(min(int64_t(chunks), c0 + (end - u)));
        u += c1 - c0;
        if (u < end) next = look(a + 1);
        const Row<W> rows[1] = {down.row(now.expert, n)};
        auto pass = [&](auto mt, auto in_flight, int first) {
            constexpr int N = decltype(mt)::value;
            Row<Planes> x[N];
            int2 entry[N];
            const int tiles = min(N, (now.last - first + 15) / 16);
#pragma unroll
            for (int m = 0; m < N; ++m) {
                entry[m] = m == 0 && first == now.first
                               ? now.entry
                               : from.list[int64_t(a) * tokens + min(first + 16 * m + r, now.last - 1)];
                const int64_t base = entry[m].y * from.padded;
                x[m] = {from.hi + base, from.lo + base};
            }
            f32x4 part[1][N] = {};
            accumulate<decltype(in_flight)::value>(part, rows, x, c0, c1, hidden, g, tiles);
#pragma unroll
            for (int m = 0; m < N; ++m)
                if (first + 16 * m + r < now.last) own[(entry[m].x - t0) * 4 + g] += part[0][m];
        };
        using std::integral_constant;
        for (int first = now.first; first < now.last; first += 16 * MT) {
            if (MT > 1 && now.last - first > 16) pass(integral_constant<int, MT>{}, integral_constant<int, 1>{}, first);
            else pass(integral_constant<int, 1>{}, integral_constant<int, 2>{}, first);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < count * 4; i += 64 * kDownWaves) {
        f32x4 sum = sums[i];
#pragma unroll
        for (int v = 1; v < kDownWaves; ++v) sum += sums[v * count * 4 + i];
        const int c = n0 + 4 * (i & 3);
        X *o = out + int64_t(t0 + i / 4) * ld_out + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < width) o[e] = rounded<X>(sum[e]);
    }
}

__global__ __launch_bounds__(256) void k_zero_out(ZeroRows z) { z.run(0); }

// --------------------------------------------------------------------- host

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

size_t carve(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, void *ws, Between *to) {
    const int64_t slots = tokens * top_k, most = std::min(slots, experts);
    char *p = static_cast<char *>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t a = at;
        at += up256(bytes);
        return p + a;
    };
    const int64_t padded = (hidden + kChunkK - 1) / kChunkK * kChunkK;
    char *count = take(4), *expert = take(size_t(most) * 4), *bounds = take(size_t(most) * (kGroups + 1) * 4);
    char *list = take(size_t(most) * size_t(tokens) * 8);
    char *hi = take(size_t(slots) * size_t(padded) * 2), *lo = take(size_t(slots) * size_t(padded) * 2);
    if (to) {
        to->count = reinterpret_cast<int *>(count);
        to->expert = reinterpret_cast<int *>(expert);
        to->bounds = reinterpret_cast<int *>(bounds);
        to->list = reinterpret_cast<int2 *>(list);
        to->hi = reinterpret_cast<bf16 *>(hi);
        to->lo = reinterpret_cast<bf16 *>(lo);
        to->padded = padded;
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
    const dim3 grid((hidden + 15) / 16, std::min(ch.tokens * ch.top_k, ch.experts));
    if (ch.tokens <= 16)
        hipLaunchKernelGGL((k_experts_up<W, X, GELU, 1>), grid, dim3(64 * kUpWaves), 0, s, ch, x, ld_x, matrix<W>(gate),
                           matrix<W>(up), width, hidden, b);
    else
        hipLaunchKernelGGL((k_experts_up<W, X, GELU, 4>), grid, dim3(64 * kUpWaves), 0, s, ch, x, ld_x, matrix<W>(gate),
                           matrix<W>(up), width, hidden, b);
    auto go = [&](auto mt) {
        constexpr int MT = decltype(mt)::value;
        const size_t lds = size_t(kDownWaves) * std::min(ch.tokens, kGroup) * 64;
        allow_lds(reinterpret_cast<const void *>(&k_experts_down<W, X, MT>), lds);
        hipLaunchKernelGGL((k_experts_down<W, X, MT>), dim3((width + 15) / 16, (ch.tokens + kGroup - 1) / kGroup),
                           dim3(64 * kDownWaves), lds, s, b, matrix<W>(down), ch.tokens, hidden, width, out, ld_out);
    };
    if (ch.tokens <= 16) go(std::integral_constant<int, 1>{});
    else go(std::integral_constant<int, 4>{});
}

}  // namespace

extern "C" {

vspmm_status vspmm_expert_mlp_workspace_size(int64_t n_tokens, int64_t top_k, int64_t n_experts, int64_t width,
                                             int64_t hidden, size_t *bytes) {
    if (!bytes) return VSPMM_ERR_NULL;
    if (vspmm_status st = check_extents(n_tokens, top_k, n_experts, width, hidden)) return st;
    const bool none = n_tokens == 0 || top_k == 0 || n_experts == 0 || width == 0 || hidden == 0;
    *bytes = none ? 0 : carve(n_tokens, top_k, n_experts, hidden, nullptr, nullptr);
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
        carve(n_tokens, top_k, n_experts, hidden, ws, &b);
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
