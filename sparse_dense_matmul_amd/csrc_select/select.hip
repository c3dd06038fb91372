// Products with a selection matrix, whose rows hold one entry (a token's row
// of an embedding table) or a few (a token's experts): the embedding lookup
// and its gradient, the routing of tokens to experts and back, and the
// routing's gradients. The matrix is its index list alone; its transpose, which
// the gradient and the routing need, is a stable counting sort of that list
// (bins.hpp). Declared in include/vspmm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "vspmm.h"
#include "bins.hpp"
#include "grad.hpp"
#include "rows.hpp"

using namespace vspmm;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kI32Max = 2147483647;
constexpr int kNoRow = 2147483647;  // a position past every row: slots number at most this
// k_embed: four chunks a lane from here on, with nontemporal stores (16,384 rows of
// 4,096 bf16 48 -> 34 us); one below, for as many waves as there are chunks
constexpr uint32_t kManyChunks = 1 << 20;
constexpr int64_t kWidthMax = 1 << 24;  // elements of a row

// ------------------------------------------------------------------ kernels

// f(count, k) for k = 0, 8, .. : eight at a time, then four, two and one.
template <typename F>
__device__ __forceinline__ void by_eights(int n, F &&f) {
    int k = 0;
    for (; k + 8 <= n; k += 8) f(std::integral_constant<int, 8>{}, k);
    if (n & 4) f(std::integral_constant<int, 4>{}, k), k += 4;
    if (n & 2) f(std::integral_constant<int, 2>{}, k), k += 2;
    if (n & 1) f(std::integral_constant<int, 1>{}, k);
}

// f(count, k, m): eight at a time, then all that are left in one batch of the
// least power of two that holds them, m of which count.
template <typename F>
__device__ __forceinline__ void by_padded_eights(int n, F &&f) {
    int k = 0;
    for (; k + 8 <= n; k += 8) f(std::integral_constant<int, 8>{}, k, 8);
    const int m = n - k;
    if (m > 4) f(std::integral_constant<int, 8>{}, k, m);
    else if (m > 2) f(std::integral_constant<int, 4>{}, k, m);
    else if (m > 1) f(std::integral_constant<int, 2>{}, k, m);
    else if (m > 0) f(std::integral_constant<int, 1>{}, k, m);
}

// The chunks of a batch of rows as one flat list: consecutive lanes take
// consecutive chunks whatever the width, a block 256 * U in a row, a lane U of
// them, 256 apart.
struct Chunks {
    uint32_t n, cpr, width;
    FastDiv by_cpr;
};

// out[t] = scale * table[ids[t]], or zeros for an id outside the table. Bound by
// memory: 57 MB of distinct rows read and 134 written for 16,384 tokens of 4,096
// bf16 in 34 us, 5.6 TB/s (a plain kernel that reads one byte for two written
// reaches 6.0). One step's 32 tokens take 2.7 us, a launch and two dependent loads.
template <typename T, typename I, int C, int U>
__global__ void __launch_bounds__(kThreads)
k_embed(const T *__restrict__ table, int64_t ld_table, int64_t n_rows, const I *__restrict__ ids,
        Chunks ch, typename Sum<T>::type scale, T *__restrict__ out, int64_t ld_out) {
    using A = typename Sum<T>::type;
    const uint32_t g0 = blockIdx.x * (kThreads * U) + threadIdx.x;
    int64_t id[U];
    uint32_t col[U], t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // lanes past the list take its last chunk again and write nothing
        const uint32_t g = g0 + u * kThreads < ch.n ? g0 + u * kThreads : ch.n - 1;
        t[u] = ch.by_cpr.div(g);
        col[u] = chunk_col<C>(g - t[u] * ch.cpr, ch.width);
        id[u] = int64_t(ids[t[u]]);
    }
    Vec<T, C> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = Vec<T, C>{};
        if (id[u] >= 0 && id[u] < n_rows) v[u] = load_vec<C>(table + id[u] * ld_table + col[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool real = id[u] >= 0 && id[u] < n_rows;
#pragma unroll
        for (int i = 0; i < C; ++i) v[u][i] = real ? rounded<T>(A(v[u][i]) * scale) : T(0);
        if (g0 + u * kThreads < ch.n) {
            T *o = out + int64_t(t[u]) * ld_out + col[u];
            if (U > 1) store_once<C>(o, v[u]);  // 37.2 -> 34.7 us at 16,384 x 4,096 bf16
            else store_vec<C>(o, v[u]);
        }
    }
}

__global__ void __launch_bounds__(kThreads) k_zero(ZeroRows zero) { zero.run(0); }

// rows[position[t, k]] = x[t]; a dropped slot (~p) has row p zeroed. A
// position past the last row is passed over. From the token's side, so that x is
// read once: from the rows' side (each reading its token) 304 us where this takes
// 226 for 16,384 tokens of 4,096 bf16 to eight rows each, 1.21 GB, 5.4 TB/s, bound
// by the scattered rows' writes (a plain fill of them takes 157).
template <typename T, int C>
__global__ void __launch_bounds__(kThreads)
k_dispatch(const T *__restrict__ x, int64_t ld_x, const int *__restrict__ position, int top_k,
           uint32_t n_slots, Chunks ch, T *__restrict__ rows, int64_t ld_rows) {
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= ch.n) return;
    const uint32_t t = ch.by_cpr.div(g), col = chunk_col<C>(g - t * ch.cpr, ch.width);
    const Vec<T, C> v = load_vec<C>(x + int64_t(t) * ld_x + col);
    const int *pos = position + int64_t(t) * top_k;
    auto put = [&](auto count, int k) {
        constexpr int N = decltype(count)::value;
        int p[N];
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = pos[k + j];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t row = uint32_t(p[j] >= 0 ? p[j] : ~p[j]);
            if (row < n_slots)
                store_vec<C>(rows + int64_t(row) * ld_rows + col, p[j] >= 0 ? v : Vec<T, C>{});
        }
    };
    by_eights(top_k, put);
}

// out[t] = sum over k of weight[t, k] * rows[position[t, k]] (weight null:
// ones), k ascending, live slots only; one rounding at the end. Up to eight
// rows in flight. ONCE: rows larger than the caches are read nontemporally. Bound
// by memory: 131,072 rows of 4,096 bf16 to 16,384 tokens, 1.21 GB, in 204 us
// (5.9 TB/s).
template <typename T, int C, bool WEIGHTED, bool ONCE>
__global__ void __launch_bounds__(kThreads)
k_combine(const T *__restrict__ rows, int64_t ld_rows, const int *__restrict__ position,
          const typename Sum<T>::type *__restrict__ weight, int top_k, uint32_t n_slots, Chunks ch,
          T *__restrict__ out, int64_t ld_out) {
    using A = typename Sum<T>::type;
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= ch.n) return;
    const uint32_t t = ch.by_cpr.div(g), col = chunk_col<C>(g - t * ch.cpr, ch.width);
    const int *pos = position + int64_t(t) * top_k;
    A acc[C] = {};
    auto take = [&](auto count, int k) {
        constexpr int N = decltype(count)::value;
        uint32_t p[N];
        A w[N];
        Vec<T, C> v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = uint32_t(pos[k + j]);
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = WEIGHTED ? weight[int64_t(t) * top_k + k + j] : A(1);
        // a dropped slot loads the row of the live one before it once more
        uint32_t from[N], last = 0;
#pragma unroll
        for (int j = N - 1; j >= 0; --j) last = p[j] < n_slots ? p[j] : last;
#pragma unroll
        for (int j = 0; j < N; ++j) from[j] = last = p[j] < n_slots ? p[j] : last;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = load_as<ONCE, C>(rows + int64_t(from[j]) * ld_rows + col);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (p[j] < n_slots) {
#pragma unroll
                for (int i = 0; i < C; ++i)
                    acc[i] = WEIGHTED ? fma(w[j], A(v[j][i]), acc[i]) : acc[i] + A(v[j][i]);
            }
    };
    by_eights(top_k, take);
    Vec<T, C> o;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = rounded<T>(acc[i]);
    store_vec<C>(out + int64_t(t) * ld_out + col, o);
}

// N sums per lane to their totals over the wave's lanes: each step sends the
// half of the values the partner keeps, so N values take 6 + N - 1 - log2 N
// exchanges. Value lane / (64 / N)'s total ends in the lane.
template <int N, typename A>
__device__ __forceinline__ A wave_totals(A (&a)[N], int lane) {
    int m = 32;
#pragma unroll
    for (int half = N / 2; half >= 1; half /= 2, m /= 2) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const A send = up ? a[i] : a[i + half];
            const A keep = up ? a[i + half] : a[i];
            a[i] = keep + __shfl_xor(send, m);
        }
    }
#pragma unroll
    for (; m >= 1; m /= 2) a[0] += __shfl_xor(a[0], m);
    return a[0];
}

// Gradients of the combine: grad_rows[position[t, k]] = weight[t, k] *
// dout[t] and grad_weight[t, k] = <dout[t], rows[position[t, k]]>; a dropped
// slot's row and weight gradient are zero. W waves share a token's width, up to
// eight of its slots at a time, so dout is read and rows and grad_rows are
// streamed once; the dots' lane sums are added over the wave, then wave by wave:
// a fixed order. Bound by memory: 131,072 rows of 2,048 bf16, 1.14 GB, in 209 us
// (5.5 TB/s, half of it written). Rows of fewer than 64 chunks leave lanes idle: as
// many rows of 128 bf16 take 28 us, 71 MB at 2.5 TB/s. float64 goes through 80 bytes
// of scratch a lane (wave_totals' choice between array elements): 131,072 rows of
// 512, 1.14 GB, 216 us.
template <typename T, int C, int W, bool ONCE>
__global__ void __launch_bounds__(kThreads)
k_combine_grad(const T *__restrict__ dout, int64_t ld_dout, const T *__restrict__ rows,
               int64_t ld_rows, const int *__restrict__ position,
               const typename Sum<T>::type *__restrict__ weight, int top_k, uint32_t n_slots,
               uint32_t n_tokens, uint32_t width, uint32_t cpr, T *__restrict__ grad_rows,
               int64_t ld_grad_rows,
               typename Sum<T>::type *__restrict__ grad_weight) {
    using A = typename Sum<T>::type;
    constexpr int PER = kThreads / 64 / W;  // tokens per block
    __shared__ A sums[PER][W][8];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // so rows are scalar
    const int mine = wave / W, part = wave % W;
    const uint32_t t = blockIdx.x * PER + mine;
    const bool real = t < n_tokens;
    const int64_t slot0 = int64_t(t) * top_k;
    auto batch = [&](auto count, int k, int m) {
        constexpr int N = decltype(count)::value;
        A dot[N] = {};
        if (real) {
            uint32_t row[N];
            bool kept[N];
            A w[N];
            const T *from[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int p = j < m ? position[slot0 + k + j] : kNoRow;
                row[j] = uint32_t(p >= 0 ? p : ~p);
                kept[j] = p >= 0 && row[j] < n_slots;
                w[j] = j < m ? weight[slot0 + k + j] : A(0);
                from[j] = kept[j] ? rows + int64_t(row[j]) * ld_rows : dout + int64_t(t) * ld_dout;
            }
            for (uint32_t c = part * 64 + lane; c < cpr; c += 64 * W) {
                const uint32_t col = chunk_col<C>(c, width);
                const int moved = int(c * C - col);
                const Vec<T, C> d = load_vec<C>(dout + int64_t(t) * ld_dout + col);
                Vec<T, C> y[N];
                // a dropped slot loads dout's chunk once more
#pragma unroll
                for (int j = 0; j < N; ++j) y[j] = load_as<ONCE, C>(from[j] + col);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    Vec<T, C> o{};
                    if (kept[j]) {
#pragma unroll
                        for (int i = 0; i < C; ++i) {
                            if (i >= moved) dot[j] = fma(A(d[i]), A(y[j][i]), dot[j]);
                            o[i] = rounded<T>(w[j] * A(d[i]));
                        }
                    }
                    if (row[j] < n_slots) {
                        T *to = grad_rows + int64_t(row[j]) * ld_grad_rows + col;
                        if constexpr (ONCE) store_once<C>(to, o);
                        else store_vec<C>(to, o);
                    }
                }
            }
        }
        const A total = wave_totals(dot, lane);
        constexpr int SPAN = 64 / N;  // lanes that hold one value's total
        if (W == 1) {
            if (real && lane % SPAN == 0 && lane / SPAN < m)
                grad_weight[slot0 + k + lane / SPAN] = total;
            return;
        }
        if (lane % SPAN == 0) sums[mine][part][lane / SPAN] = total;
        __syncthreads();
        if (real && part == 0 && lane < m) {
            A all = sums[mine][0][lane];
#pragma unroll
            for (int w2 = 1; w2 < W; ++w2) all += sums[mine][w2][lane];
            grad_weight[slot0 + k + lane] = all;
        }
        __syncthreads();
    };
    // one batch for three or five to seven slots, not two or three: each has a round
    // of loads and two barriers of its own (3,001 tokens of six slots of 1,001 f32 37
    // -> 30 us, of three 18.6 -> 16.3; the combine, without barriers, gains nothing so)
    by_padded_eights(top_k, batch);
}

// --------------------------------------------------------------------- host

vspmm_status launched() { return hipGetLastError() == hipSuccess ? VSPMM_OK : VSPMM_ERR_HIP; }

bool fits(int64_t x) { return x >= 0 && x <= kI32Max; }

int elt_bytes(int elt) {
    return elt == VSPMM_ELT_F64 ? 8 : elt == VSPMM_ELT_F32 ? 4 : 2;
}
bool known_elt(int elt) { return elt >= VSPMM_ELT_F32 && elt <= VSPMM_ELT_F16; }
bool known_index(int index) { return index == VSPMM_INDEX_I32 || index == VSPMM_INDEX_I64; }

// f(element of the type) for the element type `elt`.
template <typename F>
void with_elt(int elt, F &&f) {
    switch (elt) {
        case VSPMM_ELT_F32: f(float{}); break;
        case VSPMM_ELT_F64: f(double{}); break;
        case VSPMM_ELT_BF16: f(bf16{}); break;
        default: f(f16{}); break;
    }
}
template <typename F>
void with_index(int index, F &&f) {
    if (index == VSPMM_INDEX_I64) f(int64_t{});
    else f(int32_t{});
}

// f(chunk size): the 16-byte chunk, or one element for rows shorter than that.
template <typename T, typename F>
void with_chunk(int64_t width, F &&f) {
    if (width >= kChunk<T>) f(std::integral_constant<int, kChunk<T>>{});
    else f(std::integral_constant<int, 1>{});
}

// f(r0, chunks) over rows [r0, ..), as many at a time as have fewer than 2^31
// chunks of C elements.
template <int C, typename F>
void by_rows(int64_t n, int64_t width, F &&f) {
    const uint32_t cpr = uint32_t((width + C - 1) / C);
    const int64_t most = (kI32Max - (1 << 20)) / cpr;
    for (int64_t r0 = 0; r0 < n; r0 += most)
        f(r0, Chunks{uint32_t(std::min(most, n - r0)) * cpr, cpr, uint32_t(width), FastDiv(cpr)});
}
unsigned blocks_of(uint32_t n, int per) { return (n + per - 1) / per; }

// Rows that the 256 MB last-level cache cannot hold are read, and the
// gradient's written, nontemporally: combine at 1.07 GB 235 -> 204 us,
// combine_grad at 0.54 GB 206 -> 183; at 64 MB combine takes 15.6 us with it and
// 14.0 without.
bool streams(int64_t n, int64_t width, int elt) {
    return n * width * elt_bytes(elt) > (int64_t(256) << 20);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Lets a kernel of the current device use that much dynamic LDS.
void allow_dynamic(const void *fn, size_t bytes) {
    if (bytes > 64 * 1024)
        (void)hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

int bits_of(int64_t x) {  // bits that hold 0 .. x
    int b = 1;
    while (b < 32 && (int64_t(1) << b) <= x) ++b;
    return b;
}

// The passes of the sort of ids in [0, limit]: digits of at most 11 bits.
struct Passes {
    int count, bits;
};
Passes passes_for(int64_t limit) {
    const int bits = bits_of(limit);
    const int count = (bits + 10) / 11;
    return {count, (bits + count - 1) / count};
}

constexpr int64_t kGradGroups = 2048;
// The longest list and the largest dout of the gradient. Within them there are
// less than 2^26 pieces (segments times slices), which k_grad_rows numbers in 31
// bits: a segment of less than 64 places means at most 2^13 pieces and a row's
// slices, one of 64 at most 2^24 segments of one slice, or, where a row of more
// than 1,008 bytes has several, less than two for each KB of it.
constexpr int64_t kGradTokens = int64_t(1) << 30;
constexpr int64_t kGradBytes = int64_t(1) << 40;

// How k_grad_rows cuts the work: lanes per group, slices of the width, places
// per segment.
struct GradPlan {
    int chunk, lanes, slices, seg;
    int64_t cpr, segs;
};
GradPlan grad_plan(int elt, int64_t width, int64_t n) {
    GradPlan g;
    g.chunk = width >= 16 / elt_bytes(elt) ? 16 / elt_bytes(elt) : 1;
    g.cpr = (width + g.chunk - 1) / g.chunk;
    // narrow rows: four groups of 16 lanes a wave, and so segments of at most 16; in
    // long lists a group of 64, most of its lanes idle, for segments of 64 (1,000,000
    // tokens of 64 bf16 over 32,000 ids 410 -> 134 us, but of one id 111 -> 137). At
    // the border itself the groups of 16 are still ahead: 131,071 tokens 43.5 us and
    // 131,072 49.8, Zipf's ids 54 and 60, of one id 49 and 92.
    g.lanes = g.cpr > 16 || n >= 1 << 17 ? 64 : 16;
    g.slices = int((g.cpr + g.lanes - 1) / g.lanes);
    // 2,048 groups or more as far as segments of 4 go: shorter segments leave more
    // partial rows (16,384 tokens of 1,024 bf16 57 us at 8,192 groups, 50 at 2,048)
    const int most = g.lanes, least = 4;
    g.seg = least;
    while (g.seg < most && n * g.slices >= int64_t(2 * g.seg) * kGradGroups) g.seg *= 2;
    g.segs = (n + g.seg - 1) / g.seg;
    return g;
}

struct GradWs {
    uint32_t *keys[2];
    int *pay[2];
    int *counts;
    int *list, *listed;
    void *part;
    int64_t ld_part;
    size_t bytes;
};
GradWs carve_grad(int elt, int64_t n_rows, int64_t width, int64_t n, void *base) {
    GradWs w;
    size_t at = 0;
    char *p = static_cast<char *>(base);
    auto take = [&](size_t bytes) {
        char *r = p + at;
        at += up256(bytes);
        return r;
    };
    const GradPlan g = grad_plan(elt, width, n);
    const bool sorted = n > kRankMax;  // through a second copy
    for (int i = 0; i < 2; ++i) {
        w.keys[i] = reinterpret_cast<uint32_t *>(take(i == 0 || sorted ? size_t(n) * 4 : 0));
        w.pay[i] = reinterpret_cast<int *>(take(i == 0 || sorted ? size_t(n) * 4 : 0));
    }
    w.counts = reinterpret_cast<int *>(
        take(n > kMergeMax ? (size_t(4) * bin_blocks_most(n)) << passes_for(n_rows).bits : 0));
    w.listed = reinterpret_cast<int *>(take(4));
    // room for as many segments as any shorter list has: 4,096 groups before a
    // segment grows, of 4 places at least
    const int64_t segs =
        std::max(g.segs, std::min<int64_t>((n + 3) / 4, (2 * kGradGroups + g.slices - 1) / g.slices));
    w.list = reinterpret_cast<int *>(take(size_t(segs) * 4));
    w.ld_part = int64_t(g.slices) * g.lanes * g.chunk;
    w.part = take(2 * size_t(segs) * size_t(w.ld_part) * (elt == VSPMM_ELT_F64 ? 8 : 4));
    w.bytes = at;
    return w;
}

vspmm_status check_rows(int64_t n, int64_t width, int64_t ld, const void *p) {
    if (!fits(n) || !fits(width) || ld < 0) return VSPMM_ERR_DIM;
    if (width > kWidthMax) return VSPMM_ERR_UNSUPPORTED;
    if (n > 0 && width > 0 && !p) return VSPMM_ERR_NULL;
    return VSPMM_OK;
}
// Rows that are written must not overlap.
vspmm_status check_out(int64_t n, int64_t width, int64_t ld, const void *p) {
    if (n > 1 && ld < width) return VSPMM_ERR_DIM;
    return check_rows(n, width, ld, p);
}

template <typename T, typename G, bool ADD>
void launch_grad(const GradPlan &g, const GradWs &w, const uint32_t *keys, const int *order,
                 int64_t n, int64_t n_rows, const void *dout, int64_t ld_dout, int64_t width,
                 double scale, void *grad, int64_t ld_grad, hipStream_t s) {
    using A = typename Sum<T>::type;
    GradArgs<T, G> a;
    a.keys = keys;
    a.order = order;
    a.n = int(n);
    a.seg = g.seg;
    a.segs = int(g.segs);
    a.n_rows = uint32_t(n_rows);
    a.dout = static_cast<const T *>(dout);
    a.ld_dout = ld_dout;
    a.width = int(width);
    a.cpr = uint32_t(g.cpr);
    a.slices = uint32_t(g.slices);
    a.by_slices = FastDiv(uint32_t(g.slices));
    a.scale = A(scale);
    a.grad = static_cast<G *>(grad);
    a.ld_grad = ld_grad;
    a.part = static_cast<A *>(w.part);
    a.ld_part = w.ld_part;
    a.list = w.list;
    a.listed = w.listed;
    auto go = [&](auto chunk, auto lanes) {
        constexpr int C = decltype(chunk)::value, L = decltype(lanes)::value, PER = kGradThreads / L;
        const int64_t items = g.segs * g.slices;
        hipLaunchKernelGGL((k_grad_rows<T, G, C, L, ADD>), dim3(unsigned((items + PER - 1) / PER)),
                           dim3(kGradThreads), 0, s, a);
        if (g.segs >= kFoldSegs)
            hipLaunchKernelGGL((k_grad_fold<T, G, C, L>),
                               dim3(unsigned(g.segs / kFold), unsigned(g.slices)), dim3(kJoinThreads),
                               0, s, a);
        if (g.segs > 1)
            hipLaunchKernelGGL((k_grad_join<T, G, C, L, ADD>),
                               dim3(unsigned(std::min<int64_t>(items, 2048))), dim3(kJoinThreads), 0, s,
                               a);
    };
    const std::integral_constant<int, 64> wide;
    const std::integral_constant<int, 16> narrow;
    auto pick = [&](auto chunk) {
        if (g.lanes == 64) go(chunk, wide);
        else go(chunk, narrow);
    };
    if (g.chunk == 1) pick(std::integral_constant<int, 1>{});
    else pick(std::integral_constant<int, kChunk<T>>{});
}

}  // namespace

extern "C" {

vspmm_status vspmm_embed(vspmm_elt elt, int64_t n_rows, int64_t width, const void *table,
                         int64_t ld_table, vspmm_index index, int64_t n, const void *ids,
                         double scale, void *out, int64_t ld_out, hipStream_t stream) {
    if (!known_elt(elt) || !known_index(index)) return VSPMM_ERR_ENUM;
    if (vspmm_status st = check_rows(n_rows, width, ld_table, table)) return st;
    if (vspmm_status st = check_out(n, width, ld_out, out)) return st;
    if (n > 0 && !ids) return VSPMM_ERR_NULL;
    if (n == 0 || width == 0) return VSPMM_OK;
    with_elt(elt, [&](auto e) {
        with_index(index, [&](auto i) {
            using T = decltype(e);
            using I = decltype(i);
            with_chunk<T>(width, [&](auto chunk) {
                constexpr int C = decltype(chunk)::value;
                by_rows<C>(n, width, [&](int64_t r0, Chunks ch) {
                    auto go = [&](auto per) {
                        constexpr int U = decltype(per)::value;
                        hipLaunchKernelGGL((k_embed<T, I, C, U>), dim3(blocks_of(ch.n, kThreads * U)),
                                           dim3(kThreads), 0, stream, static_cast<const T *>(table),
                                           ld_table, n_rows, static_cast<const I *>(ids) + r0, ch,
                                           typename Sum<T>::type(scale),
                                           static_cast<T *>(out) + r0 * ld_out, ld_out);
                    };
                    if (ch.n >= kManyChunks) go(std::integral_constant<int, 4>{});
                    else go(std::integral_constant<int, 1>{});
                });
            });
        });
    });
    return launched();
}

vspmm_status vspmm_embed_grad_workspace_size(vspmm_elt elt, int64_t n_rows, int64_t width,
                                             int64_t n, size_t *bytes) {
    if (!bytes) return VSPMM_ERR_NULL;
    if (!known_elt(elt)) return VSPMM_ERR_ENUM;
    if (!fits(n_rows) || n_rows == kI32Max || !fits(width) || !fits(n)) return VSPMM_ERR_DIM;
    if (width > kWidthMax) return VSPMM_ERR_UNSUPPORTED;
    if (n > kGradTokens || n * width * elt_bytes(elt) > kGradBytes) return VSPMM_ERR_UNSUPPORTED;
    *bytes = n_rows && width && n ? carve_grad(elt, n_rows, width, n, nullptr).bytes : 0;
    return VSPMM_OK;
}

vspmm_status vspmm_embed_grad(vspmm_elt elt, vspmm_elt grad_elt, int64_t n_rows, int64_t width,
                              vspmm_index index, int64_t n, const void *ids, const void *dout,
                              int64_t ld_dout, double scale, int32_t accumulate, void *grad,
                              int64_t ld_grad, void *ws, size_t ws_bytes, hipStream_t stream) {
    if (!known_elt(elt) || !known_elt(grad_elt) || !known_index(index)) return VSPMM_ERR_ENUM;
    if (grad_elt != elt && (grad_elt != VSPMM_ELT_F32 || elt == VSPMM_ELT_F64))
        return VSPMM_ERR_ENUM;
    size_t need = 0;
    if (vspmm_status st = vspmm_embed_grad_workspace_size(elt, n_rows, width, n, &need)) return st;
    if (vspmm_status st = check_rows(n, width, ld_dout, dout)) return st;
    if (vspmm_status st = check_out(n_rows, width, ld_grad, grad)) return st;
    if (n > 0 && !ids) return VSPMM_ERR_NULL;
    if (need > 0 && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255)))
        return VSPMM_ERR_WORKSPACE;
    if (n_rows == 0 || width == 0) return VSPMM_OK;
    // Every row is zeroed first, by blocks of the first launch beside its own
    // (the sort's latency hides there), and the rows that tokens select written
    // again. Zeroing the others alone, beside the sums, mixes reads and writes:
    // 16,384 tokens, 100,000 rows of 1,024 bf16 56 us for 50; 65,536 tokens, 131,072
    // rows of 4,096, where an eighth of the writes is spared, 314 for 336.
    ZeroRows zero;
    if (!accumulate)
        zero = ZeroRows(grad, ld_grad * elt_bytes(grad_elt), n_rows, width * elt_bytes(grad_elt));
    if (n == 0) {
        if (zero.chunks)
            hipLaunchKernelGGL(k_zero, dim3(zero.blocks(kThreads)), dim3(kThreads), 0, stream, zero);
        return launched();
    }
    const GradPlan plan = grad_plan(elt, width, n);
    const GradWs w = carve_grad(elt, n_rows, width, n, ws);
    const uint32_t *keys = w.keys[0];
    const int *order = w.pay[0];
    with_index(index, [&](auto i) {
        using I = decltype(i);
        if (n <= kRankMax) {
            const int nb = int((n + kRankTile - 1) / kRankTile);
            hipLaunchKernelGGL(k_rank<I>, dim3(nb + zero.blocks(kRankThreads)), dim3(kRankThreads), 0,
                               stream, static_cast<const I *>(ids), int(n), n_rows, nb,
                               PlaceKeys{w.keys[0], w.pay[0], nullptr}, w.listed, zero);
            return;
        }
        if (n <= kMergeMax) {
            const int nb = int((n + kRankTile - 1) / kRankTile);
            hipLaunchKernelGGL(k_chunk_rank<I>, dim3(nb + zero.blocks(kChunkThreads)),
                               dim3(kChunkThreads), 0, stream, static_cast<const I *>(ids), int(n),
                               n_rows, nb, PlaceKeys{w.keys[1], w.pay[1], nullptr}, w.listed, zero);
            auto merge = [&](auto t) {
                constexpr int TILE = decltype(t)::value;
                hipLaunchKernelGGL(k_merge_rank<TILE>, dim3((int(n) + TILE - 1) / TILE),
                                   dim3(kMergeThreads), kMergeLds, stream, w.keys[1], w.pay[1],
                                   int(n), PlaceKeys{w.keys[0], w.pay[0], nullptr});
            };
            // a block for each of the 256 CUs, as far as tiles of 64 to 256 go
            if (n <= 64 * 256) merge(std::integral_constant<int, 64>{});
            else if (n <= 128 * 256) merge(std::integral_constant<int, 128>{});
            else merge(std::integral_constant<int, 256>{});
            return;
        }
        const Passes ps = passes_for(n_rows);
        const int bins = 1 << ps.bits, piece = bin_piece(n), nb = bin_blocks(n);
        order = nullptr;
        auto pass = [&](auto *src, int k) {
            using S = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
            const BinPass<S> p{src, n, n_rows, k * ps.bits, bins, piece, nb};
            if (k > 0) zero = ZeroRows();
            hipLaunchKernelGGL(k_bin_count<S>, dim3(nb + zero.blocks(kBinThreads)), dim3(kBinThreads),
                               size_t(bins) * 4, stream, p, w.counts, w.listed, zero);
            allow_dynamic(reinterpret_cast<const void *>(&k_bin_place<S, PlaceKeys>), bin_lds(bins));
            const PlaceKeys to{w.keys[k & 1], w.pay[k & 1], order};
            hipLaunchKernelGGL((k_bin_place<S, PlaceKeys>), dim3(nb), dim3(kBinThreads), bin_lds(bins),
                               stream, p, ps.bits, w.counts, to, static_cast<int *>(nullptr));
            keys = to.keys;
            order = to.pay;
        };
        pass(static_cast<const I *>(ids), 0);
        for (int k = 1; k < ps.count; ++k) pass(keys, k);
    });
    auto sum = [&](auto e, auto g) {
        using T = decltype(e);
        using G = decltype(g);
        if (accumulate)
            launch_grad<T, G, true>(plan, w, keys, order, n, n_rows, dout, ld_dout, width, scale, grad,
                                    ld_grad, stream);
        else
            launch_grad<T, G, false>(plan, w, keys, order, n, n_rows, dout, ld_dout, width, scale, grad,
                                     ld_grad, stream);
    };
    with_elt(elt, [&](auto e) {
        if (grad_elt == elt) sum(e, e);
        else if constexpr (sizeof(e) == 2) sum(e, float{});
    });
    return launched();
}

vspmm_status vspmm_route_workspace_size(int64_t n_tokens, int64_t top_k, int64_t n_experts,
                                        size_t *bytes) {
    if (!bytes) return VSPMM_ERR_NULL;
    if (!fits(n_tokens) || !fits(top_k) || !fits(n_experts) || !fits(n_tokens * top_k))
        return VSPMM_ERR_DIM;
    if (n_experts + 1 > kBinMax) return VSPMM_ERR_UNSUPPORTED;
    const int64_t n = n_tokens * top_k;
    *bytes = bin_blocks(n) > 1 ? up256(size_t(4) * bin_blocks_most(n) * size_t(n_experts + 1)) : 0;
    return VSPMM_OK;
}

vspmm_status vspmm_route(vspmm_index index, int64_t n_tokens, int64_t top_k, int64_t n_experts,
                         const void *experts, int32_t *order, int32_t *position, int32_t *offsets,
                         void *ws, size_t ws_bytes, hipStream_t stream) {
    if (!known_index(index)) return VSPMM_ERR_ENUM;
    size_t need = 0;
    if (vspmm_status st = vspmm_route_workspace_size(n_tokens, top_k, n_experts, &need)) return st;
    const int64_t n = n_tokens * top_k;
    if (!offsets || (n > 0 && (!experts || !order || !position))) return VSPMM_ERR_NULL;
    if (need > 0 && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255)))
        return VSPMM_ERR_WORKSPACE;
    const int bins = int(n_experts) + 1;
    if (n == 0) {
        const ZeroRows z(offsets, 0, 1, int64_t(bins) * 4);
        hipLaunchKernelGGL(k_zero, dim3(z.blocks(kThreads)), dim3(kThreads), 0, stream, z);
        return launched();
    }
    const int piece = bin_piece(n), nb = bin_blocks(n);
    with_index(index, [&](auto i) {
        using I = decltype(i);
        int *counts = static_cast<int *>(ws);
        const BinPass<I> p{static_cast<const I *>(experts), n, n_experts, -1, bins, piece, nb};
        if (nb > 1)
            hipLaunchKernelGGL(k_bin_count<I>, dim3(nb), dim3(kBinThreads), size_t(bins) * 4, stream,
                               p, counts, static_cast<int *>(nullptr), ZeroRows());
        allow_dynamic(reinterpret_cast<const void *>(&k_bin_place<I, PlaceRoute>), bin_lds(bins));
        hipLaunchKernelGGL((k_bin_place<I, PlaceRoute>), dim3(nb), dim3(kBinThreads), bin_lds(bins),
                           stream, p, bits_of(n_experts), counts, PlaceRoute{order, position}, offsets);
    });
    return launched();
}

vspmm_status vspmm_dispatch(vspmm_elt elt, int64_t n_tokens, int64_t top_k, int64_t width,
                            const void *x, int64_t ld_x, const int32_t *position, void *rows,
                            int64_t ld_rows, hipStream_t stream) {
    if (!known_elt(elt)) return VSPMM_ERR_ENUM;
    if (!fits(n_tokens) || !fits(top_k) || !fits(n_tokens * top_k)) return VSPMM_ERR_DIM;
    const int64_t n = n_tokens * top_k;
    if (vspmm_status st = check_rows(n > 0 ? n_tokens : 0, width, ld_x, x)) return st;
    if (vspmm_status st = check_out(n, width, ld_rows, rows)) return st;
    if (n > 0 && !position) return VSPMM_ERR_NULL;
    if (n == 0 || width == 0) return VSPMM_OK;
    with_elt(elt, [&](auto e) {
        using T = decltype(e);
        with_chunk<T>(width, [&](auto chunk) {
            constexpr int C = decltype(chunk)::value;
            by_rows<C>(n_tokens, width, [&](int64_t r0, Chunks ch) {
                hipLaunchKernelGGL((k_dispatch<T, C>), dim3(blocks_of(ch.n, kThreads)), dim3(kThreads),
                                   0, stream, static_cast<const T *>(x) + r0 * ld_x, ld_x,
                                   position + r0 * top_k, int(top_k), uint32_t(n), ch,
                                   static_cast<T *>(rows), ld_rows);
            });
        });
    });
    return launched();
}

vspmm_status vspmm_combine(vspmm_elt elt, int64_t n_tokens, int64_t top_k, int64_t width,
                           const void *rows, int64_t ld_rows, const int32_t *position,
                           const void *weight, void *out, int64_t ld_out, hipStream_t stream) {
    if (!known_elt(elt)) return VSPMM_ERR_ENUM;
    if (!fits(n_tokens) || !fits(top_k) || !fits(n_tokens * top_k)) return VSPMM_ERR_DIM;
    const int64_t n = n_tokens * top_k;
    if (vspmm_status st = check_rows(n, width, ld_rows, rows)) return st;
    if (vspmm_status st = check_out(n_tokens, width, ld_out, out)) return st;
    if (n > 0 && !position) return VSPMM_ERR_NULL;
    if (n_tokens == 0 || width == 0) return VSPMM_OK;
    with_elt(elt, [&](auto e) {
        using T = decltype(e);
        using A = typename Sum<T>::type;
        with_chunk<T>(width, [&](auto chunk) {
            constexpr int C = decltype(chunk)::value;
            by_rows<C>(n_tokens, width, [&](int64_t r0, Chunks ch) {
                auto go = [&](auto weighted, auto once) {
                    constexpr bool W = decltype(weighted)::value, ONCE = decltype(once)::value;
                    hipLaunchKernelGGL((k_combine<T, C, W, ONCE>), dim3(blocks_of(ch.n, kThreads)),
                                       dim3(kThreads), 0, stream, static_cast<const T *>(rows),
                                       ld_rows, position + r0 * top_k,
                                       W ? static_cast<const A *>(weight) + r0 * top_k : nullptr,
                                       int(top_k), uint32_t(n), ch,
                                       static_cast<T *>(out) + r0 * ld_out, ld_out);
                };
                auto pick = [&](auto once) {
                    if (weight) go(std::true_type{}, once);
                    else go(std::false_type{}, once);
                };
                if (streams(n, width, elt)) pick(std::true_type{});
                else pick(std::false_type{});
            });
        });
    });
    return launched();
}

vspmm_status vspmm_combine_grad(vspmm_elt elt, int64_t n_tokens, int64_t top_k, int64_t width,
                                const void *dout, int64_t ld_dout, const void *rows,
                                int64_t ld_rows, const int32_t *position, const void *weight,
                                void *grad_rows, int64_t ld_grad_rows, void *grad_weight,
                                hipStream_t stream) {
    if (!known_elt(elt)) return VSPMM_ERR_ENUM;
    if (!fits(n_tokens) || !fits(top_k) || !fits(n_tokens * top_k)) return VSPMM_ERR_DIM;
    const int64_t n = n_tokens * top_k;
    if (vspmm_status st = check_rows(n > 0 ? n_tokens : 0, width, ld_dout, dout)) return st;
    if (vspmm_status st = check_rows(n, width, ld_rows, rows)) return st;
    if (vspmm_status st = check_out(n, width, ld_grad_rows, grad_rows)) return st;
    if (n > 0 && (!position || !weight || !grad_weight)) return VSPMM_ERR_NULL;
    if (n == 0) return VSPMM_OK;
    with_elt(elt, [&](auto e) {
        using T = decltype(e);
        using A = typename Sum<T>::type;
        with_chunk<T>(width, [&](auto chunk) {
            constexpr int C = decltype(chunk)::value;
            const uint32_t cpr = uint32_t((width + C - 1) / C);
            auto go = [&](auto waves, auto once) {
                constexpr int W = decltype(waves)::value;
                constexpr bool ONCE = decltype(once)::value;
                const int64_t most = int64_t(1) << 22;  // tokens a launch
                for (int64_t t0 = 0; t0 < n_tokens; t0 += most) {
                    const uint32_t count = uint32_t(std::min(most, n_tokens - t0));
                    const int64_t s0 = t0 * top_k;
                    hipLaunchKernelGGL((k_combine_grad<T, C, W, ONCE>),
                                       dim3(blocks_of(count, kThreads / 64 / W)), dim3(kThreads), 0,
                                       stream, static_cast<const T *>(dout) + t0 * ld_dout, ld_dout,
                                       static_cast<const T *>(rows), ld_rows, position + s0,
                                       static_cast<const A *>(weight) + s0, int(top_k), uint32_t(n),
                                       count, uint32_t(width), cpr, static_cast<T *>(grad_rows),
                                       ld_grad_rows, static_cast<A *>(grad_weight) + s0);
                }
            };
            // a wave per 64 chunks of the width, as far as the block's four go
            auto pick = [&](auto once) {
                if (cpr > 128) go(std::integral_constant<int, 4>{}, once);
                else if (cpr > 64) go(std::integral_constant<int, 2>{}, once);
                else go(std::integral_constant<int, 1>{}, once);
            };
            if (streams(n, width, elt)) pick(std::true_type{});
            else pick(std::false_type{});
        });
    });
    return launched();
}

}  // extern "C"
