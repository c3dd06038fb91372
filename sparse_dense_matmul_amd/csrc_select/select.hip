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
#include "../csrc/launch.hpp"
#include "rows.hpp"

using namespace vspmm;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kI32Max = 2147483647;

// ------------------------------------------------------------------ kernels

// out[t] = scale * table[ids[t]], or zeros for an id outside the table. The
// rows' chunks are one flat list: consecutive lanes take consecutive chunks,
// whatever the width.
template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
k_embed(const T *__restrict__ table, int64_t ld_table, int64_t n_rows, const I *__restrict__ ids,
        uint32_t n_chunks, int width, uint32_t cpr, FastDiv by_cpr, typename Sum<T>::type scale,
        T *__restrict__ out, int64_t ld_out) {
    using A = typename Sum<T>::type;
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= n_chunks) return;
    const uint32_t t = by_cpr.div(g), col = (g - t * cpr) * kChunk<T>;
    const int live = width - int(col);
    const int64_t id = int64_t(ids[t]);
    ChunkOf<T> v{};
    if (id >= 0 && id < n_rows) {
        v = load_chunk(table + id * ld_table + col, live);
#pragma unroll
        for (int i = 0; i < kChunk<T>; ++i) v[i] = T(A(v[i]) * scale);
    }
    store_chunk(out + int64_t(t) * ld_out + col, v, live);
}

// Every row's first `width` elements = 0.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_zero_rows(T *__restrict__ out, int64_t ld, uint32_t n_chunks, int width, uint32_t cpr,
            FastDiv by_cpr) {
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= n_chunks) return;
    const uint32_t t = by_cpr.div(g), col = (g - t * cpr) * kChunk<T>;
    store_chunk(out + int64_t(t) * ld + col, ChunkOf<T>{}, width - int(col));
}

// The gradient of the lookup: sums of dout's rows over runs of equal ids in
// the sorted list of tokens. The list is cut into segments of `seg` places; a
// group of L lanes walks one segment (64 chunks of the width at a time, the
// grid's y picks which). A run inside a segment is written to its row of
// grad; a run cut by a segment's border leaves float partial rows, part[2 s]
// for a run that came in from the left of segment s and part[2 s + 1] for one
// that starts in s and goes on, which k_grad_join adds in order.
template <typename T, typename G, int L, bool ADD>
__global__ void __launch_bounds__(kThreads)
k_grad_rows(const uint32_t *__restrict__ keys, const int *__restrict__ order, int n, int seg,
            uint32_t n_rows, const T *__restrict__ dout, int64_t ld_dout, int width,
            typename Sum<T>::type scale, G *__restrict__ grad, int64_t ld_grad,
            typename Sum<T>::type *__restrict__ part, int64_t ld_part) {
    using A = typename Sum<T>::type;
    constexpr int C = kChunk<T>;
    const int lane = threadIdx.x & (L - 1);
    const int64_t s = int64_t(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
    const int64_t q0 = s * seg;
    const int64_t col = (int64_t(blockIdx.y) * L + lane) * C;
    if (q0 >= n || col >= width) return;
    const int64_t q1 = q0 + seg < n ? q0 + seg : n;
    const int live = int(width - col < C ? width - col : C);
    A acc[C] = {};
    uint32_t key = keys[q0];
    bool open_left = q0 > 0 && keys[q0 - 1] == key;
    auto close = [&](bool open_right) {
        if (key >= n_rows) return;  // ids outside the table sort last
        if (open_left || open_right) {
            A *p = part + (2 * s + (open_left ? 0 : 1)) * ld_part + col;
#pragma unroll
            for (int i = 0; i < C; ++i) p[i] = acc[i];
            return;
        }
        G *g = grad + int64_t(key) * ld_grad + col;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < live) g[i] = G(ADD ? A(g[i]) + acc[i] * scale : acc[i] * scale);
    };
    for (int64_t q = q0; q < q1; ++q) {
        const uint32_t k = keys[q];
        if (k != key) {
            close(false);
            key = k;
            open_left = false;
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = 0;
        }
        if (key >= n_rows) break;
        const ChunkOf<T> v = load_chunk(dout + int64_t(order[q]) * ld_dout + col, live);
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] += A(v[i]);
    }
    close(q1 < n && keys[q1] == key);
}

// The runs that cross segments: the group of the segment a run starts in adds
// its partial rows, left to right.
template <typename T, typename G, int L, bool ADD>
__global__ void __launch_bounds__(kThreads)
k_grad_join(const uint32_t *__restrict__ keys, int n, int seg, uint32_t n_rows, int width,
            typename Sum<T>::type scale, G *__restrict__ grad, int64_t ld_grad,
            const typename Sum<T>::type *__restrict__ part, int64_t ld_part) {
    using A = typename Sum<T>::type;
    constexpr int C = kChunk<T>;
    const int lane = threadIdx.x & (L - 1);
    const int64_t s = int64_t(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
    const int64_t q0 = s * seg, q1 = q0 + seg;
    const int64_t col = (int64_t(blockIdx.y) * L + lane) * C;
    if (q1 >= n || col >= width) return;
    const uint32_t key = keys[q1];
    if (key >= n_rows || keys[q1 - 1] != key) return;         // no run crosses out of s
    if (q0 > 0 && keys[q0] == key && keys[q0 - 1] == key) return;  // it started further left
    const int live = int(width - col < C ? width - col : C);
    A acc[C];
    const A *p = part + (2 * s + 1) * ld_part + col;
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = p[i];
    for (int64_t j = s + 1; j * seg < n && keys[j * seg] == key; ++j) {
        p = part + 2 * j * ld_part + col;
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] += p[i];
    }
    G *g = grad + int64_t(key) * ld_grad + col;
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (i < live) g[i] = G(ADD ? A(g[i]) + acc[i] * scale : acc[i] * scale);
}

// rows[position[t, k]] = x[t]; a dropped slot (~p) has row p zeroed. A
// position past the last row is passed over.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_dispatch(const T *__restrict__ x, int64_t ld_x, const int *__restrict__ position, int top_k,
           uint32_t n_slots, uint32_t n_chunks, int width, uint32_t cpr, FastDiv by_cpr,
           T *__restrict__ rows, int64_t ld_rows) {
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= n_chunks) return;
    const uint32_t t = by_cpr.div(g), col = (g - t * cpr) * kChunk<T>;
    const int live = width - int(col);
    const ChunkOf<T> v = load_chunk(x + int64_t(t) * ld_x + col, live);
    const int *pos = position + int64_t(t) * top_k;
    for (int k = 0; k < top_k; ++k) {
        const int p = pos[k];
        const uint32_t row = uint32_t(p >= 0 ? p : ~p);
        if (row < n_slots)
            store_chunk(rows + int64_t(row) * ld_rows + col, p >= 0 ? v : ChunkOf<T>{}, live);
    }
}

// out[t] = sum over k of weight[t, k] * rows[position[t, k]] (weight null:
// ones), k ascending, live slots only; one rounding at the end.
template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads)
k_combine(const T *__restrict__ rows, int64_t ld_rows, const int *__restrict__ position,
          const typename Sum<T>::type *__restrict__ weight, int top_k, uint32_t n_slots,
          uint32_t n_chunks, int width, uint32_t cpr, FastDiv by_cpr, T *__restrict__ out,
          int64_t ld_out) {
    using A = typename Sum<T>::type;
    constexpr int C = kChunk<T>;
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= n_chunks) return;
    const uint32_t t = by_cpr.div(g), col = (g - t * cpr) * C;
    const int live = width - int(col);
    const int64_t slot = int64_t(t) * top_k;
    A acc[C] = {};
    for (int k = 0; k < top_k; ++k) {
        const uint32_t p = uint32_t(position[slot + k]);
        if (p >= n_slots) continue;  // dropped
        const ChunkOf<T> v = load_chunk(rows + int64_t(p) * ld_rows + col, live);
        const A w = WEIGHTED ? weight[slot + k] : A(1);
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = WEIGHTED ? fma(w, A(v[i]), acc[i]) : acc[i] + A(v[i]);
    }
    ChunkOf<T> v;
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = T(acc[i]);
    store_chunk(out + int64_t(t) * ld_out + col, v, live);
}

// Gradients of the combine: grad_rows[position[t, k]] = weight[t, k] *
// dout[t] and grad_weight[t, k] = <dout[t], rows[position[t, k]]>; a dropped
// slot's row and weight gradient are zero. One block per token; the dots' lane
// sums are added by a butterfly, then wave by wave: a fixed order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_combine_grad(const T *__restrict__ dout, int64_t ld_dout, const T *__restrict__ rows,
               int64_t ld_rows, const int *__restrict__ position,
               const typename Sum<T>::type *__restrict__ weight, int top_k, uint32_t n_slots,
               int width, T *__restrict__ grad_rows, int64_t ld_grad_rows,
               typename Sum<T>::type *__restrict__ grad_weight) {
    using A = typename Sum<T>::type;
    constexpr int C = kChunk<T>;
    __shared__ A sums[kThreads / 64];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int k = 0; k < top_k; ++k) {
        const int64_t slot = t * top_k + k;
        const int p = position[slot];
        const uint32_t row = uint32_t(p >= 0 ? p : ~p);
        const bool there = row < n_slots, kept = there && p >= 0;
        const A w = weight[slot];
        A dot = 0;
        if (there) {
            for (int64_t col = int64_t(threadIdx.x) * C; col < width; col += kThreads * C) {
                const int live = int(width - col < C ? width - col : C);
                const ChunkOf<T> d = load_chunk(dout + t * ld_dout + col, live);
                ChunkOf<T> o{};
                if (kept) {
                    const ChunkOf<T> y = load_chunk(rows + int64_t(row) * ld_rows + col, live);
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        dot = fma(A(d[i]), A(y[i]), dot);
                        o[i] = T(w * A(d[i]));
                    }
                }
                store_chunk(grad_rows + int64_t(row) * ld_grad_rows + col, o, live);
            }
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) dot += __shfl_xor(dot, m);
        if (lane == 0) sums[wave] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            A all = sums[0];
#pragma unroll
            for (int w2 = 1; w2 < kThreads / 64; ++w2) all += sums[w2];
            grad_weight[slot] = all;
        }
        __syncthreads();
    }
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

// Rows [r0, r0 + count) at a time, so that a launch has fewer than 2^31 chunks.
template <typename F>
void by_rows(int64_t n, uint32_t cpr, F &&f) {
    const int64_t most = std::max<int64_t>(1, (kI32Max - (1 << 20)) / cpr);
    for (int64_t r0 = 0; r0 < n; r0 += most) f(r0, std::min(most, n - r0));
}
template <typename T>
uint32_t chunks_of(int64_t width) {
    return uint32_t((width + kChunk<T> - 1) / kChunk<T>);
}
unsigned blocks_of(uint32_t n_chunks) { return (n_chunks + kThreads - 1) / kThreads; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

void allow_dynamic(const void *fn, size_t bytes) {
    if (bytes > 64 * 1024) allow_lds(fn);
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

// A segment of the sorted tokens in k_grad_rows.
int segment_of(int64_t, int64_t) { return 32; }

struct GradWs {
    uint32_t *keys[2];
    int *pay[2];
    int *counts;
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
    for (int i = 0; i < 2; ++i) w.keys[i] = reinterpret_cast<uint32_t *>(take(size_t(n) * 4));
    for (int i = 0; i < 2; ++i) w.pay[i] = reinterpret_cast<int *>(take(size_t(n) * 4));
    w.counts = reinterpret_cast<int *>(take((size_t(4) * bin_blocks(n)) << passes_for(n_rows).bits));
    const int c = 16 / elt_bytes(elt);
    w.ld_part = (width + c - 1) / c * c;
    const int seg = segment_of(n, width);
    const size_t segs = size_t((n + seg - 1) / seg);
    w.part = take(2 * segs * size_t(w.ld_part) * (elt == VSPMM_ELT_F64 ? 8 : 4));
    w.bytes = at;
    return w;
}

vspmm_status check_rows(int64_t n, int64_t width, int64_t ld, const void *p) {
    if (!fits(n) || !fits(width) || ld < 0) return VSPMM_ERR_DIM;
    if (n > 0 && width > 0 && !p) return VSPMM_ERR_NULL;
    return VSPMM_OK;
}
// Rows that are written must not overlap.
vspmm_status check_out(int64_t n, int64_t width, int64_t ld, const void *p) {
    if (n > 1 && ld < width) return VSPMM_ERR_DIM;
    return check_rows(n, width, ld, p);
}

template <typename T, typename G, bool ADD>
void launch_grad(const GradWs &w, const uint32_t *keys, const int *order, int64_t n, int seg,
                 int64_t n_rows, const void *dout, int64_t ld_dout, int64_t width, double scale,
                 void *grad, int64_t ld_grad, hipStream_t s) {
    using A = typename Sum<T>::type;
    const int64_t segs = (n + seg - 1) / seg;
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const dim3 grid(unsigned((segs + kThreads / L - 1) / (kThreads / L)),
                        unsigned((chunks_of<T>(width) + L - 1) / L));
        hipLaunchKernelGGL((k_grad_rows<T, G, L, ADD>), grid, dim3(kThreads), 0, s, keys, order,
                           int(n), seg, uint32_t(n_rows), static_cast<const T *>(dout), ld_dout,
                           int(width), A(scale), static_cast<G *>(grad), ld_grad,
                           static_cast<A *>(w.part), w.ld_part);
        hipLaunchKernelGGL((k_grad_join<T, G, L, ADD>), grid, dim3(kThreads), 0, s, keys, int(n),
                           seg, uint32_t(n_rows), int(width), A(scale), static_cast<G *>(grad),
                           ld_grad, static_cast<const A *>(w.part), w.ld_part);
    };
    if (chunks_of<T>(width) > 16) go(std::integral_constant<int, 64>{});
    else go(std::integral_constant<int, 16>{});
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
            const uint32_t cpr = chunks_of<T>(width);
            by_rows(n, cpr, [&](int64_t r0, int64_t count) {
                const uint32_t chunks = uint32_t(count) * cpr;
                hipLaunchKernelGGL((k_embed<T, I>), dim3(blocks_of(chunks)), dim3(kThreads), 0,
                                   stream, static_cast<const T *>(table), ld_table, n_rows,
                                   static_cast<const I *>(ids) + r0, chunks, int(width), cpr,
                                   FastDiv(cpr), typename Sum<T>::type(scale),
                                   static_cast<T *>(out) + r0 * ld_out, ld_out);
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
    if (!accumulate)
        with_elt(grad_elt, [&](auto e) {
            using G = decltype(e);
            const uint32_t cpr = chunks_of<G>(width);
            by_rows(n_rows, cpr, [&](int64_t r0, int64_t count) {
                const uint32_t chunks = uint32_t(count) * cpr;
                hipLaunchKernelGGL(k_zero_rows<G>, dim3(blocks_of(chunks)), dim3(kThreads), 0,
                                   stream, static_cast<G *>(grad) + r0 * ld_grad, ld_grad, chunks,
                                   int(width), cpr, FastDiv(cpr));
            });
        });
    if (n == 0) return launched();
    const GradWs w = carve_grad(elt, n_rows, width, n, ws);
    const Passes ps = passes_for(n_rows);
    const int piece = bin_piece(n), nb = bin_blocks(n), bins = 1 << ps.bits;
    const size_t lds = bin_lds(bins);
    const uint32_t *keys = nullptr;
    const int *order = nullptr;
    auto pass = [&](auto *src, int k) {
        using I = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
        hipLaunchKernelGGL(k_bin_count<I>, dim3(nb), dim3(kBinThreads), size_t(bins) * 4, stream,
                           src, n, n_rows, k * ps.bits, bins, piece, w.counts);
        allow_dynamic(reinterpret_cast<const void *>(&k_bin_place<I, PlaceKeys>), lds);
        const PlaceKeys to{w.keys[k & 1], w.pay[k & 1], order};
        hipLaunchKernelGGL((k_bin_place<I, PlaceKeys>), dim3(nb), dim3(kBinThreads), lds, stream,
                           src, n, n_rows, k * ps.bits, bins, ps.bits, piece, w.counts, to,
                           static_cast<int *>(nullptr));
        keys = to.keys;
        order = to.pay;
    };
    with_index(index, [&](auto i) { pass(static_cast<const decltype(i) *>(ids), 0); });
    for (int k = 1; k < ps.count; ++k) pass(keys, k);
    const int seg = segment_of(n, width);
    auto sum = [&](auto e, auto g) {
        using T = decltype(e);
        using G = decltype(g);
        if (accumulate)
            launch_grad<T, G, true>(w, keys, order, n, seg, n_rows, dout, ld_dout, width, scale,
                                    grad, ld_grad, stream);
        else
            launch_grad<T, G, false>(w, keys, order, n, seg, n_rows, dout, ld_dout, width, scale,
                                     grad, ld_grad, stream);
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
    *bytes = up256(size_t(4) * bin_blocks(n_tokens * top_k) * size_t(n_experts + 1));
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
        const uint32_t chunks = chunks_of<int>(bins);
        hipLaunchKernelGGL(k_zero_rows<int>, dim3(blocks_of(chunks)), dim3(kThreads), 0, stream,
                           offsets, int64_t(bins), chunks, bins, chunks, FastDiv(chunks));
        return launched();
    }
    const int piece = bin_piece(n), nb = bin_blocks(n);
    const size_t lds = bin_lds(bins);
    with_index(index, [&](auto i) {
        using I = decltype(i);
        int *counts = static_cast<int *>(ws);
        hipLaunchKernelGGL(k_bin_count<I>, dim3(nb), dim3(kBinThreads), size_t(bins) * 4, stream,
                           static_cast<const I *>(experts), n, n_experts, -1, bins, piece, counts);
        allow_dynamic(reinterpret_cast<const void *>(&k_bin_place<I, PlaceRoute>), lds);
        hipLaunchKernelGGL((k_bin_place<I, PlaceRoute>), dim3(nb), dim3(kBinThreads), lds, stream,
                           static_cast<const I *>(experts), n, n_experts, -1, bins,
                           bits_of(n_experts), piece, counts, PlaceRoute{order, position}, offsets);
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
        const uint32_t cpr = chunks_of<T>(width);
        by_rows(n_tokens, cpr, [&](int64_t r0, int64_t count) {
            const uint32_t chunks = uint32_t(count) * cpr;
            hipLaunchKernelGGL(k_dispatch<T>, dim3(blocks_of(chunks)), dim3(kThreads), 0, stream,
                               static_cast<const T *>(x) + r0 * ld_x, ld_x, position + r0 * top_k,
                               int(top_k), uint32_t(n), chunks, int(width), cpr, FastDiv(cpr),
                               static_cast<T *>(rows), ld_rows);
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
        const uint32_t cpr = chunks_of<T>(width);
        by_rows(n_tokens, cpr, [&](int64_t r0, int64_t count) {
            const uint32_t chunks = uint32_t(count) * cpr;
            auto go = [&](auto weighted) {
                constexpr bool W = decltype(weighted)::value;
                hipLaunchKernelGGL((k_combine<T, W>), dim3(blocks_of(chunks)), dim3(kThreads), 0,
                                   stream, static_cast<const T *>(rows), ld_rows,
                                   position + r0 * top_k,
                                   W ? static_cast<const A *>(weight) + r0 * top_k : nullptr,
                                   int(top_k), uint32_t(n), chunks, int(width), cpr, FastDiv(cpr),
                                   static_cast<T *>(out) + r0 * ld_out, ld_out);
            };
            if (weight) go(std::true_type{});
            else go(std::false_type{});
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
        hipLaunchKernelGGL(k_combine_grad<T>, dim3(unsigned(n_tokens)), dim3(kThreads), 0, stream,
                           static_cast<const T *>(dout), ld_dout, static_cast<const T *>(rows),
                           ld_rows, position, static_cast<const A *>(weight), int(top_k),
                           uint32_t(n), int(width), static_cast<T *>(grad_rows), ld_grad_rows,
                           static_cast<A *>(grad_weight));
    });
    return launched();
}

}  // extern "C"
