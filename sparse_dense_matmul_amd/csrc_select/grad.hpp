// The embedding's gradient over the sorted list of its tokens: sums of dout's
// rows over runs of equal ids. Memory bound: every dout row is read once and
// every row of the table's gradient written once.
//
// The list is cut into segments of `seg` places. A group of L lanes walks one
// segment for L chunks of the width (a slice), eight rows in flight. A run
// inside a segment goes to its row of grad; a run cut by a segment's border
// leaves partial rows of the sums' type, part[2 s] for a run that came into
// segment s from the left and part[2 s + 1] for one that starts in s and goes
// on, and s is listed for k_grad_join, which adds a listed run's partial rows:
// L-lane groups a contiguous share each, the shares in order. Segments, shares
// and so the order of every sum depend only on the ids and sizes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rows.hpp"

namespace vspmm {

constexpr int kGradThreads = 256;
constexpr int kGradRows = 8;  // rows in flight per group

// C sums to a row of the gradient. Of a chunk moved left by `moved` elements,
// an addition leaves those to the chunk before.
template <typename G, int C, bool ADD, typename A>
__device__ __forceinline__ void write_grad(G *g, const A *acc, A scale, uint32_t moved) {
    Vec<G, C> o;
    if constexpr (ADD) {
        if (moved) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (i >= int(moved)) g[i] = G(fma(acc[i], scale, A(g[i])));
            return;
        }
        const Vec<G, C> old = load_vec<C>(g);
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = G(fma(acc[i], scale, A(old[i])));
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = G(acc[i] * scale);
    }
    store_vec<C>(g, o);
}

template <int C, typename A>
__device__ __forceinline__ void write_part(A *p, const A *acc) {
    Vec<A, C> o;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = acc[i];
    store_vec<C>(p, o);
}

// The first place in [lo, n) whose key is above `key` (keys ascending), by all
// lanes of the wave: each round probes 64 places.
__device__ __forceinline__ int wave_upper_bound(const uint32_t *keys, int lo, int n, uint32_t key) {
    const int lane = threadIdx.x & 63;
    int hi = n;  // the answer lies in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 63) / 64;
        const int64_t at = int64_t(lo) + int64_t(lane) * step;
        const uint64_t over = __ballot(at >= hi || keys[at < hi ? at : lo] > key);
        const int f = over ? __ffsll((unsigned long long)over) - 1 : 64;  // first probe above
        if (f == 0) return lo;
        const int64_t top = int64_t(lo) + int64_t(f) * step;
        lo += (f - 1) * step + 1;
        if (f < 64 && top < hi) hi = int(top);
    }
    return lo;
}

// What the sums need of the sorted list and the arrays.
template <typename T, typename G>
struct GradArgs {
    const uint32_t *keys;
    const int *order;
    int n, seg;
    uint32_t n_rows;
    const T *dout;
    int64_t ld_dout;
    int width;
    uint32_t cpr, slices;  // chunks and slices of a row
    FastDiv by_slices{1};
    typename Sum<T>::type scale;
    G *grad;
    int64_t ld_grad;
    typename Sum<T>::type *part;
    int64_t ld_part;
    int *list, *listed;  // segments whose last run goes on; how many
};

// Zeroes the rows of units [zero.lo, zero.hi) that no token selects, by the
// launch's blocks from `first` on.
template <bool ONCE>
__device__ __forceinline__ void zero_unselected(const ZeroShare &zero, unsigned first,
                                                const uint32_t *keys, int n) {
    const int64_t waves = int64_t(gridDim.x - first) * (kGradThreads / 64);
    for (int64_t u = zero.lo + int64_t(blockIdx.x - first) * (kGradThreads / 64) + threadIdx.x / 64;
         u < zero.hi; u += waves) {
        // is row r selected: the first key at or above r, by binary search
        const uint32_t r = uint32_t(u * zero.rows.unit_rows) + (threadIdx.x & 63);
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = int((unsigned(lo) + unsigned(hi)) / 2);
            if (keys[mid] < r) lo = mid + 1;
            else hi = mid;
        }
        const bool there = lo < n && keys[lo] == r;
        zero.rows.unit<ONCE>(u, __ballot(there));
    }
}

// Blocks past `sum_blocks` zero their share of rows.
template <typename T, typename G, int C, int L, bool ADD>
__global__ void __launch_bounds__(kGradThreads)
k_grad_rows(GradArgs<T, G> a, unsigned sum_blocks, ZeroShare zero) {
    using A = typename Sum<T>::type;
    if (!ADD && blockIdx.x >= sum_blocks) {
        if (zero.rows.once) zero_unselected<true>(zero, sum_blocks, a.keys, a.n);
        else zero_unselected<false>(zero, sum_blocks, a.keys, a.n);
        return;
    }
    const int lane = threadIdx.x & (L - 1);
    const uint32_t unit = blockIdx.x * (kGradThreads / L) + threadIdx.x / L;
    const uint32_t s = a.by_slices.div(unit), slice = unit - s * a.slices;
    const int64_t q0 = int64_t(s) * a.seg;
    if (q0 >= a.n) return;  // a whole group
    const int cnt = int(a.n - q0 < a.seg ? a.n - q0 : a.seg);
    const uint32_t mine = lane < cnt ? a.keys[q0 + lane] : ~0u;
    const int token = lane < cnt ? a.order[q0 + lane] : 0;
    const uint32_t left = q0 > 0 ? a.keys[q0 - 1] : ~0u;
    const uint32_t right = q0 + cnt < a.n ? a.keys[q0 + cnt] : ~0u;
    auto of = [&](auto x, int j) {
        if constexpr (L == 64) return decltype(x)(__builtin_amdgcn_readlane(int(x), j));
        else return decltype(x)(__shfl(int(x), j, L));
    };
    // bits of this group: places where a run starts, and live places
    const int shift = L == 64 ? 0 : (threadIdx.x & 63) & ~(L - 1);
    constexpr uint64_t group = L == 64 ? ~0ull : (1ull << (L & 63)) - 1;
    const uint32_t before = uint32_t(__shfl_up(int(mine), 1, L));
    const uint64_t starts = (__ballot(lane > 0 && mine != before) >> shift) & group;
    const int live_places = __popcll((__ballot(mine < a.n_rows) >> shift) & group);
    if (live_places == 0) return;

    // lanes past the width load the last chunk again and write nothing
    const uint32_t c = slice * L + lane;
    const uint32_t col = chunk_col<C>(c < a.cpr ? c : a.cpr - 1, a.width);
    const T *x = a.dout + col;
    A acc[C] = {};
    bool open_left = left == of(mine, 0);
    auto close = [&](uint32_t key, bool open_right) {
        if (open_left || open_right) {
            if (c < a.cpr)
                write_part<C>(a.part + (2 * int64_t(s) + (open_left ? 0 : 1)) * a.ld_part + c * C, acc);
            if (!open_left && slice == 0 && lane == 0) a.list[atomicAdd(a.listed, 1)] = int(s);
        } else if (c < a.cpr) {
            write_grad<G, C, ADD>(a.grad + int64_t(key) * a.ld_grad + col, acc, a.scale, c * C - col);
        }
    };
    auto add = [&](int q, Vec<T, C> v) {
        if ((starts >> q) & 1) {
            close(of(mine, q - 1), false);
            open_left = false;
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] += A(v[i]);
    };
    // dout's rows are read once: nontemporal, 345 -> 317 us for 65,536 tokens of
    // 4,096 bf16, 95 -> 80 for 16,384 of 2,048, never slower
    int q = 0;
    for (; q + kGradRows <= live_places; q += kGradRows) {
        Vec<T, C> v[kGradRows];
#pragma unroll
        for (int u = 0; u < kGradRows; ++u)
            v[u] = load_once<C>(x + int64_t(of(token, q + u)) * a.ld_dout);
#pragma unroll
        for (int u = 0; u < kGradRows; ++u) add(q + u, v[u]);
    }
    if (q < live_places) {
        Vec<T, C> v[kGradRows];
#pragma unroll
        for (int u = 0; u < kGradRows - 1; ++u)
            if (q + u < live_places) v[u] = load_once<C>(x + int64_t(of(token, q + u)) * a.ld_dout);
#pragma unroll
        for (int u = 0; u < kGradRows - 1; ++u)
            if (q + u < live_places) add(q + u, v[u]);
    }
    const uint32_t last = of(mine, live_places - 1);
    close(last, live_places == cnt && right == last);
}

// Blocks past `join_blocks` zero their share of rows.
template <typename T, typename G, int C, int L, bool ADD>
__global__ void __launch_bounds__(kGradThreads)
k_grad_join(GradArgs<T, G> a, unsigned join_blocks, ZeroShare zero) {
    using A = typename Sum<T>::type;
    if (!ADD && blockIdx.x >= join_blocks) {
        if (zero.rows.once) zero_unselected<true>(zero, join_blocks, a.keys, a.n);
        else zero_unselected<false>(zero, join_blocks, a.keys, a.n);
        return;
    }
    constexpr int GROUPS = kGradThreads / L;
    __shared__ __align__(16) A sums[kGradThreads * C];
    const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
    const int64_t items = int64_t(*a.listed) * a.slices;
    for (int64_t it = blockIdx.x; it < items; it += join_blocks) {
        const int s = a.list[it / a.slices];
        const uint32_t slice = uint32_t(it % a.slices);
        const int q1 = (s + 1) * a.seg;  // <= n: the run goes on past it
        const uint32_t key = a.keys[q1];
        const int end = wave_upper_bound(a.keys, q1, a.n, key);
        // partial rows: the tail of s, then the heads of s + 1 .. last
        const int parts = (end - 1) / a.seg - s + 1;
        const int per = (parts + GROUPS - 1) / GROUPS;
        const int p0 = group * per, p1 = p0 + per < parts ? p0 + per : parts;
        const uint32_t c = slice * L + lane;
        const uint32_t cc = c < a.cpr ? c : a.cpr - 1;
        A acc[C] = {};
        for (int p = p0; p < p1; p += kGradRows) {
            Vec<A, C> v[kGradRows];
#pragma unroll
            for (int u = 0; u < kGradRows; ++u)
                if (p + u < p1)
                    v[u] = load_vec<C>(
                        a.part + (2 * int64_t(s + p + u) + (p + u == 0 ? 1 : 0)) * a.ld_part + cc * C);
#pragma unroll
            for (int u = 0; u < kGradRows; ++u)
                if (p + u < p1) {
#pragma unroll
                    for (int i = 0; i < C; ++i) acc[i] += v[u][i];
                }
        }
        write_part<C>(sums + threadIdx.x * C, acc);
        __syncthreads();
        if (group == 0 && c < a.cpr) {
#pragma unroll
            for (int g = 1; g < GROUPS; ++g) {
                const Vec<A, C> v = load_vec<C>(sums + (g * L + lane) * C);
#pragma unroll
                for (int i = 0; i < C; ++i) acc[i] += v[i];
            }
            const uint32_t col = chunk_col<C>(c, a.width);
            write_grad<G, C, ADD>(a.grad + int64_t(key) * a.ld_grad + col, acc, a.scale, c * C - col);
        }
        __syncthreads();
    }
}

}  // namespace vspmm
