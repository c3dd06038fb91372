// The embedding's gradient over the sorted list of its tokens: sums of dout's
// rows over runs of equal ids. Memory bound: 65,536 tokens of 4,096 bf16 (540 MB
// read, 172 MB of selected rows and partial ones written) take 148 us behind the
// zeroing of 1.07 GB, whose last 256 MB still leave the last-level cache then; the
// whole call moves 1.79 GB in 335 us, 5.3 TB/s.
//
// The list is cut into segments of `seg` places. A group of L lanes walks one
// segment for L chunks of the width (a slice), eight rows in flight. A run
// inside a segment goes to its row of grad, and so does one that crosses a
// single border, summed whole in the segment it starts in. A run over two
// borders or more leaves partial rows of the sums' type, part[2 s + 1] in the
// segment s it starts in and part[2 s] in those it comes into from the left, and
// the former is listed for k_grad_join, which adds a listed run's partial rows:
// L-lane groups a contiguous share each, the shares in order. Segments, shares
// and so the order of every sum depend only on the ids and sizes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rows.hpp"

namespace vspmm {

constexpr int kGradThreads = 256;
constexpr int kJoinThreads = 512;
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
                if (i >= int(moved)) g[i] = rounded<G>(fma(acc[i], scale, A(g[i])));
            return;
        }
        const Vec<G, C> old = load_vec<C>(g);
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = rounded<G>(fma(acc[i], scale, A(old[i])));
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = rounded<G>(acc[i] * scale);
    }
    store_vec<C>(g, o);
}

// A group's C sums per lane as 16-byte pieces, all lanes' first pieces, then
// their second ones: every access of the group is contiguous.
template <int C, int L, typename A>
__device__ __forceinline__ void write_part(A *group, int lane, const A *acc) {
    constexpr int P = C * sizeof(A) < 16 ? C : int(16 / sizeof(A));
#pragma unroll
    for (int k = 0; k < C / P; ++k) {
        Vec<A, P> o;
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = acc[k * P + i];
        store_vec<P>(group + (k * L + lane) * P, o);
    }
}
template <int C, int L, typename A>
__device__ __forceinline__ Vec<A, C> read_part(const A *group, int lane) {
    constexpr int P = C * sizeof(A) < 16 ? C : int(16 / sizeof(A));
    Vec<A, C> v;
#pragma unroll
    for (int k = 0; k < C / P; ++k) {
        const Vec<A, P> o = load_vec<P>(group + (k * L + lane) * P);
#pragma unroll
        for (int i = 0; i < P; ++i) v[k * P + i] = o[i];
    }
    return v;
}

// What the sums need of the sorted list and the arrays.
template <typename T, typename G>
struct GradArgs {
    const uint32_t *keys;
    const int *order;
    int n, seg, segs;
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

template <typename T, typename G, int C, int L, bool ADD>
__global__ void __launch_bounds__(kGradThreads) k_grad_rows(GradArgs<T, G> a) {
    using A = typename Sum<T>::type;
    const int lane = threadIdx.x & (L - 1);
    const uint32_t unit = blockIdx.x * (kGradThreads / L) + threadIdx.x / L;
    const uint32_t s = a.by_slices.div(unit), slice = unit - s * a.slices;
    const int64_t q0 = int64_t(s) * a.seg;
    if (q0 >= a.n) return;  // a whole group
    const int cnt = int(a.n - q0 < a.seg ? a.n - q0 : a.seg);
    auto key_at = [&](int64_t q) { return q >= 0 && q < a.n ? a.keys[q] : ~0u; };
    // this segment's places and the next one's, a lane each, and the keys around
    const int64_t q1 = q0 + a.seg;
    const uint32_t mine = lane < cnt ? a.keys[q0 + lane] : ~0u;
    const int token = lane < cnt ? a.order[q0 + lane] : 0;
    const bool in_next = lane < a.seg && q1 + lane < a.n;
    const uint32_t next = in_next ? a.keys[q1 + lane] : ~0u;
    const int next_token = in_next ? a.order[q1 + lane] : 0;
    const uint32_t left = key_at(q0 - 1), left2 = key_at(q0 - a.seg - 1), right2 = key_at(q1 + a.seg);
    auto of = [&](auto x, int j) {
        if constexpr (L == 64) return decltype(x)(__builtin_amdgcn_readlane(int(x), j));
        else return decltype(x)(__shfl(int(x), j, L));
    };
    // of this group's lanes: places where a run starts, live places
    const int shift = L == 64 ? 0 : (threadIdx.x & 63) & ~(L - 1);
    constexpr uint64_t group = L == 64 ? ~0ull : (1ull << (L & 63)) - 1;
    auto vote = [&](bool x) { return (__ballot(x) >> shift) & group; };
    const uint32_t before = uint32_t(__shfl_up(int(mine), 1, L));
    const uint64_t starts = vote(lane > 0 && lane < cnt && mine != before);
    const int live_places = __popcll(vote(mine < a.n_rows));
    if (live_places == 0) return;
    // the first run: cut by the left border, and all the left segment's if it
    // starts there and ends here
    const uint32_t right = of(next, 0);
    const uint32_t first = of(mine, 0), last = of(mine, live_places - 1);
    bool open_left = left == first;
    int q = 0;
    if (open_left && left2 != first && right != first) {
        q = starts ? __ffsll((unsigned long long)starts) - 1 : cnt;
        open_left = false;
        if (q >= live_places) return;
    }
    // the last run: cut by the right border, and this segment's if it starts
    // here and ends in the next
    const bool open_right = live_places == cnt && right == last;
    const bool taken = open_right && (starts != 0 || !open_left) && right2 != last;
    const int more = taken ? __popcll(vote(next == last)) : 0;

    // lanes past the width load the last chunk again and write nothing
    const uint32_t c = slice * L + lane;
    const uint32_t col = chunk_col<C>(c < a.cpr ? c : a.cpr - 1, a.width);
    const T *x = a.dout + col;
    A acc[C] = {};
    auto close = [&](uint32_t key, bool cut) {
        if (open_left || cut) {
            write_part<C, L>(a.part + (2 * int64_t(s) + (open_left ? 0 : 1)) * a.ld_part +
                                 int64_t(slice) * L * C, lane, acc);
            if (!open_left && slice == 0 && lane == 0) a.list[atomicAdd(a.listed, 1)] = int(s);
        } else if (c < a.cpr) {
            write_grad<G, C, ADD>(a.grad + int64_t(key) * a.ld_grad + col, acc, a.scale, c * C - col);
        }
    };
    const int begin = q;
    auto add = [&](int at, Vec<T, C> v) {  // place `at`, or past cnt one of the next segment's
        if (at > begin && at < cnt && ((starts >> at) & 1)) {
            close(of(mine, at - 1), false);
            open_left = false;
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] += A(v[i]);
    };
    auto row = [&](int at) {
        const int t = at < cnt ? of(token, at) : of(next_token, at - cnt);
        return load_once<C>(x + int64_t(t) * a.ld_dout);
    };
    // dout's rows are read once: nontemporal, 345 -> 317 us for 65,536 tokens of
    // 4,096 bf16, 95 -> 80 for 16,384 of 2,048, never slower
    const int end = live_places + more;  // more > 0 only behind cnt live places
    for (; q + kGradRows <= end; q += kGradRows) {
        Vec<T, C> v[kGradRows];
#pragma unroll
        for (int u = 0; u < kGradRows; ++u) v[u] = row(q + u);
#pragma unroll
        for (int u = 0; u < kGradRows; ++u) add(q + u, v[u]);
    }
    if (q < end) {
        Vec<T, C> v[kGradRows];
#pragma unroll
        for (int u = 0; u < kGradRows - 1; ++u)
            if (q + u < end) v[u] = row(q + u);
#pragma unroll
        for (int u = 0; u < kGradRows - 1; ++u)
            if (q + u < end) add(q + u, v[u]);
    }
    close(last, open_right && !taken);
}

// Sums of the groups' acc in group order, in group 0.
template <int C, int L, int GROUPS, typename A>
__device__ __forceinline__ void add_groups(A *sums, A (&acc)[C], int group, int lane) {
    write_part<C, L>(sums + group * L * C, lane, acc);
    __syncthreads();
    if (group == 0) {
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) {
            const Vec<A, C> v = read_part<C, L>(sums + g * L * C, lane);
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] += v[i];
        }
    }
}

// acc += the partial rows at(p) for p in [p0, p1), eight in flight.
template <int C, int L, typename A, typename F>
__device__ __forceinline__ void add_parts(A (&acc)[C], int p0, int p1, int lane, F &&at) {
    for (int p = p0; p < p1; p += kGradRows) {
        Vec<A, C> v[kGradRows];
#pragma unroll
        for (int u = 0; u < kGradRows; ++u)
            if (p + u < p1) v[u] = read_part<C, L>(at(p + u), lane);
#pragma unroll
        for (int u = 0; u < kGradRows; ++u)
            if (p + u < p1) {
#pragma unroll
                for (int i = 0; i < C; ++i) acc[i] += v[u][i];
            }
    }
}

// In a long list (kFoldSegs segments or more) the partial rows of kFold
// segments at a time, from a multiple of kFold on, are added first where one run
// fills them all and goes on: the sum replaces the first one's row. A run of
// 1,000,000 tokens of 1,024 bf16 then leaves 370 rows to its join and not 15,625:
// 735 -> 457 us, half as many among others 606 -> 467, none 455 -> 459.
constexpr int kFold = 64;
constexpr int kFoldSegs = 4096;

template <typename T, typename G, int C, int L>
__global__ void __launch_bounds__(kJoinThreads) k_grad_fold(GradArgs<T, G> a) {
    using A = typename Sum<T>::type;
    constexpr int GROUPS = kJoinThreads / L, PER = kFold / GROUPS;
    __shared__ __align__(16) A sums[kJoinThreads * C];
    const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
    const int64_t s = (int64_t(blockIdx.x) + 1) * kFold;  // the first segments have no left
    const int64_t q0 = s * a.seg, q1 = (s + kFold) * a.seg;
    if (q1 >= a.n) return;
    const uint32_t key = a.keys[q1];
    if (key >= a.n_rows || a.keys[q0 - 1] != key) return;  // a block's threads alike
    A *const part = a.part + 2 * s * a.ld_part + int64_t(blockIdx.y) * L * C;
    A acc[C] = {};
    add_parts<C, L>(acc, group * PER, (group + 1) * PER, lane,
                    [&](int p) { return part + 2 * int64_t(p) * a.ld_part; });
    add_groups<C, L, GROUPS>(sums, acc, group, lane);
    if (group == 0) write_part<C, L>(part, lane, acc);
}

template <typename T, typename G, int C, int L, bool ADD>
__global__ void __launch_bounds__(kJoinThreads) k_grad_join(GradArgs<T, G> a) {
    using A = typename Sum<T>::type;
    constexpr int GROUPS = kJoinThreads / L;
    __shared__ __align__(16) A sums[kJoinThreads * C];
    const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
    const int listed = *a.listed;
    for (int64_t it = blockIdx.x; it < int64_t(a.segs) * a.slices; it += gridDim.x) {
        const int64_t e = it / a.slices;
        const uint32_t slice = uint32_t(it - e * a.slices);
        const int s = a.list[e];  // loaded beside `listed`: used below it alone
        if (e >= listed) return;
        // partial rows: the tail of s, then the heads of the segments whose first
        // key is still the run's, found by probes of 64 borders, next to each other
        // at first (most runs end there), then spread over what is left
        const int wl = threadIdx.x & 63;
        uint32_t key = 0;
        int lo = s + 1, hi = a.segs;  // the first border behind the run lies in [lo, hi]
        for (int step = 1; lo < hi; step = (hi - lo + 63) / 64) {
            const int64_t j = int64_t(lo) + int64_t(wl) * step;
            const uint32_t k = j < hi ? a.keys[j * a.seg] : ~0u;
            if (lo == s + 1) key = __builtin_amdgcn_readlane(k, 0);
            const uint64_t other = __ballot(j >= hi || k != key);
            const int f = other ? __ffsll((unsigned long long)other) - 1 : 64;  // first past it
            if (f == 0) break;
            const int64_t top = int64_t(lo) + int64_t(f) * step;
            lo += (f - 1) * step + 1;
            if (f < 64 && top < hi) hi = int(top);
        }
        const int parts = lo - s;
        // those in folded blocks (from segment `fold0` on, `folds` of them) are one each
        int fold0 = s + parts, folds = 0;
        if (a.segs >= kFoldSegs) {
            const int f0 = (s + kFold) / kFold * kFold, last = s + parts - 1;
            if (f0 + kFold <= last) {
                fold0 = f0;
                folds = (last - f0) / kFold;
            }
        }
        const int rows = parts - folds * (kFold - 1);
        const int per = (rows + GROUPS - 1) / GROUPS;
        const int p0 = group * per, p1 = p0 + per < rows ? p0 + per : rows;
        const uint32_t c = slice * L + lane;
        A acc[C] = {};
        add_parts<C, L>(acc, p0, p1, lane, [&](int p) {
            int64_t j = int64_t(s) + p;  // the p-th row's segment
            if (j >= fold0) {
                const int64_t f = j - fold0;
                j = f < folds ? fold0 + f * kFold : fold0 + int64_t(folds) * kFold + (f - folds);
            }
            return a.part + (2 * j + (p == 0 ? 1 : 0)) * a.ld_part + int64_t(slice) * L * C;
        });
        add_groups<C, L, GROUPS>(sums, acc, group, lane);
        if (group == 0 && c < a.cpr) {
            const uint32_t col = chunk_col<C>(c, a.width);
            write_grad<G, C, ADD>(a.grad + int64_t(key) * a.ld_grad + col, acc, a.scale, c * C - col);
        }
        __syncthreads();
    }
}

}  // namespace vspmm
