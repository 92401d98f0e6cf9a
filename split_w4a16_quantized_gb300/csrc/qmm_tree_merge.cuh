// The states that a merge adds up: which runs hold one of an item, and a row's running
// sum of them.
#pragma once

#include "qmm_tree.cuh"

namespace qmm {

constexpr int kMergeAhead = 4;   // states whose loads a thread has in flight

// Runs that hold a stretch of an item: [c0, c1].
struct Runs {
    int c0, c1;
};
__device__ __forceinline__ Runs runs_of(const TreeParams& p, const Seq& s, long long before,
                                        int item, long long len) {
    const int units = item_units(p, s);
    const long long start = before + static_cast<long long>(item) * units;
    const long long first = start + p.setup, last = start + units - 1;
    // (a division of 64 bits takes ten times as long, and batches of that size are rare)
    if (((last | len) >> 32) == 0)
        return {static_cast<int>(static_cast<uint32_t>(first) / static_cast<uint32_t>(len)),
                static_cast<int>(static_cast<uint32_t>(last) / static_cast<uint32_t>(len))};
    return {static_cast<int>(first / len), static_cast<int>(last / len)};
}

// A row's state: its maximum, its sum, and columns 4 j .. 4 j + 3 at o + j step.
struct StateAt {
    const float *m, *l, *o;
    int step;
};
// The one that run c left of row `in` of a cut item, c0 the item's first run.
template <int D>
__device__ __forceinline__ StateAt run_state(const TreeParams& p, int c, int c0, int in) {
    const PartialAt x = partial_at<D>(p, 2 * c + (c == c0 ? 1 : 0));
    return {x.m + in, x.l + in, x.at(in, 0), 4 << p.row_shift};
}

// A row's running state: the largest maximum so far, the sum and TURNS groups of 4
// columns.
template <int TURNS>
struct Acc {
    float M = -INFINITY, den = 0.f;
    float4 num[TURNS];
    __device__ __forceinline__ Acc() {
#pragma unroll
        for (int u = 0; u < TURNS; ++u) num[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // K states at once: their maxima m, sums l and columns o, as many as `real`
    template <int K>
    __device__ __forceinline__ void add(const float* m, const float* l, const float4 (*o)[TURNS],
                                        int real) {
        float top = M;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k < real) top = fmaxf(top, m[k]);
        const float sub = finite_max(top), old = fast_exp2(M - sub);
        M = top;
        den *= old;
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
            num[u].x *= old, num[u].y *= old;
            num[u].z *= old, num[u].w *= old;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k >= real) break;
            const float f = fast_exp2(m[k] - sub);
            den = fmaf(f, l[k], den);
#pragma unroll
            for (int u = 0; u < TURNS; ++u) {
                num[u].x = fmaf(f, o[k][u].x, num[u].x), num[u].y = fmaf(f, o[k][u].y, num[u].y);
                num[u].z = fmaf(f, o[k][u].z, num[u].z), num[u].w = fmaf(f, o[k][u].w, num[u].w);
            }
        }
    }
    // n states, in order: at(k) says where state k lies; column groups j0, j0 + jump, ...
    template <class F>
    __device__ __forceinline__ void add_all(int n, int j0, int jump, F&& at) {
        for (int k0 = 0; k0 < n; k0 += kMergeAhead) {
            float m[kMergeAhead], l[kMergeAhead];
            float4 o[kMergeAhead][TURNS];
#pragma unroll
            for (int k = 0; k < kMergeAhead; ++k) {
                if (k0 + k >= n) continue;
                const StateAt x = at(k0 + k);
                m[k] = *x.m;
                l[k] = *x.l;
#pragma unroll
                for (int u = 0; u < TURNS; ++u)
                    o[k][u] = *reinterpret_cast<const float4*>(x.o + (j0 + u * jump) * x.step);
            }
            add<kMergeAhead>(m, l, o, n - k0);
        }
    }
    // 1 / the sum, with the scale of V: 0 for a row that sees nothing
    __device__ __forceinline__ float inverse(float vscale) const {
        return den > 0.f ? vscale / den : (den == 0.f ? 0.f : den);
    }
};

}  // namespace qmm
