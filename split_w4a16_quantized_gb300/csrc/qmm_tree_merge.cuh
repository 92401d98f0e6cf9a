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
    return {static_cast<int>((start + p.setup) / len), static_cast<int>((start + units - 1) / len)};
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
    // The states of row `in` of a cut item, in run order; column groups j0, j0 + jump, ...
    template <int D>
    __device__ __forceinline__ void add_runs(const TreeParams& p, Runs c, int in, int j0, int jump) {
        for (int k0 = c.c0; k0 <= c.c1; k0 += kMergeAhead) {
            float m[kMergeAhead], l[kMergeAhead];
            float4 o[kMergeAhead][TURNS];
#pragma unroll
            for (int k = 0; k < kMergeAhead; ++k) {
                if (k0 + k > c.c1) continue;
                const PartialAt x = partial_at<D>(p, 2 * (k0 + k) + (k0 + k == c.c0 ? 1 : 0));
                m[k] = x.m[in];
                l[k] = x.l[in];
#pragma unroll
                for (int u = 0; u < TURNS; ++u)
                    o[k][u] = *reinterpret_cast<const float4*>(x.at(in, 4 * (j0 + u * jump)));
            }
            add<kMergeAhead>(m, l, o, c.c1 - k0 + 1);
        }
    }
    // 1 / the sum, with the scale of V: 0 for a row that sees nothing
    __device__ __forceinline__ float inverse(float vscale) const {
        return den > 0.f ? vscale / den : (den == 0.f ? 0.f : den);
    }
};

}  // namespace qmm
