// Tree attention's work split (qmm_tree_attention), shared by its kernels: the
// batch's work items, their tiles laid end to end, and the run of tiles that a
// CTA takes.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "qmm_paged.cuh"
#include "qmm_sm100.cuh"

namespace qmm {

constexpr int kTile = 64;              // positions per tile
constexpr int kWords = kMaxTree / 32;  // ancestor bits of a token

struct TreeParams {
    PagedDims d;
    const __nv_bfloat16* q;
    __nv_bfloat16* O;
    const int *cu, *parents;
    float* ws;    // partial states: m [2 ctas][rows], l the same, o [2 ctas][rows][D]
    int* status;
    int64_t q_stride;
    int N, T, Hq, QG, ctas;
    int row_shift;   // log2 of the query rows of a work item
    int min_run;     // tiles of the shortest run
    int box_shift;   // log2 of the positions of one copy: min(page, tile)
    float qscale;    // scale * log2(e) * k_scale
    float vscale;
};

// ---- work split ----------------------------------------------------------------

struct Seq {
    int first, n;      // its rows of q
    int len, total;    // cached tokens; with the new ones
    int tiles;         // of 64 positions
    int row_tiles;
};

__device__ __forceinline__ Seq sequence(const TreeParams& p, int b) {
    Seq s;
    token_range(p.cu, p.N, p.T, b, &s.first, &s.n);
    s.len = cached_tokens(p.d, b);
    s.total = s.len + s.n < p.d.cap ? s.len + s.n : p.d.cap;
    s.tiles = (s.total + kTile - 1) / kTile;
    s.row_tiles = (s.n * p.QG + (1 << p.row_shift) - 1) >> p.row_shift;
    return s;
}
__device__ __forceinline__ long long tiles_of(const TreeParams& p, const Seq& s) {
    return static_cast<long long>(s.tiles) * s.row_tiles * p.d.Hkv;
}

// Sum of v over the block and over the threads before this one.  Every thread
// of the block calls it; kN threads, red is kN / 32 values of shared memory.
template <int kN>
__device__ __forceinline__ long long block_scan(long long v, long long* red, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kN / 32; ++w) {
        if (w < warp) before += red[w];
        all += red[w];
    }
    *total = all;
    return before + x - v;
}

__device__ __forceinline__ long long run_length(const TreeParams& p, long long all) {
    const long long r = (all + p.ctas - 1) / p.ctas;
    return r < p.min_run ? p.min_run : r;
}

// A CTA's place in the list of tiles.
struct Run {
    int b;            // sequence
    long long at;     // tile within the sequence's list
    long long left;   // tiles of the run still to do
};

// The CTA's run: whole block of kN threads; sh: shared scratch.
struct RunShared {
    long long red[32];
    long long at;
    int b;
};
template <int kN>
__device__ __forceinline__ Run find_run(const TreeParams& p, RunShared& sh) {
    const int per = (p.d.B + kN - 1) / kN;
    const int b0 = min(p.d.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.d.B, b0 + per);
    long long mine = 0, all;
    for (int b = b0; b < b1; ++b) mine += tiles_of(p, sequence(p, b));
    if (threadIdx.x == 0) sh.b = -1;
    const long long before = block_scan<kN>(mine, sh.red, &all);
    const long long len = run_length(p, all);
    const long long start = len * blockIdx.x;
    if (start >= before && start < before + mine) {
        // this thread's sequences hold the start
        long long at = start - before;
        for (int b = b0; b < b1; ++b) {
            const long long t = tiles_of(p, sequence(p, b));
            if (at < t) {
                sh.b = b;
                sh.at = at;
                break;
            }
            at -= t;
        }
    }
    __syncthreads();
    Run r;
    r.b = sh.b;
    r.at = sh.at;
    r.left = r.b < 0 ? 0 : (all - start < len ? all - start : len);
    return r;
}

// The next stretch of one work item in the run.
struct Stretch {
    Seq s;
    int b, g, row0;    // sequence, KV head, first row
    int t0, t1;        // tiles
};
__device__ __forceinline__ bool next_stretch(const TreeParams& p, Run& r, Stretch* x) {
    if (r.left <= 0) return false;
    x->s = sequence(p, r.b);
    while (r.at >= tiles_of(p, x->s)) {
        r.at -= tiles_of(p, x->s);
        if (++r.b >= p.d.B) return false;   // (not reached: the run ends with the list)
        x->s = sequence(p, r.b);
    }
    const int item = static_cast<int>(r.at / x->s.tiles);
    x->b = r.b;
    x->g = item / x->s.row_tiles;
    x->row0 = (item % x->s.row_tiles) << p.row_shift;
    x->t0 = static_cast<int>(r.at % x->s.tiles);
    const long long end = x->t0 + r.left;
    x->t1 = end < x->s.tiles ? static_cast<int>(end) : x->s.tiles;
    r.at += x->t1 - x->t0;
    r.left -= x->t1 - x->t0;
    return true;
}

// Where partial state `slot` lies: run c's last stretch, when the item starts
// in it, is slot 2c + 1, its first slot 2c.
struct PartialAt {
    float *m, *l, *o;   // of the item's row 0; o rows are D values
};
template <int D>
__device__ __forceinline__ PartialAt partial_at(const TreeParams& p, int slot) {
    const size_t all = static_cast<size_t>(2 * p.ctas) << p.row_shift;
    const size_t r = static_cast<size_t>(slot) << p.row_shift;
    PartialAt a;
    a.m = p.ws + r;
    a.l = p.ws + all + r;
    a.o = p.ws + 2 * all + r * D;
    return a;
}

// 4-D tile load (c0 innermost), completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(smem_addr(bar))
        : "memory");
}

// Two E4M3 numbers (the low 16 bits) as an F16 pair; every E4M3 number is an F16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Maximum that every later exp2 can subtract: 0 while nothing is visible.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// 2^x, one instruction (ex2.approx: 2 ulp, results below 2^-126 are 0).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One launch of the tcgen05 kernel (qmm_tree_attention_tc.cu); the merge
// kernel is the caller's.
int launch_tree_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                   bool fp8, cudaStream_t st);

}  // namespace qmm
