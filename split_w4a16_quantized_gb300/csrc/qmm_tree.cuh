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
#include "qmm_paged_host.h"
#include "qmm_sm100.cuh"

namespace qmm {

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
    uint32_t qg_inv;   // ceil(2^22 / QG)
    int row_shift;   // log2 of the query rows of a work item
    int tile_shift;  // log2 of the positions of a tile
    int min_run;     // units of the shortest run
    int setup;       // units an item counts for beside its tiles
    int box_shift;   // log2 of the positions of one copy: min(page, tile)
    float qscale;    // scale * log2(e) * k_scale
    float vscale;
};

// Token of row r of a sequence's heads: r / QG, exact for r < 2^14 and QG <= 64
// (r (QG - 1) < 2^22).
__device__ __forceinline__ int row_node(const TreeParams& p, int r) {
    return static_cast<int>((static_cast<uint64_t>(r) * p.qg_inv) >> 22);
}

// Ask for the lengths and the page table while the kernels before this one may
// still run: a CTA reads them one after the other before its first copy, a trip
// to HBM each.  (Only L2 is touched: what those kernels write is seen.)
__device__ __forceinline__ void prefetch_plan(const TreeParams& p, int tid, int threads) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * threads + tid) * 32;
    const int64_t table = static_cast<int64_t>(p.d.B) * p.d.max_pages;
    if (at < table) prefetch_l2(p.d.table + at);
    if (at < p.d.B) {
        prefetch_l2(p.d.lens + at);
        if (p.cu) prefetch_l2(p.cu + at);
    }
    if (p.parents && at < p.N) prefetch_l2(p.parents + at);
}

// ---- work split ----------------------------------------------------------------

struct Seq {
    int first, n;      // its rows of q
    int len, total;    // cached tokens; with the new ones
    int tiles;
    int row_tiles;
};

template <bool kFromL2 = false>
__device__ __forceinline__ Seq sequence(const TreeParams& p, int b) {
    Seq s;
    token_range<kFromL2>(p.cu, p.N, p.T, b, &s.first, &s.n);
    s.len = cached_tokens<kFromL2>(p.d, b);
    s.total = s.len + s.n < p.d.cap ? s.len + s.n : p.d.cap;
    s.tiles = (s.total + (1 << p.tile_shift) - 1) >> p.tile_shift;
    s.row_tiles = (s.n * p.QG + (1 << p.row_shift) - 1) >> p.row_shift;
    return s;
}
// Units of work of one item, and of all the sequence's items (the host keeps a
// sequence's below 2^31).
__device__ __forceinline__ int item_units(const TreeParams& p, const Seq& s) {
    return s.tiles + p.setup;
}
__device__ __forceinline__ int units_of(const TreeParams& p, const Seq& s) {
    return s.row_tiles * p.d.Hkv * item_units(p, s);
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

// A CTA's place in the list of units.
struct Run {
    Seq s;            // sequence b
    int b;
    int at;           // unit within the sequence's list
    int left;         // units of the run still to do
};

// The CTA's run: whole block of kN threads; sh: shared scratch.
struct RunShared {   // (s and at hold nothing where b < 0)
    long long red[32];
    Seq s;
    int at, b;
};
// Units of the whole batch and of the sequences before b; of up to 32
// sequences: a lane's sequence each, every warp for itself, no barrier.
__device__ __forceinline__ long long warp_scan(long long v, long long* total) {
    const int lane = threadIdx.x & 31;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    *total = __shfl_sync(0xffffffffu, x, 31);
    return x - v;
}

template <int kN>
__device__ __forceinline__ Run find_run(const TreeParams& p, RunShared& sh) {
    Run r;
    if (p.d.B <= 32) {
        const int lane = threadIdx.x & 31;
        Seq s = {};
        if (lane < p.d.B) s = sequence(p, lane);
        const int mine = lane < p.d.B ? units_of(p, s) : 0;
        long long all;
        const long long before = warp_scan(mine, &all);
        const long long len = run_length(p, all), start = len * blockIdx.x;
        const uint32_t owner = __ballot_sync(0xffffffffu, start >= before && start < before + mine);
        r.b = owner ? __ffs(owner) - 1 : -1;
        const int from = owner ? r.b : 0;
        r.at = __shfl_sync(0xffffffffu, static_cast<int>(start - before), from);
        r.s.first = __shfl_sync(0xffffffffu, s.first, from);
        r.s.n = __shfl_sync(0xffffffffu, s.n, from);
        r.s.len = __shfl_sync(0xffffffffu, s.len, from);
        r.s.total = __shfl_sync(0xffffffffu, s.total, from);
        r.s.tiles = __shfl_sync(0xffffffffu, s.tiles, from);
        r.s.row_tiles = __shfl_sync(0xffffffffu, s.row_tiles, from);
        r.left = r.b < 0 ? 0 : static_cast<int>(all - start < len ? all - start : len);
        return r;
    }
    const int per = (p.d.B + kN - 1) / kN;
    const int b0 = min(p.d.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.d.B, b0 + per);
    long long mine = 0, all;
    Seq s;
    for (int b = b0; b < b1; ++b) {
        s = sequence(p, b);
        mine += units_of(p, s);
    }
    if (threadIdx.x == 0) sh.b = -1;
    const long long before = block_scan<kN>(mine, sh.red, &all);
    const long long len = run_length(p, all);
    const long long start = len * blockIdx.x;
    if (start >= before && start < before + mine) {
        // this thread's sequences hold the start
        long long at = start - before;
        for (int b = b0; b < b1; ++b) {
            if (per > 1) s = sequence(p, b);
            const int u = units_of(p, s);
            if (at < u) {
                sh.b = b;
                sh.at = static_cast<int>(at);
                sh.s = s;
                break;
            }
            at -= u;
        }
    }
    __syncthreads();
    r.b = sh.b;
    r.at = sh.at;
    r.s = sh.s;
    r.left = r.b < 0 ? 0 : static_cast<int>(all - start < len ? all - start : len);
    return r;
}

// The next stretch of one work item in the run.
struct Stretch {
    Seq s;
    int b, g, row0;    // sequence, KV head, first row
    int t0, t1;        // tiles
};
__device__ __forceinline__ bool next_stretch(const TreeParams& p, Run& r, Stretch* x) {
    while (r.left > 0) {
        while (r.at >= units_of(p, r.s)) {
            r.at -= units_of(p, r.s);
            if (++r.b >= p.d.B) return false;   // (not reached: the run ends with the list)
            r.s = sequence(p, r.b);
        }
        x->s = r.s;
        const int units = item_units(p, x->s);
        const int item = r.at / units, u0 = r.at - item * units;
        x->b = r.b;
        x->g = item / x->s.row_tiles;
        x->row0 = (item - x->g * x->s.row_tiles) << p.row_shift;
        const int u1 = r.left < units - u0 ? u0 + r.left : units;
        r.at += u1 - u0;
        r.left -= u1 - u0;
        // the first `setup` units stand for the item's fixed cost: a run that
        // ends among them leaves the whole item to the next
        x->t0 = u0 > p.setup ? u0 - p.setup : 0;
        x->t1 = u1 - p.setup;
        if (x->t1 > x->t0) return true;
    }
    return false;
}

// Where partial state `slot` lies: run c's last stretch, when the item starts
// in it, is slot 2c + 1, its first slot 2c.
// o is [D / 4][rows][4]: the tcgen05 kernel's threads hold a row each, so
// neighbouring lanes store neighbouring 16 bytes (row after row, 512 bytes
// apart, its stores took 32 passes through the load/store unit each).
struct PartialAt {
    float *m, *l, *o;
    int row_shift;
    __device__ __forceinline__ float* at(int r, int c) const {
        return o + ((static_cast<size_t>(c >> 2) << row_shift) + r) * 4 + (c & 3);
    }
};
template <int D>
__device__ __forceinline__ PartialAt partial_at(const TreeParams& p, int slot) {
    const size_t all = static_cast<size_t>(2 * p.ctas) << p.row_shift;
    const size_t r = static_cast<size_t>(slot) << p.row_shift;
    PartialAt a;
    a.m = p.ws + r;
    a.l = p.ws + all + r;
    a.o = p.ws + 2 * all + r * D;
    a.row_shift = p.row_shift;
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

// One lane of a converged warp, the same one every time.  The compiler knows
// that a block under it has a single active thread, and feeds the copies' and
// MMAs' uniform operands straight from registers; under `lane == 0` it goes
// through the active lanes in a loop, which measured 160 clocks per MMA and 400
// per copy.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n"
                 : "=r"(one));
    return one != 0;
}

// The table entries of a stretch, looked up by a warp 32 pieces at a time and
// one batch ahead.
template <int kTile>
struct PageWalk {
    const int* row;
    int c_end, c0, cur, nxt;
    __device__ __forceinline__ int entry(const TreeParams& p, int c) const {
        return c < c_end ? row[(c << p.box_shift) >> p.d.page_shift] : -1;
    }
    __device__ __forceinline__ void start(const TreeParams& p, const Stretch& x, int lane) {
        c_end = (x.s.total + (1 << p.box_shift) - 1) >> p.box_shift;   // pieces that hold positions
        row = p.d.table + static_cast<int64_t>(x.b) * p.d.max_pages;
        c0 = x.t0 * (kTile >> p.box_shift);
        cur = entry(p, c0 + lane);
        nxt = entry(p, c0 + 32 + lane);
    }
    // Whole warp: the page numbers of a tile's pieces into `pages` (kTile / 8 of
    // shared memory), for the thread that issues the copies; returns one bit per
    // piece that exists.  A missing page (or a piece past the last position) is
    // num_pages: outside the map, where a copy fills zeros.
    __device__ __forceinline__ uint32_t tile(const TreeParams& p, int t, int lane, int* pages) {
        const int pieces = kTile >> p.box_shift;
        if (t * pieces >= c0 + 32) {
            c0 += 32;
            cur = nxt;
            nxt = entry(p, c0 + 32 + lane);
        }
        const int at = t * pieces - c0;
        const bool real = cur >= 0 && cur < p.d.num_pages;
        const uint32_t ok = __ballot_sync(0xffffffffu, real);
        if (lane >= at && lane < at + pieces) pages[lane - at] = real ? cur : p.d.num_pages;
        __syncwarp();
        return (ok >> at) & ((1u << pieces) - 1u);
    }
};

// The copies of one K or V tile, issued by one thread: page pieces by
// column blocks of `kBox` bytes (kElems values), kTile rows of a block together.
template <int kTile, int kBoxes, int kBox, int kElems>
__device__ __forceinline__ void copy_tile(const TreeParams& p, const CUtensorMap* map, uint64_t* bar,
                                          uint32_t dst, const int* pages, int t, int g) {
    const int pieces = kTile >> p.box_shift;
    const int slot_mask = (1 << p.d.page_shift) - 1;
#pragma unroll 1
    for (int k = 0; k < pieces; ++k) {
        const int row = k << p.box_shift;
#pragma unroll
        for (int x = 0; x < kBoxes; ++x)
            tma_load_4d(dst + x * (kTile * kBox) + row * kBox, map, bar, x * kElems,
                        (t * kTile + row) & slot_mask, g, pages[k]);
    }
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

// A positive factor on scores, kept from 0 and infinity (0 times a masked score
// is NaN, and so is infinity times a score of 0).
__device__ __forceinline__ float finite_factor(float x) {
    return fminf(fmaxf(x, __uint_as_float(1u)), __uint_as_float(0x7f7fffffu));
}

// 2^x, one instruction (ex2.approx: 2 ulp, results below 2^-126 are 0).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One launch of the tcgen05 kernel (qmm_tree_attention_tc.cu); the merge
// kernel is the caller's.  Items of up to 128 rows (row_shift 7, two CTAs per
// SM) or 256 (8, one); device: the current one.
constexpr int kTcTileShift = 6;
int launch_tree_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                   bool fp8, int device, cudaStream_t st);

}  // namespace qmm
