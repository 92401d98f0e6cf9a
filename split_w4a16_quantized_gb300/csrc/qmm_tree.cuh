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

// Prefixes that runs of sequences share (qmm_prefix_attention): each is an entry of
// its own in the list of work, in front of the sequences, whose query rows are those
// of all its sequences.
struct SharedPrefixes {
    const int *table, *lens, *first;
    int G, max_pages, cap;
    float* direct;   // states of items that one run holds (DirectAt)
};

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
    float* lse;      // (nullable) [B][T][Hq] log2 of a row's sum of 2^score, as stat_of
    float lift;      // log2 of the factor on the weights that the sums hold
    float* scores;   // [B][Hkv][T QG][score_stride]: each row's scores, for up to 8 rows
    int64_t score_stride;
    long long* plan;     // units before each entry, and of all: for the merge
    long long* chunks;   // the same of chunks of kChunk positions of a KV head
    SharedPrefixes pre;
};

// Token of row r of a sequence's heads: r / QG, exact for r < 2^14 and QG <= 64
// (r (QG - 1) < 2^22).  A shared prefix may have more rows.
template <bool kShared = false>
__device__ __forceinline__ int row_node(const TreeParams& p, int r) {
    if (kShared) return r / p.QG;
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
    if (p.pre.G > 0) {
        if (at < static_cast<int64_t>(p.pre.G) * p.pre.max_pages) prefetch_l2(p.pre.table + at);
        if (at < p.pre.G) {
            prefetch_l2(p.pre.lens + at);
            prefetch_l2(p.pre.first + at);
        }
    }
}

// ---- work split ----------------------------------------------------------------

struct Seq {
    int first, n;      // its rows of q
    int len, total;    // cached tokens; with the new ones
    int tiles;
    int row_tiles;
};

// Entries of the list: the sequences, behind the shared prefixes where there are any.
template <bool kShared>
__device__ __forceinline__ int entries(const TreeParams& p) {
    return kShared ? p.pre.G + p.d.B : p.d.B;
}

// Sequences [b0, b1) of prefix g (the caller's device data, so clamped).
template <bool kFromL2>
__device__ __forceinline__ void group_range(const TreeParams& p, int g, int* b0, int* b1) {
    const int a = plan_value<kFromL2>(p.pre.first + g), e = plan_value<kFromL2>(p.pre.first + g + 1);
    *b0 = a < 0 ? 0 : (a > p.d.B ? p.d.B : a);
    *b1 = e < *b0 ? *b0 : (e > p.d.B ? p.d.B : e);
}

// Prefix g as an entry: its rows are the tokens of its sequences, all of which see all
// of it.
template <bool kFromL2>
__device__ __forceinline__ Seq shared_prefix(const TreeParams& p, int g) {
    Seq s;
    int b0, b1;
    group_range<kFromL2>(p, g, &b0, &b1);
    if (p.cu) {
        const int a = plan_value<kFromL2>(p.cu + b0), e = plan_value<kFromL2>(p.cu + b1);
        s.first = a < 0 ? 0 : (a > p.N ? p.N : a);
        s.n = (e < s.first ? s.first : (e > p.N ? p.N : e)) - s.first;
    } else {
        s.first = b0 * p.T;
        s.n = (b1 - b0) * p.T;
    }
    const int len = plan_value<kFromL2>(p.pre.lens + g);
    s.len = b0 == b1 || len < 0 ? 0 : (len > p.pre.cap ? p.pre.cap : len);
    s.total = s.len;
    s.tiles = (s.total + (1 << p.tile_shift) - 1) >> p.tile_shift;
    s.row_tiles = s.total > 0 ? (s.n * p.QG + (1 << p.row_shift) - 1) >> p.row_shift : 0;
    return s;
}

template <bool kFromL2 = false, bool kShared = false>
__device__ __forceinline__ Seq sequence(const TreeParams& p, int b) {
    if (kShared) {
        if (b < p.pre.G) return shared_prefix<kFromL2>(p, b);
        b -= p.pre.G;
    }
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
    const long long sum = all + p.ctas - 1;
    const long long r = (sum >> 32) == 0 ? static_cast<uint32_t>(sum) / static_cast<uint32_t>(p.ctas)
                                         : sum / p.ctas;
    return r < p.min_run ? p.min_run : r;
}

// A CTA's place in the list of units.
struct Run {
    Seq s;            // sequence b
    int b;
    int at;           // unit within the sequence's list
    int left;         // units of the run still to do
};

// Positions that the pass over the scores takes at a time, and a sequence's pieces of them.
constexpr int kChunk = 1024;
__device__ __forceinline__ long long chunks_of(const TreeParams& p, const Seq& s) {
    return static_cast<long long>((s.total + kChunk - 1) / kChunk) * p.d.Hkv;
}

// The CTA's run: whole block of kN threads; sh: shared scratch.  kPlan: the first block
// writes down what lies before each entry, for the launch that merges (p.plan and, where
// it is not NULL, p.chunks).
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

template <int kN, bool kShared = false, bool kPlan = kShared>
__device__ __forceinline__ Run find_run(const TreeParams& p, RunShared& sh) {
    Run r;
    const int count = entries<kShared>(p);
    if (count <= 32) {
        const int lane = threadIdx.x & 31;
        Seq s = {};
        if (lane < count) s = sequence<false, kShared>(p, lane);
        const int mine = lane < count ? units_of(p, s) : 0;
        long long all;
        const long long before = warp_scan(mine, &all);
        if (kPlan && blockIdx.x == 0 && threadIdx.x < 32) {
            if (lane < count) p.plan[lane] = before;
            if (lane == 0) p.plan[count] = all;
            if (p.chunks) {
                long long total;
                const long long c = warp_scan(lane < count ? chunks_of(p, s) : 0, &total);
                if (lane < count) p.chunks[lane] = c;
                if (lane == 0) p.chunks[count] = total;
            }
        }
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
    const int per = (count + kN - 1) / kN;
    const int b0 = min(count, static_cast<int>(threadIdx.x) * per), b1 = min(count, b0 + per);
    long long mine = 0, all;
    Seq s;
    for (int b = b0; b < b1; ++b) {
        s = sequence<false, kShared>(p, b);
        mine += units_of(p, s);
    }
    if (threadIdx.x == 0) sh.b = -1;
    const long long before = block_scan<kN>(mine, sh.red, &all);
    const long long len = run_length(p, all);
    const long long start = len * blockIdx.x;
    if (kPlan && blockIdx.x == 0) {   // (the whole block)
        long long at = before, chunks = 0, all_chunks;
        for (int b = b0; b < b1; ++b) {
            p.plan[b] = at;
            if (per > 1) s = sequence<false, kShared>(p, b);
            at += units_of(p, s);
            chunks += chunks_of(p, s);
        }
        if (threadIdx.x == 0) p.plan[count] = all;
        if (p.chunks) {
            __syncthreads();   // sh.red has been read
            at = block_scan<kN>(chunks, sh.red, &all_chunks);
            for (int b = b0; b < b1; ++b) {
                p.chunks[b] = at;
                if (per > 1) s = sequence<false, kShared>(p, b);
                at += chunks_of(p, s);
            }
            if (threadIdx.x == 0) p.chunks[count] = all_chunks;
        }
    }
    if (start >= before && start < before + mine) {
        // this thread's sequences hold the start
        long long at = start - before;
        for (int b = b0; b < b1; ++b) {
            if (per > 1) s = sequence<false, kShared>(p, b);
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
template <bool kShared = false>
__device__ __forceinline__ bool next_stretch(const TreeParams& p, Run& r, Stretch* x) {
    while (r.left > 0) {
        while (r.at >= units_of(p, r.s)) {
            r.at -= units_of(p, r.s);
            if (++r.b >= entries<kShared>(p)) return false;   // (not reached: the run ends with the list)
            r.s = sequence<false, kShared>(p, r.b);
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

// Where the state of an item that one run holds lies, with shared prefixes: row
// (token, head) of the sequences' own part (0) or of the prefixes' (1).
struct DirectAt {
    float *m, *l, *o;   // o: the row's D values
};
template <int D>
__device__ __forceinline__ DirectAt direct_at(const TreeParams& p, int part, int64_t row) {
    const int64_t rows = static_cast<int64_t>(p.N) * p.Hq, r = part * rows + row;
    return {p.pre.direct + r, p.pre.direct + 2 * rows + r, p.pre.direct + 4 * rows + r * D};
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

// The same, whose lines are the first that L2 gives up.
__device__ __forceinline__ void tma_load_4d_once(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                                 int c0, int c1, int c2, int c3) {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(smem_addr(bar)), "l"(policy)
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
template <int kTile, bool kFromL2 = false>
struct PageWalk {
    const int* row;
    int c_end, c0, cur, nxt;
    __device__ __forceinline__ int entry(const TreeParams& p, int c) const {
        return c < c_end ? plan_value<kFromL2>(row + ((c << p.box_shift) >> p.d.page_shift)) : -1;
    }
    template <bool kShared = false>
    __device__ __forceinline__ void start(const TreeParams& p, const Stretch& x, int lane) {
        c_end = (x.s.total + (1 << p.box_shift) - 1) >> p.box_shift;   // pieces that hold positions
        if (kShared && x.b < p.pre.G)
            row = p.pre.table + static_cast<int64_t>(x.b) * p.pre.max_pages;
        else
            row = p.d.table + static_cast<int64_t>(x.b - (kShared ? p.pre.G : 0)) * p.d.max_pages;
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
// kOnce: the tile is not read again.
template <int kTile, int kBoxes, int kBox, int kElems, bool kOnce = false>
__device__ __forceinline__ void copy_tile(const TreeParams& p, const CUtensorMap* map, uint64_t* bar,
                                          uint32_t dst, const int* pages, int t, int g) {
    const int pieces = kTile >> p.box_shift;
    const int slot_mask = (1 << p.d.page_shift) - 1;
#pragma unroll 1
    for (int k = 0; k < pieces; ++k) {
        const int row = k << p.box_shift;
#pragma unroll
        for (int x = 0; x < kBoxes; ++x) {
            const uint32_t to = dst + x * (kTile * kBox) + row * kBox;
            const int slot = (t * kTile + row) & slot_mask;
            if (kOnce) tma_load_4d_once(to, map, bar, x * kElems, slot, g, pages[k]);
            else tma_load_4d(to, map, bar, x * kElems, slot, g, pages[k]);
        }
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

// log2 of the sum of 2^score of a row with maximum (or reference) m and sum l of
// weights lifted by 2^lift; infinity for a row that sees nothing, whose weights are 0.
__device__ __forceinline__ float stat_of(const TreeParams& p, float m, float l) {
    return l == 0.f ? INFINITY : m + (log2f(l) - p.lift);
}
// Where it goes: row `node`, `head` of sequence b.
__device__ __forceinline__ float* stat_at(const TreeParams& p, int b, int node, int head) {
    return p.lse + (static_cast<int64_t>(b) * p.T + node) * p.Hq + head;
}

// 2^x, one instruction (ex2.approx: 2 ulp, results below 2^-126 are 0).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// scale log2(e) k_scale, for exp2 of the scaled score.  Neither 0 nor infinity, whatever
// scale and k_scale: times a masked score (-inf) or a score of 0 those would be NaN.
float score_factor(const qmm_kv_cache& c, float scale);

// A launch's parameters and the maps of its K and V (qmm_tree_attention.cu); returns a
// cudaError_t.
int tree_setup(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N, int T, int Hq,
               const int* cu, const int* parents, float scale, float* ws, int ctas, int row_shift,
               int tile_shift, int min_run, int setup, TreeParams* out, CUtensorMap* kmap,
               CUtensorMap* vmap);

// One launch of the tcgen05 kernel (qmm_tree_attention_tc.cu); the merge
// kernel is the caller's.  Items of up to 128 rows (row_shift 7, two CTAs per
// SM) or 256 (8, one); device: the current one.
constexpr int kTcTileShift = 6;
constexpr float kTcLift = 7.f;   // log2 of its factor on F16 weights
int launch_tree_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                   bool fp8, int device, cudaStream_t st);
// One launch of the kernel for up to 8 rows (qmm_tree_attention.cu) with shared prefixes
// (p.pre), or that also leaves each row's scores in p.scores; the merge is the caller's.
constexpr int kFewRowShift = 3, kFewTileShift = 6, kFewCtasPerSm = 2, kFewMinRun = 2, kFewSetup = 1;
constexpr float kFewLift = 15.f;   // log2 of its factor on F16 weights
int launch_tree_few_shared(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p,
                           int D, bool fp8, int device, cudaStream_t st);
int launch_tree_scores(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                       bool fp8, int device, cudaStream_t st);
// The tcgen05 kernel with shared prefixes (p.pre), items of up to 128 rows: every item leaves a
// state, and the merge is the caller's (qmm_prefix_attention.cu).
int launch_prefix_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                     bool fp8, int device, cudaStream_t st);

}  // namespace qmm
