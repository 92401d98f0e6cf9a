// Eviction from the paged KV cache by the weight each slot has received
// (qmm_kv_evict).
//
// A cache column (layer, sequence, KV head) of len slots goes back to `keep`: the
// first `sinks` and the last `recent` slots stay, and of those between the keep -
// sinks - recent with the largest weights, the lowest slot first among equals.
//
// Where rows go.  Attention does not look at the order of the slots, so only what
// lies behind the budget has to move: a chosen row below `line` = keep - recent stays,
// the evicted slots below it take the chosen rows from the line on, both in ascending
// order, and the recent rows follow in order at [line, keep).  So the last `recent`
// slots are the newest tokens at the next eviction too.  Moved are `recent` rows and
// the chosen ones between line and len - recent, instead of all rows behind the first
// evicted slot.
//
// Two kernels.  evict_select, a block a column, or up to 8 in a cluster where a column is
// long or columns are few: the weights come to shared memory once; the threshold is found
// by its bits, 8 a pass (a weight's bits, ordered as the weights are); then every warp takes
// a stretch of the slots, and the ranks of evicted slots below the line and of chosen ones
// behind it pair them.  Columns that eight blocks do not hold go through two queues
// filled in ascending order instead.
// evict_move, a block a column of K or V (and, where columns are few, a piece of its
// rows' bytes, and several blocks in a cluster): moves the rows in ascending order of their
// targets, a batch at a time: all of a batch is in registers before any of it is stored.
// A row moves to a lower slot, so a target is never the source of a later batch, and the
// batches before have read theirs.
//
// 16 sequences of 2500 to 7000 slots to 2048, 12 layers, D = 128, BF16: 372 us, floor 321:
// the moves 326 us, 2.15 GB at 6.6 TB/s, in pieces of 64 bytes 400; the choice 55, bound
// by its instructions (53 % of the issue slots), streamed from memory 113.  One sequence,
// 1151 slots to 1024, 36 layers: 34 us, floor 16: 10 and 20 us, each a few trips to memory
// in a row.  One of 100,000 to 16,384, one layer: 79 us; a block a column, through memory,
// 484.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_evict_split.h"
#include "qmm_internal.h"
#include "qmm_paged.cuh"
#include "qmm_paged_host.h"
#include "qmm_per_device.h"
#include "qmm_sm100.cuh"

namespace qmm {
namespace {

// Neither kernel lets the next start early: blocks that wait take the room of those that
// work (16 sequences of 12 layers 377 us, the choice's blocks letting the moves start 457;
// one of 36 layers 34 and 38).
constexpr int kSelectThreads = 256;
constexpr int kMoveThreads = kEvictMoveThreads;
constexpr int kMoveRows = 8;      // rows a lane group has in flight

struct EvictParams {
    PagedDims d;
    const float* mass;
    float* mass_out;
    int64_t layer_stride, row_stride;   // of the weights
    int *kept, *new_lens;
    int keep, sinks, recent;
    int first;                  // this launch's first layer
    int elem, slices, lanes;    // bytes a value; pieces of a row, 16 * lanes bytes each
    int held;                   // slots that a block's shared memory holds
    int cluster, spread;        // blocks of a column; whether it takes them all
    int movers;                 // blocks of a column's piece
    uint8_t* pools[2 * kMaxEvictCaches];   // K and V of each layer
};

// Weights in order: larger weight, larger number; both zeros alike, and NaN below all.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);   // (-0 + 0 = +0)
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one, and over the block.
__device__ __forceinline__ int scan_block(int v, int* red, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w < warp) before += red[w];
        all += red[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// The digit (of 256) that the `want`-th largest falls into, given that `above` are larger:
// every warp reads the counts for itself.  *above and *count: larger ones, and those in
// the digit.
__device__ __forceinline__ int find_digit(const int* hist, int want, int* above, int* count) {
    const int lane = threadIdx.x & 31;
    // lane l: digits 255 - 8 l down to 248 - 8 l
    const int4 lo = *reinterpret_cast<const int4*>(hist + 248 - 8 * lane);
    const int4 hi = *reinterpret_cast<const int4*>(hist + 252 - 8 * lane);
    const int c[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += c[i];
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    before += *above - sum;   // larger than this lane's digits
    int digit = -1, at = before, n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (digit < 0 && at < want && at + c[i] >= want) digit = 255 - 8 * lane - i, n = c[i];
        if (digit < 0) at += c[i];
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, digit >= 0)) - 1;
    *above = __shfl_sync(0xffffffffu, at, from);
    *count = __shfl_sync(0xffffffffu, n, from);
    return __shfl_sync(0xffffffffu, digit, from);
}

struct SelectShared {
    alignas(16) int hist[4][256];
    alignas(16) int total[256];         // of a cluster's blocks
    int red[2][kSelectThreads / 32];
    int count[3];                       // of this block: ties, evicted below the line, chosen behind
    int digit, above;
    int queue[2][2 * kSelectThreads];   // evicted slots below the line, chosen ones behind
};

__device__ __forceinline__ uint32_t cluster_ld_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_ld_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared::cluster.u16 %0, [%1];\n" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// A column in the shared memory of C blocks of a cluster, `seg` slots each (a multiple of
// 32, at most p.held; one block: all of them).  row: this block's weights; holes: room for
// its evicted slots below the line, from its first slot on; bits: one a slot.
// kMany: C may be over 1.
template <bool kMany>
__device__ __forceinline__ void select_held(const EvictParams& p, SelectShared& sh, float* row,
                                            uint16_t* holes, uint32_t* bits, int len, int blocks,
                                            int me, int seg, const float* mass, float* mass_out,
                                            int* kept) {
    const int C = kMany ? blocks : 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int keep = p.keep, line = keep - p.recent, want = line - p.sinks;
    const int a0 = min(len, me * seg), a1 = min(len, a0 + seg);   // this block's slots
    const int m0 = max(p.sinks, a0), m1 = min(len - p.recent, a1);   // of them, those in question
    row -= a0;   // (by slot)
    bits -= a0 >> 5;
    // every block of the column; the order of what they wrote to shared memory
    auto meet = [&] {
        if (C > 1) cluster_barrier();
        else __syncthreads();
    };
    for (int i = tid; i < 4 * 256; i += kSelectThreads) sh.hist[0][i] = 0;
    // (rows are 16-byte aligned and a multiple of 4 slots long)
#pragma unroll 4
    for (int i = a0 + 4 * tid; i < a1; i += 4 * kSelectThreads)
        *reinterpret_cast<float4*>(row + i) = *reinterpret_cast<const float4*>(mass + i);
    __syncthreads();
    uint32_t top = 0;
    int above = 0, ties = 0;
    if (want > 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int shift = 24 - 8 * k;
            int* const hist = sh.hist[k];
            // Behind the first pass most slots are out of the running, and their bits as
            // they are say so, where neither zeros nor NaN are near.
            const uint32_t first = top >> 24;
            if (k > 0 && first != 0 && first != 0x7f && first != 0x80 && first != 0xff) {
                const uint32_t prefix = (top >> 31 ? top ^ 0x80000000u : ~top) >> ((shift + 8) & 31);
                const uint32_t flip = top >> 31 ? 0u : 255u;
                auto count = [&](float w) {
                    const uint32_t u = __float_as_uint(w);
                    if ((u >> ((shift + 8) & 31)) == prefix)
                        atomicAdd(&hist[((u >> shift) & 255u) ^ flip], 1);
                };
                const int q0 = (m0 + 3) & ~3, q1 = m1 & ~3;   // whole quarters of 16 bytes
                for (int i = q0 + 4 * tid; i < q1; i += 4 * kSelectThreads) {
                    const float4 w = *reinterpret_cast<const float4*>(row + i);
                    count(w.x), count(w.y), count(w.z), count(w.w);
                }
                // (and those that m0 and m1 cut)
                const int i = tid < 4 ? m0 + tid : max(q0, q1) + tid - 4;
                if (tid < 8 && i < m1 && (tid < 4 ? i < q0 : i >= q0)) count(row[i]);
            } else {
                for (int i = m0 + tid; i < m1; i += kSelectThreads) {
                    const uint32_t r = rank_of(row[i]);
                    if (k == 0 || (r >> ((shift + 8) & 31)) == (top >> ((shift + 8) & 31)))
                        atomicAdd(&hist[(r >> shift) & 255u], 1);
                }
            }
            meet();
            if (C > 1) {
                int sum = 0;
                for (int r = 0; r < C; ++r) sum += cluster_ld_u32(cluster_map(smem_addr(&hist[tid]), r));
                sh.total[tid] = sum;   // (the blocks met since it was last read)
                __syncthreads();
            }
            top |= static_cast<uint32_t>(find_digit(C > 1 ? sh.total : hist, want, &above, &ties)) << shift;
        }
    }
    // of the slots equal to the threshold, the first `equal` stay
    const int equal = want - above;
    // a warp's stretch of the block's slots, 32 at a time
    const int per = ((a1 - a0 + kSelectThreads - 1) / kSelectThreads) * 32;
    const int s0 = a0 + warp * per, s1 = min(a1, s0 + per);
    // of a count by lanes: those of the warps before this one; the block's to sh.count[at]
    auto before_warp = [&](int mine, int* red, int at) {
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) red[warp] = mine;
        __syncthreads();
        const int n = lane < kSelectThreads / 32 ? red[lane] : 0;
        if (warp == 0) {
            const int all = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) sh.count[at] = all;
        }
        return __reduce_add_sync(0xffffffffu, lane < warp ? n : 0);
    };
    // the same of the blocks before block r
    auto before_block = [&](int at, int r) {
        const int n = lane < r ? static_cast<int>(cluster_ld_u32(cluster_map(smem_addr(&sh.count[at]), lane))) : 0;
        return __reduce_add_sync(0xffffffffu, n);
    };
    // a weight above the threshold, or equal to it (a threshold below everything: NaN)
    const float least = __uint_as_float(top >> 31 ? top ^ 0x80000000u : ~top);
    auto larger = [&](float w) { return top == 0 ? w == w : w > least; };
    auto equals = [&](float w) { return top == 0 ? w != w : w == least; };
    const bool all_ties = equal >= ties;
    const uint32_t below = (1u << lane) - 1u;
    const int e1 = min(s1, m1), l1 = min(s1, line);   // ends of the stretch's slots in question
    int tie_at = 0;
    if (want > 0 && !all_ties) {   // (the same for all blocks)
        int mine = 0;
        for (int i = s0 + lane; i < e1; i += 32) mine += i >= m0 && equals(row[i]);
        tie_at = before_warp(mine, sh.red[0], 0);
        meet();
        if (C > 1) tie_at += before_block(0, me);
    }
    int n_holes = 0, n_late = 0;   // of this lane
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = want > 0 && i >= m0 && i < e1;
        const float w = in ? row[i] : 0.f;
        bool yes = in && (larger(w) || (all_ties && equals(w)));
        if (!all_ties) {
            const bool tie = in && equals(w);
            const uint32_t same = __ballot_sync(0xffffffffu, tie);
            yes = yes || (tie && tie_at + __popc(same & below) < equal);
            tie_at += __popc(same);
        }
        const uint32_t all = __ballot_sync(0xffffffffu, yes);
        if (lane == 0) bits[i0 >> 5] = all;
        n_holes += i >= m0 && i < l1 && !yes;
        n_late += yes && i >= line;
    }
    int hole = before_warp(n_holes, sh.red[0], 1), late = before_warp(n_late, sh.red[1], 2);
    for (int i0 = s0; i0 < l1; i0 += 32) {
        const int i = i0 + lane;
        const bool evicted = i >= m0 && i < l1 && !((bits[i0 >> 5] >> lane) & 1u);
        const uint32_t out = __ballot_sync(0xffffffffu, evicted);
        if (evicted) {
            holes[hole + __popc(out & below)] = static_cast<uint16_t>(i - a0);
        } else if (i < l1) {
            kept[i] = i;
            if (mass_out != mass) mass_out[i] = row[i];
        }
        hole += __popc(out);
    }
    meet();
    int first_hole = 0;   // lane r: of the column's, block r's first
    if (C > 1) {
        late += before_block(2, me);
        int n = lane < C ? static_cast<int>(cluster_ld_u32(cluster_map(smem_addr(&sh.count[1]), lane))) : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        first_hole = x - n;
    }
    for (int i0 = max(s0, line & ~31); i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        uint32_t in = bits[i0 >> 5];
        if (i0 < line) in &= ~0u << (line - i0);   // (line - i0 < 32; the bits end at m1)
        const bool yes = (in >> lane) & 1u;
        const int at = late + __popc(in & below);
        int j = -1;
        if (C > 1) {
            int r = 0, from = 0;   // the block that holds evicted slot `at`
            for (int k = 1; k < C; ++k) {
                const int f = __shfl_sync(0xffffffffu, first_hole, k);
                if (f <= at) r = k, from = f;
            }
            if (yes) j = r * seg + cluster_ld_u16(cluster_map(smem_addr(holes + (at - from)), r));
        } else if (yes) {
            j = holes[at];
        }
        if (i >= len - p.recent && i < s1) j = i - (len - keep);
        if (j >= 0) {
            kept[j] = i;
            mass_out[j] = row[i];
        }
        late += __popc(in);
    }
    if (C > 1) cluster_barrier();   // nobody reads this block's shared memory any more
}

template <bool kMany>
__global__ void __launch_bounds__(kSelectThreads, 4)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ __align__(16) float select_row[];
    __shared__ SelectShared sh;
    const int tid = threadIdx.x;
    const int cluster = kMany ? p.cluster : 1;
    const int me = blockIdx.x % cluster, column = blockIdx.x / cluster;
    const int h = column % p.d.Hkv, layer = p.first + column / p.d.Hkv, b = blockIdx.y;
    pdl_wait();
    const int len = cached_tokens(p.d, b), keep = p.keep;
    const int64_t col = static_cast<int64_t>(b) * p.d.Hkv + h;
    const float* mass = p.mass + layer * p.layer_stride + col * p.row_stride;
    float* mass_out = p.mass_out + layer * p.layer_stride + col * p.row_stride;
    int* kept = p.kept + (static_cast<int64_t>(layer) * p.d.B * p.d.Hkv + col) * keep;
    if (layer == 0 && h == 0 && me == 0 && tid == 0) p.new_lens[b] = min(len, keep);
    // Blocks of the cluster that the column takes (the others leave): all where they run at
    // once, else as many as hold it.
    const int C = p.spread ? cluster : min(cluster, (len - 1) / p.held + 1);
    const int seg = ((len + C - 1) / C + 31) & ~31;
    const bool fits = len > keep && seg <= p.held;
    if (me >= (fits ? C : 1)) return;
    if (len <= keep) {
        for (int64_t j = tid; j < keep; j += kSelectThreads) {
            kept[j] = j < len ? static_cast<int>(j) : -1;
            if (j < len && mass_out != mass) mass_out[j] = mass[j];
        }
        return;
    }
    if (fits) {
        uint16_t* holes = reinterpret_cast<uint16_t*>(select_row + p.held);
        select_held<kMany>(p, sh, select_row, holes, reinterpret_cast<uint32_t*>(holes + (kMany ? p.held : p.held / 2)), len, C,
                    me, seg, mass, mass_out, kept);
        return;
    }
    const int m0 = p.sinks, m1 = len - p.recent;        // the slots in question
    const int want = keep - p.sinks - p.recent;         // how many of them stay
    const int line = keep - p.recent;
    int* const hist = sh.hist[0];
    int* const red = sh.red[0];
    int (*const queue)[2 * kSelectThreads] = sh.queue;

    // The want-th largest number: its digits from the top, 8 bits a pass.  `above`:
    // slots known to be larger.
    uint32_t top = 0;
    int above = 0;
    if (want > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int64_t i = m0 + tid; i < m1; i += kSelectThreads) {
                const uint32_t r = rank_of(mass[i]);
                if (shift == 24 || (r >> (shift + 8)) == (top >> (shift + 8)))
                    atomicAdd(&hist[(r >> shift) & 255u], 1);
            }
            __syncthreads();
            // thread t < 256: how many lie in digits above 255 - t
            const int mine = tid < 256 ? hist[255 - tid] : 0;
            int all;
            const int before = scan_block(mine, red, &all);
            if (tid < 256 && above + before < want && above + before + mine >= want) {
                sh.digit = 255 - tid;
                sh.above = above + before;
            }
            __syncthreads();
            top |= static_cast<uint32_t>(sh.digit) << shift;
            above = sh.above;
            __syncthreads();
        }
    }
    // of the slots equal to it, the first `equal` stay
    const int equal = want - above;

    // Queues of evicted slots below the line and of chosen ones from it on; what both
    // hold is paired.  (below the line: sinks are chosen; there are as many evicted
    // there as chosen behind it)
    auto chosen = [&](int64_t i, bool in, int* ties) {   // whole block, ascending i
        const uint32_t r = in ? rank_of(mass[i]) : 0u;
        const bool tie = in && want > 0 && r == top;
        int all;
        const int before = scan_block(tie ? 1 : 0, red, &all);
        const bool yes = in && want > 0 && (r > top || (tie && *ties + before < equal));
        *ties += all;
        return yes;
    };
    // ties below the line come first
    int low_ties = 0, high_ties = 0;
    {
        int mine = 0;
        for (int64_t i = m0 + tid; i < line; i += kSelectThreads)
            mine += want > 0 && rank_of(mass[i]) == top;
        scan_block(mine, red, &high_ties);
    }
    for (int64_t j = tid; j < m0; j += kSelectThreads) kept[j] = static_cast<int>(j);
    for (int64_t j = line + tid; j < keep; j += kSelectThreads)
        kept[j] = static_cast<int>(j + (len - keep));
    int64_t low = m0, high = line;   // next slots to look at
    int held[2] = {0, 0};            // slots in each queue
    while (true) {
        // refill each queue to at least a slot, or to its end
        while (held[0] == 0 && low < line) {
            const int64_t i = low + tid;
            const bool in = i < line, yes = chosen(i, in, &low_ties);
            if (yes) kept[i] = static_cast<int>(i);
            int all;
            const int at = scan_block(in && !yes ? 1 : 0, red, &all);
            if (in && !yes) queue[0][at] = static_cast<int>(i);
            held[0] = all;
            low += kSelectThreads;
        }
        while (held[0] > 0 && held[1] < kSelectThreads && high < m1) {
            const int64_t i = high + tid;
            const bool yes = chosen(i, i < m1, &high_ties);
            int all;
            const int at = scan_block(yes ? 1 : 0, red, &all);
            if (yes) queue[1][held[1] + at] = static_cast<int>(i);
            held[1] += all;
            high += kSelectThreads;
        }
        __syncthreads();
        const int both = min(held[0], held[1]);
        if (both == 0) break;   // (no evicted slot is left)
        if (tid < both) kept[queue[0][tid]] = queue[1][tid];
        // what is left of either moves to its front
        int keep0 = 0, keep1 = 0, keep2 = 0;
        if (both + tid < held[0]) keep0 = queue[0][both + tid];
        if (both + tid < held[1]) keep1 = queue[1][both + tid];
        if (both + tid + kSelectThreads < held[1]) keep2 = queue[1][both + tid + kSelectThreads];
        __syncthreads();
        if (both + tid < held[0]) queue[0][tid] = keep0;
        if (both + tid < held[1]) queue[1][tid] = keep1;
        if (both + tid + kSelectThreads < held[1]) queue[1][tid + kSelectThreads] = keep2;
        held[0] -= both;
        held[1] -= both;
        __syncthreads();
    }
    __syncthreads();
    // the weights go with their slots, ascending: mass_out may be mass
    for (int64_t j0 = 0; j0 < keep; j0 += kSelectThreads) {
        const int64_t j = j0 + tid;
        const float w = j < keep ? mass[kept[j]] : 0.f;
        __syncthreads();
        if (j < keep) mass_out[j] = w;
    }
}

// kMany: the p.movers blocks of a cluster take the parts of a batch in turn (each part in
// registers at once: pieces of 64 bytes).
template <bool kMany>
__global__ void __launch_bounds__(kMoveThreads, 4)
    evict_move_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int64_t src[kMoveThreads], dst[kMoveThreads];   // bytes from the column's start
    __shared__ int red[2][kMoveThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
    const int movers = kMany ? p.movers : 1;
    int at = blockIdx.x;
    const int me = at % movers;
    at /= movers;
    const int slice = at % p.slices;
    at /= p.slices;
    const int kv = at & 1;
    at >>= 1;
    const int h = at % p.d.Hkv, layer = at / p.d.Hkv;   // of this launch
    pdl_wait();
    const int len = cached_tokens(p.d, b), keep = p.keep;
    if (len <= keep) return;   // (the same for the whole cluster)
    const int* kept = p.kept +
        ((static_cast<int64_t>(p.first + layer) * p.d.B + b) * p.d.Hkv + h) * keep;
    uint8_t* pool = p.pools[2 * layer + kv] + h * p.d.head_stride * p.elem +
                    (slice * p.lanes + tid % p.lanes) * 16;
    const int groups = kMoveThreads / p.lanes, group = tid / p.lanes;
    int odd = 0;
    const int step = movers * kMoveThreads;
    int64_t j = p.sinks + static_cast<int64_t>(me) * kMoveThreads + tid;
    int from_slot = j < keep ? kept[j] : -1;
    for (int64_t j0 = p.sinks; j0 < keep; j0 += step, j += step, odd ^= 1) {
        // the rows that move, in order (a missing page on either side: not moved)
        int64_t from = -1, to = -1;
        if (j < keep && from_slot != j) {
            from = slot_offset(p.d, b, from_slot);
            to = slot_offset(p.d, b, static_cast<int>(j));
        }
        from_slot = j + step < keep ? kept[j + step] : -1;
        const bool moves = from >= 0 && to >= 0;
        const uint32_t all = __ballot_sync(0xffffffffu, moves);
        if (lane == 0) red[odd][warp] = __popc(all);
        __syncthreads();   // (the batches before have been stored: src and dst are free)
        int before = 0, count = 0;
#pragma unroll
        for (int w = 0; w < kMoveThreads / 32; ++w) {
            if (w < warp) before += red[odd][w];
            count += red[odd][w];
        }
        if (moves) {
            const int i = before + __popc(all & ((1u << lane) - 1u));
            src[i] = from * p.elem;
            dst[i] = to * p.elem;
        }
        __syncthreads();
        for (int r0 = group; kMany ? r0 == group : r0 - group < count; r0 += kMoveRows * groups) {
            uint4 x[kMoveRows];
#pragma unroll
            for (int u = 0; u < kMoveRows; ++u) {
                const int r = r0 + u * groups;
                if (r < count) x[u] = *reinterpret_cast<const uint4*>(pool + src[r]);
            }
            if (kMany) cluster_barrier();
            else __syncthreads();
#pragma unroll
            for (int u = 0; u < kMoveRows; ++u) {
                const int r = r0 + u * groups;
                if (r < count) *reinterpret_cast<uint4*>(pool + dst[r]) = x[u];
            }
        }
    }
}

}  // namespace

int launch_kv_evict(const qmm_kv_cache* caches, int n, int first, const float* mass,
                    float* mass_out, int64_t layer_stride, int64_t row_stride, int keep, int sinks,
                    int recent, int* kept, int* new_lens, int num_sms, void* stream) {
    const qmm_kv_cache& c = caches[0];
    EvictParams p = {};
    p.d = paged_dims(c);
    p.mass = mass;
    p.mass_out = mass_out;
    p.layer_stride = layer_stride;
    p.row_stride = row_stride;
    p.kept = kept;
    p.new_lens = new_lens;
    p.keep = keep;
    p.sinks = sinks;
    p.recent = recent;
    p.first = first;
    p.elem = c.dtype == QMM_CACHE_E4M3 ? 1 : 2;
    const EvictSplit split =
        evict_split(static_cast<int64_t>(n) * c.Hkv * c.B, p.d.cap, keep, c.D * p.elem / 16, num_sms);
    p.slices = split.slices;
    p.lanes = split.lanes;
    p.movers = split.movers;
    p.cluster = split.cluster;
    p.spread = split.spread;
    p.held = split.held;
    const size_t smem = static_cast<size_t>(p.held) * (p.cluster > 1 ? 6 : 5) + p.held / 8;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return cudaErrorInvalidDevice;
    static PerDevice<bool> opted_in;
    if (!opted_in.get(device, [&] {
            auto opt_in = [](auto kernel) {
                return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kEvictSlots * 6 + kEvictSlots / 8) == cudaSuccess;
            };
            return opt_in(evict_select_kernel<false>) && opt_in(evict_select_kernel<true>);
        }))
        return cudaErrorInvalidValue;
    for (int i = 0; i < n; ++i) {
        p.pools[2 * i] = static_cast<uint8_t*>(caches[i].K);
        p.pools[2 * i + 1] = static_cast<uint8_t*>(caches[i].V);
    }
    // a launch in clusters of `blocks`
    auto run = [&](auto kernel, int64_t grid, int threads, size_t dynamic, int blocks) {
        cudaLaunchConfig_t cfg = {};
        LaunchAttrs la;
        apply_pdl(cfg, la);
        cudaLaunchAttribute attrs[2];
        if (blocks > 1) {
            attrs[0].id = cudaLaunchAttributeClusterDimension;
            attrs[0].val.clusterDim.x = static_cast<unsigned>(blocks);
            attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
            if (cfg.numAttrs > 0) attrs[1] = la.attr[0];
            ++cfg.numAttrs;
            cfg.attrs = attrs;
        }
        cfg.gridDim = dim3(static_cast<unsigned>(grid * blocks), c.B, 1);
        cfg.blockDim = dim3(threads, 1, 1);
        cfg.dynamicSmemBytes = dynamic;
        cfg.stream = static_cast<cudaStream_t>(stream);
        return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p));
    };
    const int64_t heads = static_cast<int64_t>(n) * c.Hkv;
    const int rc = p.cluster > 1
                       ? run(evict_select_kernel<true>, heads, kSelectThreads, smem, p.cluster)
                       : run(evict_select_kernel<false>, heads, kSelectThreads, smem, 1);
    if (rc != cudaSuccess) return rc;
    return p.movers > 1
               ? run(evict_move_kernel<true>, heads * 2 * p.slices, kMoveThreads, 0, p.movers)
               : run(evict_move_kernel<false>, heads * 2 * p.slices, kMoveThreads, 0, 1);
}

}  // namespace qmm
